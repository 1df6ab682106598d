// Distillation from a teacher's top logits: loss, gradient, and both in one
// pass over the student's logits.
#include "lm_rows.cuh"

namespace dpz {

namespace {

// The teacher's entries of one row in shared memory: tokens (-1: absent), the
// student's logits there, probabilities and their logarithms.
struct Teacher {
    int id[DPZ_LM_MAX_TEACHER];
    float x[DPZ_LM_MAX_TEACHER], q[DPZ_LM_MAX_TEACHER], logq[DPZ_LM_MAX_TEACHER];
    int any, repeats;   // whether there is an entry; whether two name one token
};

// Hashed sets of tokens, zero between uses, to find repeats without comparing
// every pair of entries.
struct TokenHash {
    uint32_t seen[256], twice[256];
    static __device__ __forceinline__ uint32_t of(int id) { return (uint32_t)id * 2654435761u >> 19; }
};

__device__ __forceinline__ float warp_max_nan(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float warp_sum_all(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Entries that a lane of the warp that has them works on at once, so that their
// loads and latencies overlap.  The warp's work on a row's entries has to fit
// into the others' on the row: the step of 8,192 rows of 32,000 bf16 with 128
// entries takes 275 us with 1 at a time, 260 with 2, 224 with 4 and 254 with 8.
constexpr int kEntries = 4;

// Whether two of the entries name one token, by one warp: entries whose hash
// another entry has too are compared with all of them.
__device__ __forceinline__ bool find_repeats(const int* id, int K, TokenHash& h)
{
    const int lane = threadIdx.x & 31;
    __syncwarp();
    bool twice = false;
    for (int k0 = lane; k0 < K; k0 += 32 * kEntries) {
        uint32_t b[kEntries], was[kEntries];
#pragma unroll
        for (int l = 0; l < kEntries; ++l) {
            const int v = k0 + 32 * l < K ? id[k0 + 32 * l] : -1;
            b[l] = TokenHash::of(v);
            was[l] = v < 0 ? 0u : atomicOr(&h.seen[b[l] >> 5], 1u << (b[l] & 31));
        }
#pragma unroll
        for (int l = 0; l < kEntries; ++l)
            if (was[l] >> (b[l] & 31) & 1) {
                twice = true;
                atomicOr(&h.twice[b[l] >> 5], 1u << (b[l] & 31));
            }
    }
    twice = __any_sync(0xffffffffu, twice);
    __syncwarp();
    bool found = false;
    for (int k0 = 0; twice && k0 < K; k0 += 32) {
        const int v = k0 + lane < K ? id[k0 + lane] : -1;
        const uint32_t b = TokenHash::of(v);
        unsigned m = __ballot_sync(0xffffffffu, v >= 0 && (h.twice[b >> 5] >> (b & 31) & 1));
        while (m != 0) {
            const int u = __shfl_sync(0xffffffffu, v, __ffs(m) - 1);
            m &= m - 1;
            int same = 0;
            for (int i = lane; i < K; i += 32) same += id[i] == u;
            found |= __reduce_add_sync(0xffffffffu, same) > 1;
        }
    }
    __syncwarp();
    for (int k = lane; k < K; k += 32)
        if (id[k] >= 0) h.seen[TokenHash::of(id[k]) >> 5] = h.twice[TokenHash::of(id[k]) >> 5] = 0;
    __syncwarp();
    return found;
}

__device__ __forceinline__ void clear_hash(TokenHash& h)
{
    for (int i = threadIdx.x & 31; i < 256; i += 32) h.seen[i] = h.twice[i] = 0;
}

// One warp loads a row's entries and their softmax; the student's logits of
// those in [lo, hi).
template <int DT>
__device__ __forceinline__ void load_teacher(const DistillArgs& a, int64_t t, const char* row,
                                             int lo, int hi, Teacher& w)
{
    const int lane = threadIdx.x & 31;
    float m = -INFINITY;
    for (int k0 = lane; k0 < a.K; k0 += 32 * kEntries) {
        int id[kEntries];
        float v[kEntries], x[kEntries];
#pragma unroll
        for (int l = 0; l < kEntries; ++l) {
            const int64_t at = t * a.K + k0 + 32 * l;
            id[l] = -1;
            v[l] = -INFINITY;
            if (k0 + 32 * l < a.K) {
                id[l] = load_token(a.ids, at, a.V);
                v[l] = a.teacher.dt == DPZ_F32 ? El<DPZ_F32>::load(a.teacher.p + at * 4)
                                               : El<DPZ_BF16>::load(a.teacher.p + at * 2);
            }
        }
#pragma unroll
        for (int l = 0; l < kEntries; ++l)
            x[l] = id[l] < max(lo, 0) || id[l] >= hi ? 0.0f
                                             : El<DT>::load(row + (int64_t)id[l] * El<DT>::kBytes);
#pragma unroll
        for (int l = 0; l < kEntries; ++l) {
            const int k = k0 + 32 * l;
            if (k >= a.K) break;
            if (v[l] == -INFINITY) id[l] = -1;
            if (id[l] < 0) v[l] = -INFINITY;
            w.id[k] = id[l];
            w.x[k] = x[l];
            w.logq[k] = v[l];
            m = max_nan(m, v[l]);
        }
    }
    m = warp_max_nan(m);
    float S = 0.0f;
    for (int k0 = lane; k0 < a.K; k0 += 32 * kEntries) {
        float v[kEntries];
#pragma unroll
        for (int l = 0; l < kEntries; ++l) {
            const int k = k0 + 32 * l;
            v[l] = k < a.K ? w.logq[k] : -INFINITY;
        }
#pragma unroll
        for (int l = 0; l < kEntries; ++l) {
            // the difference before the product: the type's lowest value stays finite
            if (v[l] != -INFINITY) {
                v[l] = (v[l] - m) * a.inv_tau;
                S += expf(v[l]);
            }
        }
    }
    S = warp_sum_all(S);
    const float logS = logf(S);
    for (int k0 = lane; k0 < a.K; k0 += 32 * kEntries) {
        float v[kEntries];
#pragma unroll
        for (int l = 0; l < kEntries; ++l) {
            const int k = k0 + 32 * l;
            v[l] = k < a.K ? w.logq[k] : -INFINITY;
        }
#pragma unroll
        for (int l = 0; l < kEntries; ++l) {
            const int k = k0 + 32 * l;
            if (k >= a.K) break;
            const bool none = v[l] == -INFINITY;
            if (!none) v[l] = (v[l] - m) * a.inv_tau - logS;
            w.logq[k] = v[l];
            w.q[k] = none ? 0.0f : expf(v[l]);
        }
    }
    if (lane == 0) w.any = m != -INFINITY;
    __syncwarp();
}

// By one warp: sum_k q_k (log q_k - log p_k), in a fixed order; lane 0 writes.
__device__ __forceinline__ void write_loss(const DistillArgs& a, int64_t t, const Teacher& w,
                                           const Stat& s, const RowResult& r)
{
    const int lane = threadIdx.x & 31;
    float sum = 0.0f;
    for (int i0 = lane; i0 < a.K; i0 += 32 * kEntries) {
        float q[kEntries], d[kEntries];
#pragma unroll
        for (int l = 0; l < kEntries; ++l) {
            const int i = min(i0 + 32 * l, a.K - 1);
            q[l] = i0 + 32 * l < a.K ? w.q[i] : 0.0f;
            d[l] = w.logq[i] - logprob_of(w.x[i], s, r, a.inv_tau);
        }
#pragma unroll
        for (int l = 0; l < kEntries; ++l)
            if (q[l] != 0.0f) sum += q[l] * d[l];
    }
    sum = warp_sum_all(sum);
    if (lane == 0) {
        a.loss[t] = w.any ? sum : 0.0f;
        if (a.lse != nullptr) a.lse[t] = r.lse;
    }
}

// The gradient without the teacher's part: (w / tau) p, in pairs.  From lse:
struct StudentGrad {
    F2 it, l, e, ws;
    __device__ __forceinline__ StudentGrad(float inv_tau, float lse, float weight)
        : it(pack2(inv_tau, inv_tau)), l(pack2(-lse, -lse)), e(pack2(kLog2e, kLog2e)),
          ws(pack2(weight, weight))
    {
    }
    __device__ __forceinline__ F2 p(F2 x) const { return ex2x2(mul2(fma2(x, it, l), e)); }
    __device__ __forceinline__ F2 operator()(F2 x) const { return mul2(ws, p(x)); }
};

// From the row's statistics, p = 2^((x - m) c - log2 S): lse, which holds a
// large m's sum only to 2^-24 of it, is not passed through.
struct StepGrad {
    F2 m, c, l, ws;
    __device__ __forceinline__ StepGrad(const StatScale& k, const Stat& s, const RowResult& r,
                                        float weight)
        : m(pack2(-s.m, -s.m)), c(pack2(k.c, k.c)), l(pack2(-r.log2S, -r.log2S)),
          ws(pack2(weight, weight))
    {
    }
    __device__ __forceinline__ F2 p(F2 x) const { return ex2x2(fma2(add2(x, m), c, l)); }
    __device__ __forceinline__ F2 operator()(F2 x) const { return mul2(ws, p(x)); }
};

// The same for a bf16 result with w > 0 and |m c| up to 2^10, with everything
// in one exponent: 2^(x c + log2(w / tau) - log2 S - m c).  The roundings of m c
// and of the constant, below 2^11, are at most 2^-13 together, a fiftieth of
// the result's own half unit (2^-9 to 2^-8).
struct StepGradExp {
    F2 c, b;
    __device__ __forceinline__ StepGradExp(const StatScale& k, const Stat& s, const RowResult& r,
                                           float weight)
    {
        const float bb = (log2f(weight) - r.log2S) - s.m * k.c;
        c = pack2(k.c, k.c);
        b = pack2(bb, bb);
    }
    static __device__ __forceinline__ bool holds(int DT, const StatScale& k, const Stat& s,
                                                 float weight)
    {
        return DT == DPZ_BF16 && weight > 0.0f && fabsf(s.m * k.c) <= 1024.0f;
    }
    __device__ __forceinline__ F2 operator()(F2 x) const { return ex2x2(fma2(x, c, b)); }
};

// The elements of the teacher's tokens in a slice again, now with their q, by
// one warp.  An entry that repeats an earlier one's token leaves it to that one.
template <int DT, class F>
__device__ __forceinline__ void write_teacher_part(const DistillArgs& a, const Teacher& w,
                                                   const Slice& s, const F& f, char* out)
{
    const int lane = threadIdx.x & 31;
    const auto value = [&](float x, float q) { return lo2(f.ws) * (lo2(f.p(pack2(x, 0.0f))) - q); };
    if (!w.repeats) {
        for (int i0 = lane; i0 < a.K; i0 += 32 * kEntries) {
            int id[kEntries];
            float d[kEntries];
#pragma unroll
            for (int l = 0; l < kEntries; ++l) {
                const int i = min(i0 + 32 * l, a.K - 1);
                id[l] = i0 + 32 * l < a.K ? w.id[i] : -1;
                d[l] = value(w.x[i], w.q[i]);
            }
#pragma unroll
            for (int l = 0; l < kEntries; ++l)
                if (id[l] >= s.first && id[l] < s.last)
                    El<DT>::store(out + (int64_t)id[l] * El<DT>::kBytes, d[l]);
        }
        return;
    }
    for (int i = lane; i < a.K; i += 32) {
        const int id = w.id[i];
        if (id < s.first || id >= s.last) continue;
        float q = 0.0f;
        bool once = true;
        for (int j = 0; j < a.K; ++j)
            if (w.id[j] == id) {
                if (j < i) once = false;
                q += w.q[j];
            }
        if (once) El<DT>::store(out + (int64_t)id * El<DT>::kBytes, value(w.x[i], q));
    }
}

// The statistics of this thread's elements of a slice.
template <int DT, int NT>
__device__ __forceinline__ Stat slice_stat(const char* row, const Slice& sl, const StatScale& k)
{
    RefStat<DT> rs;
    thread_rows<DT, NT>(rs, row, sl, sl.lo + threadIdx.x, k);
    Stat own = rs.get(k);
    if (!rs.good()) {
        ThreadStat<DT, NT, false, false> ts;
        thread_rows<DT, NT>(ts, row, sl, sl.lo + threadIdx.x, k);
        own = ts.get(k);
    }
    return thread_rest<DT>(own, row, sl, k);
}

// ------------------------------------------------------------ loss alone

// A row per block (or cluster) of NT threads, and a warp more that loads the
// entries meanwhile.
template <int DT, int NT>
__global__ void __launch_bounds__(NT + 32, kLossBlocks<DT, NT>) k_distill(DistillArgs a)
{
    __shared__ Teacher w;
    __shared__ StatShared<NT> ssh;
    const unsigned rank = cluster_rank(), n = cluster_size();
    if (n > 1) cluster_arrive_relaxed();
    pdl_enter();
    const int64_t t = blockIdx.x >> (31 - __clz(n));
    const char* row = a.x.p + t * a.x.ld * El<DT>::kBytes;
    const StatScale k(a.inv_tau);
    if (threadIdx.x >= NT) {
        if (rank == 0) load_teacher<DT>(a, t, row, 0, a.V, w);
        row_stat_beside(k, ssh, n);
        return;
    }
    const Slice sl = row_slice<DT>(row, a.V, rank, n);
    const Stat s = row_stat<NT>(slice_stat<DT, NT>(row, sl, k), k, ssh, rank, n, [] {});
    if (rank == 0 && threadIdx.x < 32) write_loss(a, t, w, s, row_result(s, a.inv_tau));
}

// ------------------------------------------------------------ gradient alone

// Blocks (row, slice) of NT threads, and a warp more that loads the entries
// meanwhile.  In place the others wait for it before they write, since it
// reads logits; otherwise they do not, and a row that turns out to have no
// entry is written again.
template <int DT, int NT>
__global__ void __launch_bounds__(NT + 32, kGradBlocks<NT>) k_distill_grad(DistillArgs a)
{
    __shared__ Teacher w;
    __shared__ TokenHash hash;
    pdl_enter();
    const unsigned rank = blockIdx.y, n = gridDim.y;
    const int64_t t = blockIdx.x;
    const char* row = a.x.p + t * a.x.ld * El<DT>::kBytes;
    char* out = a.dx.p + t * a.dx.ld * El<DT>::kBytes;
    const bool in_place = row == out;
    const Slice sl = row_slice<DT>(row, a.V, rank, n);
    const float wt = a.dloss[t], lse = a.lse_in[t];
    if (wt == 0.0f || lse == -INFINITY) {
        if (threadIdx.x < NT) zero_slice<DT, NT>(out, sl);
        return;
    }
    const StudentGrad f(a.inv_tau, lse, wt * a.inv_tau);
    if (threadIdx.x >= NT) {
        clear_hash(hash);
        // other blocks' slices may be overwritten already
        load_teacher<DT>(a, t, row, sl.first, sl.last, w);
        const bool repeats = find_repeats(w.id, a.K, hash);
        if (threadIdx.x == NT) w.repeats = repeats;
        if (in_place) __syncthreads();
        __syncthreads();
        if (w.any) write_teacher_part<DT>(a, w, sl, f, out);
        return;
    }
    uint4 v[kMapLoads];
    map_load<DT, NT>(row, sl, sl.lo + threadIdx.x, v);
    if (in_place) __syncthreads();
    map_row<DT, NT>(row, out, sl, sl.lo + threadIdx.x, v, f);
    __syncthreads();
    if (!w.any) zero_slice<DT, NT>(out, sl);
}

// ------------------------------------------------------------ both in one pass
//
// The row (or the slice of a cluster's block) stays in shared memory between
// the statistics and the gradient, so the logits are read from memory once.
// Each thread copies its own vectors asynchronously and is the only one to use
// them, so nothing but its own copies is waited for.  What does not fit is
// read again, from L2 as a rule.
//
// Blocks are persistent and take every gridDim-th row.  As a vector's gradient
// is written, the copy of the next row's vector into its place begins, so
// loads go on while the block computes and writes.  One more warp, the
// teacher's, works beside the NT threads: it loads the next row's entries
// while the others are at this one, computes the loss, and writes the teacher's
// tokens' gradients once the others have written theirs.
constexpr int kStageGroups = 4;    // copies are waited for in this many parts

__device__ __forceinline__ void copy_async16(void* sdst, const void* gsrc)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(smem_addr(sdst)), "l"(gsrc)
                 : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int LEFT>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// Barriers of the block: 0 (__syncthreads) once per row, when the threads'
// statistics and the teacher's entries are there; kRowWritten when the
// gradient is written but for the teacher's tokens, which only the teacher's
// warp waits for.
constexpr int kRowWritten = 1;

template <int N>
__device__ __forceinline__ void barrier_arrive()
{
    __threadfence_block();
    asm volatile("barrier.cta.arrive %0, %1;" ::"n"(kRowWritten), "n"(N) : "memory");
}

template <int N>
__device__ __forceinline__ void barrier_wait()
{
    asm volatile("barrier.cta.sync %0, %1;" ::"n"(kRowWritten), "n"(N) : "memory");
}

// A row's statistics from the warps' (and in a cluster the blocks') parts; by
// whole warps, every thread of the block and cluster taking part.
template <int NT>
__device__ __forceinline__ Stat step_stat(const StatScale& k, StatShared<NT>& sh, unsigned rank,
                                          unsigned n)
{
    const int lane = threadIdx.x & 31;
    Stat s = warp_stat(lane < NT / 32 ? sh.warp[lane] : Stat{-INFINITY, 0.0f, 0.0f}, k);
    if (n == 1) return s;
    if (threadIdx.x < n) {
        store_rank_f32(&sh.block[rank].m, threadIdx.x, s.m);
        store_rank_f32(&sh.block[rank].S, threadIdx.x, s.S);
        store_rank_f32(&sh.block[rank].U, threadIdx.x, s.U);
    }
    __syncwarp();
    cluster_arrive_release();
    cluster_wait();
    s = sh.block[0];
    for (unsigned r = 1; r < n; ++r) s = stat_join(s, sh.block[r], k);
    return s;
}

template <int DT, int NT>
__global__ void __launch_bounds__(NT + 32, kStepBlocks) k_distill_step(DistillArgs a, int stage)
{
    extern __shared__ uint4 staged[];           // [stage][NT]
    __shared__ Teacher w[2];                    // this row's and the next one's
    __shared__ StatShared<NT> ssh[2];           // a warp may be one row ahead
    __shared__ TokenHash hash;
    constexpr int kB = El<DT>::kBytes;
    const unsigned rank = cluster_rank(), n = cluster_size();
    if (n > 1) cluster_arrive_relaxed();
    pdl_enter();
    if (n > 1) cluster_wait();
    const int log_n = 31 - __clz(n);
    const int64_t step = gridDim.x >> log_n;
    int64_t t = blockIdx.x >> log_n;
    const StatScale k(a.inv_tau);
    const auto row_of = [&](int64_t r) { return a.x.p + r * a.x.ld * kB; };
    int b = 0;

    if (threadIdx.x >= NT) {                    // the teacher's warp
        clear_hash(hash);
        const auto load = [&](int64_t r, Teacher& e) {
            load_teacher<DT>(a, r, row_of(r), 0, a.V, e);
            const bool repeats = find_repeats(e.id, a.K, hash);
            if (threadIdx.x == NT) e.repeats = repeats;
            __syncwarp();
        };
        load(t, w[0]);
        for (; t < a.T; t += step, b ^= 1) {
            const float wt = a.dloss[t];
            __syncthreads();
            const Stat s = step_stat<NT>(k, ssh[b], rank, n);
            const RowResult r = row_result(s, a.inv_tau);
            if (rank == 0) write_loss(a, t, w[b], s, r);
            if (t + step < a.T) load(t + step, w[b ^ 1]);
            barrier_wait<NT + 32>();
            if (wt == 0.0f || !w[b].any || r.lse == -INFINITY) continue;
            write_teacher_part<DT>(a, w[b], row_slice<DT>(row_of(t), a.V, rank, n),
                                   StepGrad(k, s, r, wt * a.inv_tau),
                                   a.dx.p + t * a.dx.ld * kB);
        }
        return;
    }

    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int per = (stage + kStageGroups - 1) / kStageGroups;
    uint4* own = staged + threadIdx.x;
    // the row at hand: its slice, this thread's first vector, and how many of
    // its vectors are staged
    const char* row = row_of(t);
    Slice sl = row_slice<DT>(row, a.V, rank, n);
    const auto first_of = [&](const Slice& s) { return s.lo + (int)threadIdx.x; };
    const auto staged_of = [&](const Slice& s) {
        return min(stage, max(0, (s.hi - first_of(s) + NT - 1) / NT));
    };
    {
        const int have = staged_of(sl);
        const char* p = row + sl.vec0 * kB + (int64_t)first_of(sl) * 16;
        for (int g = 0; g < kStageGroups; ++g) {
            for (int i = g * per; i < min((g + 1) * per, have); ++i)
                copy_async16(own + i * NT, p + i * (NT * 16));
            copy_commit();
        }
    }
    for (; t < a.T; t += step, b ^= 1) {
        const float wt = a.dloss[t];
        const int first = first_of(sl), have = staged_of(sl);
        RefStat<DT> rs;
        const auto add_group = [&](int g) {
            int i = g * per;
            const int end = min((g + 1) * per, have);
            for (; i + 3 < end; i += 4) {
                const uint4 v[4] = {own[i * NT], own[(i + 1) * NT], own[(i + 2) * NT],
                                    own[(i + 3) * NT]};
                rs.add(v, 0, k, nullptr);
            }
#pragma unroll 1
            for (; i < end; ++i) {
                const uint4 v[1] = {own[i * NT]};
                rs.add(v, 0, k, nullptr);
            }
        };
#pragma unroll 1
        for (int g = 0; g < kStageGroups; ++g) {
            if (g == 0) copy_wait<3>();
            else if (g == 1) copy_wait<2>();
            else if (g == 2) copy_wait<1>();
            else copy_wait<0>();
            add_group(g);
        }
        thread_rows<DT, NT>(rs, row, sl, first + have * NT, k);
        Stat mine = rs.get(k);
        if (!rs.good()) {
            ThreadStat<DT, NT, false, false> ts;
#pragma unroll 1
            for (int i = 0; i < have; ++i) {
                const uint4 v[1] = {own[i * NT]};
                ts.add(v, 0, k, nullptr);
            }
            thread_rows<DT, NT>(ts, row, sl, first + have * NT, k);
            mine = ts.get(k);
        }
        mine = warp_stat(thread_rest<DT>(mine, row, sl, k), k);
        if (lane == 0) ssh[b].warp[wid] = mine;
        __syncthreads();
        const Stat s = step_stat<NT>(k, ssh[b], rank, n);
        const RowResult r = row_result(s, a.inv_tau);
        char* out = a.dx.p + t * a.dx.ld * kB;
        const bool same = same_alignment(row, out);
        const bool zero = wt == 0.0f || !w[b].any || r.lse == -INFINITY;
        char* q = out + sl.vec0 * kB + (int64_t)first * 16;
        // the next row's copies take the places as they become free
        const bool more = t + step < a.T;
        const char* next = more ? row_of(t + step) : row;
        const Slice ns = row_slice<DT>(next, a.V, rank, n);
        const int will = more ? staged_of(ns) : 0;
        const char* np = next + ns.vec0 * kB + (int64_t)first_of(ns) * 16;
        // all of a row's elements in one form, whichever rows are beside it
        const StepGrad f(k, s, r, wt * a.inv_tau);
        const StepGradExp fe(k, s, r, wt * a.inv_tau);
        const bool exp = StepGradExp::holds(DT, k, s, wt * a.inv_tau);
        const auto form = [&](F2 x) { return exp ? fe(x) : f(x); };
        const int fast = same && !zero && exp ? have : 0;   // vectors written without more checks
#pragma unroll 1
        for (int g = 0; g < kStageGroups; ++g) {
            int i = g * per;
            const int end = min(i + per, max(have, will));
#pragma unroll 4
            for (; i < min(end, fast); ++i) {
                map_vector<DT, false>(own[i * NT], q + i * (NT * 16), true, fe);
                if (i < will) copy_async16(own + i * NT, np + i * (NT * 16));
            }
#pragma unroll 1
            for (; i < end; ++i) {
                if (i < have && !zero)
                    map_vector<DT, false>(own[i * NT], q + i * (NT * 16), same, form);
                if (i < will) copy_async16(own + i * NT, np + i * (NT * 16));
            }
            copy_commit();
        }
        if (zero) zero_slice<DT, NT>(out, sl);
        else {
            uint4 v[kMapLoads];
            map_load<DT, NT>(row, sl, first + have * NT, v);
            map_row<DT, NT>(row, out, sl, first + have * NT, v, form);
        }
        barrier_arrive<NT + 32>();
        row = next;
        sl = ns;
    }
}

// The same for short rows: a block (or cluster) per row, which reads it twice,
// the second time from L1 or L2.  Enough blocks are resident to load while
// others compute, without a row ahead.
template <int DT, int NT>
__global__ void __launch_bounds__(NT + 32, kRereadBlocks<NT>) k_distill_step_reread(DistillArgs a)
{
    __shared__ Teacher w;
    __shared__ StatShared<NT> ssh;
    __shared__ TokenHash hash;
    const unsigned rank = cluster_rank(), n = cluster_size();
    if (n > 1) cluster_arrive_relaxed();
    pdl_enter();
    const int64_t t = blockIdx.x >> (31 - __clz(n));
    const char* row = a.x.p + t * a.x.ld * El<DT>::kBytes;
    char* out = a.dx.p + t * a.dx.ld * El<DT>::kBytes;
    const float wt = a.dloss[t];
    const StatScale k(a.inv_tau);
    const Slice sl = row_slice<DT>(row, a.V, rank, n);
    if (threadIdx.x >= NT) {
        clear_hash(hash);
        load_teacher<DT>(a, t, row, 0, a.V, w);
        const bool repeats = find_repeats(w.id, a.K, hash);
        if (threadIdx.x == NT) w.repeats = repeats;
        const Stat s = row_stat_beside(k, ssh, n);
        const RowResult r = row_result(s, a.inv_tau);
        if (rank == 0) write_loss(a, t, w, s, r);
        barrier_wait<NT + 32>();
        if (wt == 0.0f || !w.any || r.lse == -INFINITY) return;
        write_teacher_part<DT>(a, w, sl, StepGrad(k, s, r, wt * a.inv_tau), out);
        return;
    }
    const Stat s = row_stat<NT>(slice_stat<DT, NT>(row, sl, k), k, ssh, rank, n, [] {});
    const RowResult r = row_result(s, a.inv_tau);
    if (wt == 0.0f || !w.any || r.lse == -INFINITY) zero_slice<DT, NT>(out, sl);
    else {
        const int first = sl.lo + threadIdx.x;
        uint4 v[kMapLoads];
        map_load<DT, NT>(row, sl, first, v);
        if (StepGradExp::holds(DT, k, s, wt * a.inv_tau))
            map_row<DT, NT>(row, out, sl, first, v, StepGradExp(k, s, r, wt * a.inv_tau));
        else
            map_row<DT, NT>(row, out, sl, first, v, StepGrad(k, s, r, wt * a.inv_tau));
    }
    barrier_arrive<NT + 32>();
}

// Blocks of a persistent kernel that fit on the current device together, by the
// vectors each thread stages; asked for once.
template <int DT, int NT>
cudaError_t resident_blocks(int stage, int sms, int* blocks)
{
    static PerDevice<kStageMax / (NT * 16) + 1> known;
    return known.get(stage, blocks, [&](int, int* n) {
        int per_sm = 0;
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
            &per_sm, k_distill_step<DT, NT>, NT + 32, (size_t)stage * NT * 16);
        *n = std::max(1, sms * per_sm);
        return e;
    });
}

template <int DT, int NT>
cudaError_t launch_step(const DistillArgs& a, int sms, cudaStream_t s)
{
    static SmemRaisedOn raised;
    const int64_t bytes = row_bytes(a.V, DT);
    // two blocks where one cannot stage a row (4,096 rows of 50,257 fp32: 299 us,
    // 342 with one block that reads half of the row again; 2,048 of 128,256 bf16:
    // 216 and 238; with four blocks 350, their barriers being more than that)
    const unsigned n = std::max(row_cluster(a.T, bytes, NT, sms), bytes > kStageMax ? 2u : 1u);
    const int64_t vecs = (bytes / 16 + n - 1) / n + 1;
    const int stage = (int)std::min<int64_t>((vecs + NT - 1) / NT, kStageMax / (NT * 16));
    cudaError_t e =
        raise_smem(raised, reinterpret_cast<const void*>(k_distill_step<DT, NT>), kStageMax);
    int blocks = 0;
    if (e == cudaSuccess) e = resident_blocks<DT, NT>(stage, sms, &blocks);
    if (e != cudaSuccess) return e;
    const unsigned grid = n * (unsigned)std::min<int64_t>(a.T, std::max(1u, blocks / n));
    return launch_kernel(k_distill_step<DT, NT>, dim3(grid), dim3(NT + 32), (size_t)stage * NT * 16, s,
                         true, n > 1 ? n : 0u, a, stage);
}

template <int DT>
cudaError_t step_typed(const DistillArgs& a, int sms, cudaStream_t s)
{
    const int64_t bytes = row_bytes(a.V, DT);
    if (bytes > kMidRow) return launch_step<DT, kStepThreads>(a, sms, s);
    return by_row_threads(a.T, bytes, sms, [&](auto threads) {
        constexpr int NT = threads;
        const unsigned n = row_cluster(a.T, bytes, NT, sms);
        return launch_kernel(k_distill_step_reread<DT, NT>, dim3((unsigned)a.T * n), dim3(NT + 32), 0,
                             s, true, n > 1 ? n : 0u, a);
    });
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t s)
{
    const bool b = a.x.dt == DPZ_BF16;
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    if (a.loss != nullptr && a.dx.p != nullptr) {
        set_last_kernel_name("lm_distill_step");
        return b ? step_typed<DPZ_BF16>(a, sms, s) : step_typed<DPZ_F32>(a, sms, s);
    }
    const int64_t bytes = row_bytes(a.V, a.x.dt);
    set_last_kernel_name(a.loss != nullptr ? "lm_distill" : "lm_distill_grad");
    return by_row_threads(a.T, bytes, sms, [&](auto threads) {
        constexpr int NT = threads;
        unsigned n = row_cluster(a.T, bytes, NT, sms);
        if (a.loss != nullptr)
            return launch_kernel(b ? k_distill<DPZ_BF16, NT> : k_distill<DPZ_F32, NT>,
                                 dim3((unsigned)a.T * n), dim3(NT + 32), 0, s, true, n > 1 ? n : 0u,
                                 a);
        // two independent blocks per row share the last wave better than one
        // (1,000 rows of 32,000 fp32: 41.4 us, 45.7 with one).  Four blocks take
        // 40.8 there, but each loads the entries again, which shorter rows pay
        // for: 8,192 rows of 16,000 bf16 take 82 us with two blocks of 256
        // threads and 80 with one of 128.
        if (bytes > kMidRow) n = std::max(n, 2u);
        return launch_kernel(b ? k_distill_grad<DPZ_BF16, NT> : k_distill_grad<DPZ_F32, NT>,
                             dim3((unsigned)a.T, n), dim3(NT + 32), 0, s, true, 0u, a);
    });
}

}  // namespace dpz
