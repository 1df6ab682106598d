// Log probabilities of given tokens, with entropy and top alternatives, and
// their gradient.
#include "lm_rows.cuh"

namespace dpz {

namespace {

// ------------------------------------------------------------ top alternatives
//
// An element's rank key: the value's order in the upper word, the complement
// of its index in the lower, so that the largest key is the largest value of
// the lowest index.  0 is below every key.

constexpr uint32_t kOrderMasked = 0x007fffffu;      // value_order(-inf)

__device__ __forceinline__ float value_of_order(uint32_t o)
{
    return o == 0xffffff00u ? quiet_nan()
                            : __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

__device__ __forceinline__ uint64_t rank_key(uint32_t order, int j)
{
    return (uint64_t)order << 32 | (0xffffffffu - (uint32_t)j);
}

__device__ __forceinline__ uint64_t warp_max64(uint64_t k)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t b = __shfl_xor_sync(0xffffffffu, k, o);
        k = b > k ? b : k;
    }
    return k;
}

// How many of n keys are above this one.
__device__ __forceinline__ int keys_above(const uint64_t* keys, int n, uint64_t key)
{
    int above = 0;
#pragma unroll 8
    for (int q = 0; q < n; ++q) above += keys[q] > key;
    return above;
}

// Where a thread's largest elements are: the order of its largest one (0
// without elements), the first of the `count` vectors that were loaded with
// it, and the order of the largest element elsewhere.
struct ThreadTop {
    uint32_t max, second;
    int best, count;
};

constexpr int kTopCap = 512;                        // candidates a block can hold

// Vectors that a thread loads at once, and keeps of its largest element's
// batch.  Two of fp32 take half the shared memory of four: 1,021 rows of 50,304
// with 20 alternatives 39 us with 2 and 47 with 4; bf16, 4,096 rows of 50,257
// with 8, 88 us with 2 and 82 with 4.
template <int DT>
constexpr int kTopLoads = DT == DPZ_F32 ? 2 : 4;

template <int NT, int LOADS>
struct TopShared {
    uint4 kept[LOADS * NT];                            // each thread's vectors with its largest element
    uint64_t cand[kTopCap];
    uint64_t merged[kMaxCluster * DPZ_LM_MAX_TOP];  // a cluster's first block: every block's best
    uint64_t best[NT / 32];
    uint32_t lane_max[NT / 32][32];                 // each thread's largest
    int2 flag[NT];                                  // threads that reach the threshold
    uint32_t threshold;
    int n, flags;
};

// The statistics of this thread's elements of a slice, and where the largest are.
template <int DT, int NT, bool ENT, bool TOP>
__device__ __forceinline__ Stat thread_stat(const char* row, const Slice& s, const StatScale& k,
                                            ThreadTop* top, uint4* kept)
{
    const int t = threadIdx.x;
    ThreadStat<DT, NT, ENT, TOP> ts;
    constexpr int kLoads = TOP ? kTopLoads<DT> : 4;
    thread_rows<DT, NT, kLoads>(ts, row, s, s.lo + t, k, kept);
    const Stat st = thread_rest<DT>(ts.get(k), row, s, k);
    if (TOP) {
        const bool single = t < s.head || t < s.tail;
        top->max = single || s.lo + t < s.hi ? value_order(st.m) : 0u;
        top->second = single ? top->max : value_order(ts.second);
        top->best = ts.best;
        // the batches of thread_rows
        const int mine = s.hi - s.lo - t, at = (ts.best - s.lo - t) / NT;
        const int n = (mine + NT - 1) / NT - at;
        top->count = n >= kLoads ? kLoads : n >= 2 ? 2 : 1;
    }
    return st;
}

// Calls f(x, j) for each element x of index j that this thread has.
template <int DT, int NT, class F>
__device__ __forceinline__ void for_elements(const char* row, const Slice& s, F&& f)
{
    constexpr int kB = El<DT>::kBytes, kV = El<DT>::kVec;
    const char* body = row + s.vec0 * kB;
    const int t = threadIdx.x;
    for (int i = s.lo + t; i < s.hi; i += NT) {
        float x[kV];
        El<DT>::unpack(ld16(body + (int64_t)i * 16), x);
#pragma unroll
        for (int j = 0; j < kV; ++j) f(x[j], s.vec0 + i * kV + j);
    }
    if (t < s.head) f(El<DT>::load(row + t * kB), t);
    if (t < s.tail) f(El<DT>::load(row + (int64_t)(s.tail0 + t) * kB), s.tail0 + t);
}

// By one warp: the K-th largest of 64 groups' maxima (K <= 32).  A group is the
// threads of one lane in the even or the odd warps.  Elements that lie side by
// side (a vocabulary's frequent tokens come first) are in different lanes, so
// large ones do not crowd in few groups.
template <int NT, int LOADS>
__device__ __forceinline__ void top_threshold(int K, TopShared<NT, LOADS>& sh)
{
    const int lane = threadIdx.x & 31;
    uint32_t a = 0, b = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; w += 2) {
        a = max(a, sh.lane_max[w][lane]);
        b = max(b, sh.lane_max[w + 1][lane]);
    }
    int above_a = 0, above_b = 0;
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {
        const uint32_t x = __shfl_sync(0xffffffffu, a, i), y = __shfl_sync(0xffffffffu, b, i);
        above_a += (x > a || (x == a && i < lane)) + (y > a);
        above_b += (x >= b) + (y > b || (y == b && i < lane));
    }
    if (above_a == K - 1) sh.threshold = a;
    if (above_b == K - 1) sh.threshold = b;
    if (lane == 0) sh.n = sh.flags = 0;
}

// Calls emit(k, key) once for each of the slice's K largest keys (of all, if
// it has fewer elements), k being its rank, from any thread of the block.
//
// The K-th largest of 64 groups' maxima is a threshold that at least K
// elements reach, and few more do: a random row of any length has
// 64 (H(64) - H(64 - K)) of them, 9 for K = 8, 24 for K = 20 and 44 for
// K = 32 (H: harmonic numbers).  Only the elements of threads whose own maximum
// reaches it are looked at again, the warps taking turns with the threads: the
// kept vectors if nothing else of the thread's reaches it, else all of them.
// The candidates are ranked against each other.  If more than kTopCap elements
// reach it (rows of few distinct values), K rounds of a block-wide maximum
// are run instead.  If only masked elements are left below the threshold
// (fewer than K groups have any other), the unmasked ones are candidates and
// the masked ones of lowest index, which are ties, fill up.
template <int DT, int NT, class F>
__device__ __forceinline__ void block_top(const char* row, const Slice& s, const ThreadTop& own,
                                          int K, TopShared<NT, kTopLoads<DT>>& sh, F&& emit)
{
    constexpr int kB = El<DT>::kBytes, kV = El<DT>::kVec;
    static_assert(kTopLoads<DT> * kV <= 32, "one lane per kept element");
    static_assert(2 * DPZ_LM_MAX_TOP <= NT, "one thread per element that fills up");
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const uint32_t th = max(sh.threshold, 1u);
    const bool fill = th <= kOrderMasked;
    const uint32_t least = fill ? kOrderMasked + 1 : th;
    const auto offer = [&](float x, int j) {
        const uint32_t o = value_order(x);
        if (o >= least) {
            const int at = atomicAdd(&sh.n, 1);
            if (at < kTopCap) sh.cand[at] = rank_key(o, j);
        }
    };
    const bool flagged = own.max >= least;
    const unsigned m = __ballot_sync(0xffffffffu, flagged);
    if (m != 0) {
        int at = 0;
        if (lane == 0) at = atomicAdd(&sh.flags, __popc(m));
        at = __shfl_sync(0xffffffffu, at, 0) + __popc(m & ((1u << lane) - 1u));
        if (flagged) sh.flag[at] = make_int2(own.second >= least ? -1 : own.best, threadIdx.x << 3 | own.count);
    }
    __syncthreads();
    for (int q = wid; q < sh.flags; q += NT / 32) {
        const int2 e = sh.flag[q];
        const int t = e.y >> 3, count = e.y & 7;
        if (e.x >= 0) {
            const int l = lane / kV, j = lane % kV;
            if (l < count)
                offer(El<DT>::load(reinterpret_cast<const char*>(&sh.kept[l * NT + t]) + j * kB),
                      s.vec0 + (e.x + l * NT) * kV + j);
            continue;
        }
        for (int i = s.lo + t + lane * NT; i < s.hi; i += 32 * NT) {
            const uint4 v[1] = {ld16(row + s.vec0 * kB + (int64_t)i * 16)};
            if (value_order(El<DT>::vec_max(v)) < least) continue;
            float x[kV];
            El<DT>::unpack(v[0], x);
#pragma unroll
            for (int j = 0; j < kV; ++j) offer(x[j], s.vec0 + i * kV + j);
        }
        if (lane == 0) {
            if (t < s.head) offer(El<DT>::load(row + t * kB), t);
            if (t < s.tail) offer(El<DT>::load(row + (int64_t)(s.tail0 + t) * kB), s.tail0 + t);
        }
    }
    __syncthreads();
    int n = sh.n;
    if (fill && n < K) {
        // masked elements among the slice's first K + n hold the lowest indices
        __syncthreads();
        const int j = s.first + threadIdx.x;
        if ((int)threadIdx.x < K + n && j < s.last &&
            value_order(El<DT>::load(row + (int64_t)j * kB)) == kOrderMasked)
            sh.cand[atomicAdd(&sh.n, 1)] = rank_key(kOrderMasked, j);
        __syncthreads();
        n = sh.n;
    }
    if (n <= kTopCap) {
        for (int i = threadIdx.x; i < n; i += NT) {
            const uint64_t key = sh.cand[i];
            const int above = keys_above(sh.cand, n, key);
            if (above < K) emit(above, key);
        }
        return;
    }
    // K rounds: the largest key below the last one.  Each thread keeps its own
    // best and looks for the next one only when its best was taken.
    uint64_t prev = ~uint64_t(0), best = 0;
    bool stale = true;
    for (int k = 0; k < K; ++k) {
        if (stale) {
            best = 0;
            for_elements<DT, NT>(row, s, [&](float x, int j) {
                const uint64_t key = rank_key(value_order(x), j);
                if (key < prev && key > best) best = key;
            });
        }
        const uint64_t wb = warp_max64(best);
        if (lane == 0) sh.best[wid] = wb;
        __syncthreads();
        prev = warp_max64(lane < NT / 32 ? sh.best[lane] : 0);
        __syncthreads();
        stale = best == prev;
        if (threadIdx.x == 0) emit(k, prev);
    }
}

// ------------------------------------------------------------ log probabilities

// One block, or one cluster of blocks, per row: one pass over the logits.
template <int DT, int NT, bool ENT, bool TOP>
__global__ void __launch_bounds__(NT, (DT == DPZ_F32 ? 7 : 6) * kRowThreads / NT)
    k_logprobs(LogprobArgs a)
{
    __shared__ StatShared<NT> ssh;
    __shared__ TopShared<TOP ? NT : 64, kTopLoads<DT>> tsh;
    __shared__ RowResult s_result;
    const unsigned rank = cluster_rank(), n = cluster_size();
    if (n > 1) cluster_arrive_relaxed();
    pdl_enter();
    const int64_t t = blockIdx.x >> (31 - __clz(n));
    const char* row = a.x.p + t * a.x.ld * El<DT>::kBytes;
    float target = 0.0f;
    int y = -1;
    if (rank == 0 && threadIdx.x == 0 && a.targets.p != nullptr) {
        y = load_token(a.targets, t, a.V);
        if (y >= 0) target = El<DT>::load_now(row + (int64_t)y * El<DT>::kBytes);
    }
    const Slice sl = row_slice<DT>(row, a.V, rank, n);
    const StatScale k(a.scale);
    ThreadTop own;
    const Stat mine = thread_stat<DT, NT, ENT, TOP>(row, sl, k, &own, tsh.kept);
    if constexpr (TOP) {
        tsh.lane_max[threadIdx.x >> 5][threadIdx.x & 31] = own.max;
        if (n > 1 && rank == 0)
            for (unsigned i = threadIdx.x; i < n * a.K; i += NT) tsh.merged[i] = 0;
    }
    const Stat s = row_stat<NT>(mine, k, ssh, rank, n, [&] {
        if constexpr (TOP) top_threshold(a.K, tsh);
    });
    if (rank == 0 && threadIdx.x < 32) {
        const RowResult r = row_result(s, a.scale);
        if (threadIdx.x == 0) {
            if (TOP) s_result = r;          // read after block_top's barrier
            if (a.logprob != nullptr)
                a.logprob[t] = y < 0 ? 0.0f : logprob_of(target, s, r, a.scale);
            if (a.lse != nullptr) a.lse[t] = r.lse;
            if (ENT) a.entropy[t] = r.entropy;
        }
    }
    if constexpr (TOP) {
        const auto write = [&](int at, uint64_t key) {
            const int j = (int)(0xffffffffu - (uint32_t)key);
            const float x = value_of_order((uint32_t)(key >> 32));
            const int64_t o = t * a.K + at;
            if (a.targets.it == DPZ_I64) static_cast<int64_t*>(a.top_ids)[o] = j;
            else static_cast<int*>(a.top_ids)[o] = j;
            a.top_logprobs[o] = logprob_of(x, s, s_result, a.scale);
        };
        if (n == 1) {
            block_top<DT, NT>(row, sl, own, a.K, tsh, write);
            return;
        }
        // every block's best to the first block, which ranks them
        block_top<DT, NT>(row, sl, own, a.K, tsh, [&](int at, uint64_t key) {
            store_rank_u64(&tsh.merged[rank * a.K + at], 0, key);
        });
        cluster_arrive_release();
        cluster_wait();
        if (rank != 0) return;
        for (unsigned i = threadIdx.x; i < n * a.K; i += NT) {
            const uint64_t key = tsh.merged[i];
            const int above = keys_above(tsh.merged, n * a.K, key);
            if (key != 0 && above < a.K) write(above, key);
        }
    }
}

// ------------------------------------------------------------ gradient

// Blocks (row, slice): reads and writes each element once.
template <int DT, int NT>
__global__ void __launch_bounds__(NT) k_logprobs_grad(LogprobGradArgs a)
{
    pdl_enter();
    const unsigned rank = blockIdx.y, n = gridDim.y;
    const int64_t t = blockIdx.x;
    const char* row = a.x.p + t * a.x.ld * El<DT>::kBytes;
    char* out = a.dx.p + t * a.dx.ld * El<DT>::kBytes;
    const int y = load_token(a.targets, t, a.V);
    const float g = y < 0 ? 0.0f : a.dlogprob[t];
    const float h = a.dentropy != nullptr ? a.dentropy[t] : 0.0f;
    const float lse = a.lse[t];
    if ((g == 0.0f && h == 0.0f) || lse == -INFINITY) {
        zero_slice<DT, NT>(out, row_slice<DT>(row, a.V, rank, n));
        return;
    }
    const float H = h != 0.0f ? a.entropy[t] : 0.0f;
    // -p (g + h (log p + H)) = p (A + B log2 p); the exponent is held at a
    // finite value so that a masked element's p = 0 gives 0
    const float A = -__fmaf_rn(h, H, g) * a.scale, B = -h * kLn2 * a.scale;
    const F2 A2 = pack2(A, A), B2 = pack2(B, B), s2 = pack2(a.scale, a.scale);
    const F2 l2 = pack2(-lse, -lse), e2 = pack2(kLog2e, kLog2e);
    const auto d = [&](F2 x) {
        F2 u = mul2(fma2(x, s2, l2), e2);
        u = pack2(max_nan(lo2(u), kMinExp), max_nan(hi2(u), kMinExp));
        return mul2(ex2x2(u), fma2(B2, u, A2));
    };
    const Slice s = row_slice<DT>(row, a.V, rank, n);
    // the target's element has g more
    float at_y = 0.0f;
    const bool mine = g != 0.0f && y >= s.first && y < s.last;
    if (mine && threadIdx.x == 0)
        at_y = lo2(d(pack2(El<DT>::load_now(row + (int64_t)y * El<DT>::kBytes), 0.0f)));
    uint4 w[kMapLoads];
    map_load<DT, NT>(row, s, s.lo + threadIdx.x, w);
    if (mine) __syncthreads();     // in place, before it is overwritten
    map_row<DT, NT>(row, out, s, s.lo + threadIdx.x, w, d);
    if (!mine) return;
    __syncthreads();
    if (threadIdx.x == 0)
        El<DT>::store(out + (int64_t)y * El<DT>::kBytes, __fmaf_rn(g, a.scale, at_y));
}

template <int DT, int NT>
void (*logprobs_kernel(bool ent, bool top))(LogprobArgs)
{
    return ent ? (top ? k_logprobs<DT, NT, true, true> : k_logprobs<DT, NT, true, false>)
               : (top ? k_logprobs<DT, NT, false, true> : k_logprobs<DT, NT, false, false>);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t s)
{
    set_last_kernel_name("lm_logprobs");
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const bool ent = a.entropy != nullptr, top = a.K > 0, b = a.x.dt == DPZ_BF16;
    return by_row_threads(a.T, row_bytes(a.V, a.x.dt), sms, [&](auto threads) {
        constexpr int NT = threads;
        const unsigned n = row_cluster(a.T, row_bytes(a.V, a.x.dt), NT, sms);
        void (*fn)(LogprobArgs) = b ? logprobs_kernel<DPZ_BF16, NT>(ent, top)
                                    : logprobs_kernel<DPZ_F32, NT>(ent, top);
        return launch_kernel(fn, dim3((unsigned)a.T * n), dim3(NT), 0, s, true, n > 1 ? n : 0u, a);
    });
}

cudaError_t launch_logprobs_grad(const LogprobGradArgs& a, cudaStream_t s)
{
    set_last_kernel_name("lm_logprobs_grad");
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    return by_row_threads(a.T, row_bytes(a.V, a.x.dt), sms, [&](auto threads) {
        constexpr int NT = threads;
        const unsigned n = row_cluster(a.T, row_bytes(a.V, a.x.dt), NT, sms);
        return launch_kernel(a.x.dt == DPZ_BF16 ? k_logprobs_grad<DPZ_BF16, NT>
                                                : k_logprobs_grad<DPZ_F32, NT>,
                             dim3((unsigned)a.T, n), dim3(NT), 0, s, true, 0u, a);
    });
}

}  // namespace dpz
