// Rows of logits over a vocabulary: log probabilities of given tokens with
// entropy and top alternatives, distillation from a teacher's top logits, and
// the gradients of both.
#include <cfloat>
#include <cmath>

#include "bulk.cuh"
#include "device.cuh"
#include "internal.h"
#include "lm.h"

namespace dpz {

namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kRowLoads = 4;         // vectors a thread loads at once (then 2, then 1)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int load_token(const Ids& ids, int64_t i, int64_t V)
{
    const int64_t v = ids.it == DPZ_I64 ? static_cast<const int64_t*>(ids.p)[i]
                                        : (int64_t) static_cast<const int*>(ids.p)[i];
    return v >= 0 && v < V ? (int)v : -1;
}

// 2^u by the hardware's instruction: at most 2 units in the last place off,
// which is below the rounding of the exponent that it is given here.
__device__ __forceinline__ float ex2(float u)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(u));
    return e;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// fp32 values as integers of the same order: -0 equals +0, NaN is highest, and
// 0 is below every value's.
__device__ __forceinline__ uint32_t value_order(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);   // -0 becomes +0
    return x != x ? 0xffffff00u : b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Two floats in one register pair, for the paired fp32 operations (sm_100 and
// later): each half is rounded as the single operation rounds it, and one
// instruction is issued instead of two.
using F2 = uint64_t;

__device__ __forceinline__ F2 pack2(float lo, float hi)
{
    F2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}

__device__ __forceinline__ float lo2(F2 a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float hi2(F2 a) { return __uint_as_float((uint32_t)(a >> 32)); }

__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

// ------------------------------------------------------------ a row's elements
//
// A row may begin at any element (a vocabulary of 50,257 shifts each row), so
// it is a head of single elements up to the first 16-byte boundary, a body of
// 16-byte vectors, and a tail.

template <int DT>
struct El;

template <>
struct El<DPZ_F32> {
    static constexpr int kBytes = 4, kVec = 4;
    static __device__ __forceinline__ float load(const char* p)
    {
        return *reinterpret_cast<const float*>(p);
    }
    // the same, not to be moved to where its value is used
    static __device__ __forceinline__ float load_now(const char* p)
    {
        float x;
        asm volatile("ld.global.f32 %0, [%1];" : "=f"(x) : "l"(p));
        return x;
    }
    static __device__ __forceinline__ void store(char* p, float x)
    {
        *reinterpret_cast<float*>(p) = x;
    }
    static __device__ __forceinline__ void unpack(const uint4& w, float x[kVec])
    {
        x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float x[kVec])
    {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
    // The largest of N vectors, NaN if any is.
    template <int N>
    static __device__ __forceinline__ float vec_max(const uint4 (&w)[N])
    {
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float x[kVec];
            unpack(w[k], x);
            m = max_nan(m, max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3])));
        }
        return m;
    }
    // Pairs of elements, none below `low`.
    static __device__ __forceinline__ void pairs_above(const uint4& w, float low, F2 (&x)[kVec / 2])
    {
        const auto at = [&](uint32_t u) { return fmaxf(__uint_as_float(u), low); };
        x[0] = pack2(at(w.x), at(w.y));
        x[1] = pack2(at(w.z), at(w.w));
    }
};

template <>
struct El<DPZ_BF16> {
    static constexpr int kBytes = 2, kVec = 8;
    static __device__ __forceinline__ float load(const char* p)
    {
        return __uint_as_float((uint32_t)*reinterpret_cast<const unsigned short*>(p) << 16);
    }
    static __device__ __forceinline__ float load_now(const char* p)
    {
        unsigned short u;
        asm volatile("ld.global.u16 %0, [%1];" : "=h"(u) : "l"(p));
        return __uint_as_float((uint32_t)u << 16);
    }
    static __device__ __forceinline__ void store(char* p, float x)
    {
        *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(x);
    }
    static __device__ __forceinline__ void unpack(const uint4& w, float x[kVec])
    {
        Group<1>::unpack({w}, x);
    }
    static __device__ __forceinline__ uint4 pack(const float x[kVec])
    {
        return Group<1>::pack(x).w;
    }
    static __device__ __forceinline__ __nv_bfloat162 pair(uint32_t u)
    {
        return *reinterpret_cast<const __nv_bfloat162*>(&u);
    }
    // The largest of N vectors, NaN if any is (paired bf16 comparisons).
    template <int N>
    static __device__ __forceinline__ float vec_max(const uint4 (&w)[N])
    {
        __nv_bfloat162 m = pair(0xff80ff80u);   // -inf
#pragma unroll
        for (int k = 0; k < N; ++k)
            m = __hmax2_nan(m, __hmax2_nan(__hmax2_nan(pair(w[k].x), pair(w[k].y)),
                                           __hmax2_nan(pair(w[k].z), pair(w[k].w))));
        return max_nan(__low2float(m), __high2float(m));
    }
    // Pairs of elements, none below `low`.
    static __device__ __forceinline__ void pairs_above(const uint4& w, float low, F2 (&x)[kVec / 2])
    {
        const __nv_bfloat162 l = __float2bfloat162_rn(low);
        const auto at = [&](uint32_t u) {
            const __nv_bfloat162 m = __hmax2(pair(u), l);
            const uint32_t v = *reinterpret_cast<const uint32_t*>(&m);
            return pack2(bf16_lo(v), bf16_hi(v));
        };
        x[0] = at(w.x);
        x[1] = at(w.y);
        x[2] = at(w.z);
        x[3] = at(w.w);
    }
};

struct RowSpan {
    int head;      // elements before the first 16-byte boundary
    int nvec;      // 16-byte vectors
    int tail;      // elements after the last
};

template <int DT>
__device__ __forceinline__ RowSpan row_span(const char* p, int V)
{
    constexpr int kB = El<DT>::kBytes, kV = El<DT>::kVec;
    const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15);
    RowSpan s;
    s.head = min(V, ((16 - off) & 15) / kB);
    s.nvec = (V - s.head) / kV;
    s.tail = V - s.head - s.nvec * kV;
    return s;
}

// ------------------------------------------------------------ a row in slices
//
// A row is taken by a thread-block cluster of C blocks (C = 1: a plain
// block), each with an equal share of the body's vectors; the first block has
// the head too and the last one the tail.  Thread i of a block has the
// vectors lo + i, lo + i + kRowThreads, ...

__device__ __forceinline__ unsigned cluster_rank()
{
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ unsigned cluster_size()
{
    unsigned n;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}

__device__ __forceinline__ uint32_t addr_of_rank(const void* p, unsigned rank)
{
    uint32_t remote;
    asm("mapa.shared::cluster.u32 %0, %1, %2;"
        : "=r"(remote)
        : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return remote;
}

__device__ __forceinline__ void store_rank_f32(float* p, unsigned rank, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr_of_rank(p, rank)), "f"(v) : "memory");
}

__device__ __forceinline__ void store_rank_u64(uint64_t* p, unsigned rank, uint64_t v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr_of_rank(p, rank)), "l"(v) : "memory");
}

constexpr int kMaxCluster = 8;

struct Slice {
    int head, lo, hi, tail;   // single elements, vectors [lo, hi), single elements
    int vec0, tail0;          // index of the body's first element, of the tail's first
};

template <int DT>
__device__ __forceinline__ Slice row_slice(const char* p, int V, unsigned rank, unsigned n)
{
    const RowSpan r = row_span<DT>(p, V);
    const int log_n = 31 - __clz(n);   // n is a power of two, at most kMaxCluster
    Slice s;
    s.head = rank == 0 ? r.head : 0;
    s.tail = rank == n - 1 ? r.tail : 0;
    s.lo = (int)((unsigned)r.nvec * rank >> log_n);          // nvec < 2^28
    s.hi = (int)((unsigned)r.nvec * (rank + 1) >> log_n);
    s.vec0 = r.head;
    s.tail0 = r.head + r.nvec * El<DT>::kVec;
    return s;
}

// Calls f(x, j) for each element x of index j that thread `t` of the block
// has.  part, parts: only every parts-th of its vectors, from part (and the
// single elements with part 0), for threads that share the work of one.
template <int DT, class F>
__device__ __forceinline__ void for_elements(const char* row, const Slice& s, int t, int part,
                                             int parts, F&& f)
{
    constexpr int kB = El<DT>::kBytes, kV = El<DT>::kVec;
    const char* body = row + s.vec0 * kB;
    for (int64_t i = s.lo + t + (int64_t)part * kRowThreads; i < s.hi;
         i += (int64_t)parts * kRowThreads) {
        float x[kV];
        El<DT>::unpack(ld16(body + i * 16), x);
#pragma unroll
        for (int j = 0; j < kV; ++j) f(x[j], s.vec0 + (int)i * kV + j);
    }
    if (part != 0) return;
    if (t < s.head) f(El<DT>::load(row + t * kB), t);
    if (t < s.tail) f(El<DT>::load(row + (int64_t)(s.tail0 + t) * kB), s.tail0 + t);
}

// ------------------------------------------------------------ softmax statistics
//
// Running maximum m, S = sum 2^u and U = sum u 2^u (where ENT) over a part of
// a row, with u = (x - m) c and c = scale * log2(e): one pass over the logits,
// whatever came before a larger maximum being rescaled.  u is computed as
// x c - (m c) in one fused operation; m c is rounded once and the same value
// is used wherever m is, so its rounding cancels.  Elements below kLowest
// count as kLowest there, whose 2^u is 0, so that a masked element (-inf) gives
// 0 * u = 0 to U.  That needs a maximum well above kLowest and an ordinary
// scale; otherwise (a row of the type's lowest value, or nothing but -inf so
// far) u is (x - m) c and -inf is left out.
struct Stat {
    float m, S, U;
};

constexpr float kMinExp = -16384.0f;
constexpr float kLowest = -1e20f;

// c, and the smallest maximum for which the fused form holds.
struct StatScale {
    float c, low_max;
    __device__ __forceinline__ explicit StatScale(float scale)
        : c(scale * kLog2e), low_max(c > 1e-15f && c < 1e17f ? -1e19f : INFINITY)
    {
    }
};

// (a - m) c for the maxima a <= m of two parts.
__device__ __forceinline__ float max_step(float a, float m, const StatScale& k)
{
    const float d = m < k.low_max ? (a - m) * k.c : a * k.c - m * k.c;
    return fmaxf(d, kMinExp);
}

__device__ __forceinline__ void stat_rebase(Stat& s, float m, const StatScale& k)
{
    // u against the new maximum is u + d, so 2^u gets the factor 2^d
    const float d = max_step(s.m, m, k);
    const float f = ex2(d);
    s.U = f * __fmaf_rn(d, s.S, s.U);
    s.S *= f;
    s.m = m;
}

__device__ __forceinline__ Stat stat_join(Stat a, Stat b, const StatScale& k)
{
    const float m = max_nan(a.m, b.m);
    if (m == -INFINITY) return a;             // nothing in either
    stat_rebase(a, m, k);
    stat_rebase(b, m, k);
    return {m, a.S + b.S, a.U + b.U};
}

// One element.
__device__ __forceinline__ void stat_add(Stat& s, float x, const StatScale& k)
{
    if (!(x <= s.m)) stat_rebase(s, max_nan(s.m, x), k);
    if (x == -INFINITY) return;
    const float u = fmaxf(s.m < k.low_max ? (x - s.m) * k.c : __fmaf_rn(x, k.c, -(s.m * k.c)), kMinExp);
    const float e = ex2(u);
    s.S += e;
    s.U = __fmaf_rn(e, u, s.U);
}

// A thread's running statistics, S and U in two halves.  With TOP also the
// first of the vectors that were added together with the largest element, a
// copy of these in `kept` (shared memory), and the largest element elsewhere.
template <int DT, bool ENT, bool TOP>
struct ThreadStat {
    float m = -INFINITY;
    F2 S = 0, U = 0;
    int best = 0;
    float second = -INFINITY;

    // N vectors at once, the first of them number i.
    template <int N>
    __device__ __forceinline__ void add(const uint4 (&w)[N], int i, const StatScale& k, uint4* kept)
    {
        constexpr int kV = El<DT>::kVec;
        const float vm = El<DT>::vec_max(w);
        if (TOP && vm <= m) second = max_nan(second, vm);
        if (!(vm <= m)) {
            if (TOP) {
                second = m;
                best = i;
#pragma unroll
                for (int l = 0; l < N; ++l) kept[l * kRowThreads + threadIdx.x] = w[l];
            }
            const float mm = max_nan(m, vm);
            const float d = max_step(m, mm, k);
            const F2 f = pack2(ex2(d), ex2(d));
            if (ENT) U = fma2(f, fma2(pack2(d, d), S, U), 0);
            S = fma2(f, S, 0);
            m = mm;
        }
        if (m < k.low_max) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float x[kV];
                El<DT>::unpack(w[i], x);
                Stat s{m, 0.0f, 0.0f};
                for (int j = 0; j < kV; ++j) stat_add(s, x[j], k);
                S = add2(S, pack2(s.S, 0.0f));
                U = add2(U, pack2(s.U, 0.0f));
            }
            return;
        }
        const F2 c2 = pack2(k.c, k.c), b2 = pack2(-(m * k.c), -(m * k.c));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            F2 x[kV / 2];
            El<DT>::pairs_above(w[i], kLowest, x);
#pragma unroll
            for (int j = 0; j < kV / 2; ++j) {
                const F2 u = fma2(x[j], c2, b2);
                const F2 e = pack2(ex2(lo2(u)), ex2(hi2(u)));
                S = add2(S, e);
                if (ENT) U = fma2(e, u, U);
            }
        }
    }

    __device__ __forceinline__ Stat get() const
    {
        return {m, lo2(S) + hi2(S), ENT ? lo2(U) + hi2(U) : 0.0f};
    }
};

// Where a thread's largest elements are, for block_top: the order of its
// largest one (0 without elements), the first of the `count` vectors
// that were loaded with it, and the order of the largest element elsewhere.
struct ThreadTop {
    uint32_t max, second;
    int best, count;
};

// The statistics of this thread's elements of a slice.
template <int DT, bool ENT, bool TOP>
__device__ __forceinline__ Stat thread_stat(const char* row, const Slice& s, const StatScale& k,
                                            ThreadTop* top, uint4* kept)
{
    constexpr int kB = El<DT>::kBytes;
    const int t = threadIdx.x;
    ThreadStat<DT, ENT, TOP> ts;
    const char* body = row + s.vec0 * kB;
    int i = s.lo + t;
    for (; i < s.hi - (kRowLoads - 1) * kRowThreads; i += kRowLoads * kRowThreads) {
        uint4 w[kRowLoads];
#pragma unroll
        for (int l = 0; l < kRowLoads; ++l) w[l] = ld16(body + (int64_t)(i + l * kRowThreads) * 16);
        ts.add(w, i, k, kept);
    }
    if (i < s.hi - kRowThreads) {
        const uint4 w[2] = {ld16(body + (int64_t)i * 16), ld16(body + (int64_t)(i + kRowThreads) * 16)};
        ts.add(w, i, k, kept);
        i += 2 * kRowThreads;
    }
    if (i < s.hi) {
        const uint4 w[1] = {ld16(body + (int64_t)i * 16)};
        ts.add(w, i, k, kept);
    }
    Stat st = ts.get();
    if (t < s.head) stat_add(st, El<DT>::load(row + t * kB), k);
    if (t < s.tail) stat_add(st, El<DT>::load(row + (int64_t)(s.tail0 + t) * kB), k);
    if (TOP) {
        const bool single = t < s.head || t < s.tail;
        top->max = single || s.lo + t < s.hi ? value_order(st.m) : 0u;
        top->second = single ? top->max : value_order(ts.second);
        top->best = ts.best;
        // full batches of kRowLoads, then one of two, then a single one
        const int mine = s.hi - s.lo - t, at = (ts.best - s.lo - t) / kRowThreads;
        const int n = (mine + kRowThreads - 1) / kRowThreads - at;
        top->count = n >= kRowLoads ? kRowLoads : n >= 2 ? 2 : 1;
    }
    return st;
}

// The statistics of a warp's lanes together: the maximum first, then sums of
// the parts rebased to it.
__device__ __forceinline__ Stat warp_stat(Stat s, const StatScale& k)
{
    float m = s.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m != -INFINITY) stat_rebase(s, m, k);   // (also NaN)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s.S += __shfl_xor_sync(0xffffffffu, s.S, o);
        s.U += __shfl_xor_sync(0xffffffffu, s.U, o);
    }
    return s;
}

struct StatShared {
    Stat warp[kRowWarps];
    Stat block[kMaxCluster];   // by cluster rank
};

// The statistics of the whole row, in every thread, from each thread's own.
// In a cluster every block must have announced itself with
// cluster_arrive_relaxed before.  Contains barriers.
__device__ __forceinline__ Stat row_stat(Stat s, const StatScale& k, StatShared& sh, unsigned rank,
                                         unsigned n)
{
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    s = warp_stat(s, k);
    if (lane == 0) sh.warp[wid] = s;
    __syncthreads();
    if (wid == 0) {
        s = warp_stat(lane < kRowWarps ? sh.warp[lane] : Stat{-INFINITY, 0.0f, 0.0f}, k);
        if (n == 1) {
            if (lane == 0) sh.block[0] = s;
        } else {
            cluster_wait();
            if (lane < (int)n) {
                store_rank_f32(&sh.block[rank].m, lane, s.m);
                store_rank_f32(&sh.block[rank].S, lane, s.S);
                store_rank_f32(&sh.block[rank].U, lane, s.U);
            }
        }
    } else if (n > 1) {
        cluster_wait();
    }
    if (n == 1) {
        __syncthreads();
        return sh.block[0];
    }
    cluster_arrive_release();
    cluster_wait();
    s = sh.block[0];
    for (unsigned r = 1; r < n; ++r) s = stat_join(s, sh.block[r], k);
    return s;
}

// lse and entropy of a row's statistics; m NaN or +inf: NaN, m -inf: -inf and 0.
struct RowResult {
    float lse, log2S, entropy;
    bool empty, bad;
};

__device__ __forceinline__ RowResult row_result(const Stat& s, float scale, const StatScale& k)
{
    RowResult r;
    r.empty = s.m == -INFINITY;
    r.bad = !(s.m < INFINITY);
    r.log2S = log2f(s.S);
    r.lse = r.bad ? quiet_nan()
            : r.empty ? -INFINITY
            : s.m < k.low_max ? __fmaf_rn(s.m, scale, r.log2S * kLn2)
                              : (s.m * k.c + r.log2S) * kLn2;
    r.entropy = r.bad ? quiet_nan() : r.empty ? 0.0f : (r.log2S - s.U / s.S) * kLn2;
    return r;
}

__device__ __forceinline__ float logprob_of(float x, const Stat& s, const RowResult& r, float scale,
                                            const StatScale& k)
{
    if (r.bad) return quiet_nan();
    if (r.empty) return -INFINITY;
    if (s.m < k.low_max || x < kLowest) return __fmaf_rn(x - s.m, scale, -r.log2S * kLn2);
    return (__fmaf_rn(x, k.c, -(s.m * k.c)) - r.log2S) * kLn2;
}

// ------------------------------------------------------------ top alternatives
//
// An element's rank key: the value's order in the upper word (NaN highest),
// the complement of its index in the lower, so that the largest key is the
// largest value of the lowest index.  0 is below every key.

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

constexpr int kTopCap = 512;                        // candidates a block can hold
constexpr int kTopGroup = kRowThreads / 32;         // threads per group, 32 groups

struct TopShared {
    uint4 kept[kRowLoads * kRowThreads];            // each thread's vectors with its largest element
    uint64_t cand[kTopCap];
    uint64_t merged[kMaxCluster * DPZ_LM_MAX_TOP];  // a cluster's first block: every block's best
    uint64_t best[kRowWarps];
    uint32_t group[32];
    uint32_t threshold;
    int n;
};

// The block's K largest keys of its slice into out[0..K) of shared memory (0
// where it has fewer elements), for K <= 32.
//
// The K-th largest of 32 groups' maxima is a threshold that at least K
// elements reach, and few more do: a random row of any length has
// 32 (H(32) - H(32 - K)) of them, 9 for K = 8, 31 for K = 20 and 130 for
// K = 32 (H: harmonic numbers).  Only threads whose own maximum reaches it
// look at their elements again, a warp's lanes sharing the work for each: at
// the kept vectors if nothing else of theirs reaches it, else at all.  The candidates are ranked against each other.  If more than kTopCap elements
// reach it (rows of few distinct values), K rounds of a block-wide maximum
// are run instead.  If only masked elements are left below the threshold
// (fewer than K groups have any other), the unmasked ones are candidates and
// the masked ones of lowest index, which are ties, fill up.
template <int DT>
__device__ __forceinline__ void block_top(const char* row, const Slice& s, const ThreadTop& own,
                                          int K, TopShared& sh, uint64_t* out)
{
    constexpr int kB = El<DT>::kBytes, kV = El<DT>::kVec;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    uint32_t g = own.max;
#pragma unroll
    for (int o = 1; o < kTopGroup; o <<= 1) g = max(g, __shfl_xor_sync(0xffffffffu, g, o));
    if (threadIdx.x % kTopGroup == 0) sh.group[threadIdx.x / kTopGroup] = g;
    if (threadIdx.x < K) out[threadIdx.x] = 0;
    __syncthreads();
    if (wid == 0) {
        const uint32_t v = sh.group[lane];
        int above = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const uint32_t w = __shfl_sync(0xffffffffu, v, i);
            above += w > v || (w == v && i < lane);
        }
        if (above == K - 1) sh.threshold = v;
        if (lane == 0) sh.n = 0;
    }
    __syncthreads();
    const uint32_t th = max(sh.threshold, 1u);
    const bool fill = th <= kOrderMasked;
    const uint32_t floor_ = fill ? kOrderMasked + 1 : th;
    const auto offer = [&](float x, int j) {
        const uint32_t o = value_order(x);
        if (o >= floor_) {
            const int at = atomicAdd(&sh.n, 1);
            if (at < kTopCap) sh.cand[at] = rank_key(o, j);
        }
    };
    static_assert(kRowLoads * kV <= 32, "one lane per kept element");
    unsigned m = __ballot_sync(0xffffffffu, own.max >= floor_ && own.second < floor_);
    while (m != 0) {
        const int src = __ffs(m) - 1, l = lane / kV, j = lane % kV;
        m &= m - 1;
        const int best = __shfl_sync(0xffffffffu, own.best, src);
        const int count = __shfl_sync(0xffffffffu, own.count, src);
        if (l < count) {
            const uint4* v = &sh.kept[l * kRowThreads + (wid << 5) + src];
            offer(El<DT>::load(reinterpret_cast<const char*>(v) + j * kB),
                  s.vec0 + (best + l * kRowThreads) * kV + j);
        }
    }
    m = __ballot_sync(0xffffffffu, own.max >= floor_ && own.second >= floor_);
    while (m != 0) {
        const int owner = (wid << 5) + __ffs(m) - 1;
        m &= m - 1;
        for_elements<DT>(row, s, owner, lane, 32, offer);
    }
    __syncthreads();
    int n = sh.n;
    if (fill && n < K) {
        // masked elements among the slice's first K + n hold the lowest indices
        __syncthreads();
        const int first = s.head > 0 ? 0 : s.vec0 + s.lo * El<DT>::kVec;
        const int last = s.tail > 0 ? s.tail0 + s.tail : s.vec0 + s.hi * El<DT>::kVec;
        const int j = first + threadIdx.x;
        if ((int)threadIdx.x < K + n && j < last &&
            value_order(El<DT>::load(row + (int64_t)j * kB)) == kOrderMasked)
            sh.cand[atomicAdd(&sh.n, 1)] = rank_key(kOrderMasked, j);
        __syncthreads();
        n = sh.n;
    }
    if (n <= kTopCap) {
        for (int i = threadIdx.x; i < n; i += kRowThreads) {
            const uint64_t key = sh.cand[i];
            int above = 0;
            for (int q = 0; q < n; ++q) above += sh.cand[q] > key;
            if (above < K) out[above] = key;
        }
        return;
    }
    // K rounds: the largest key below the last one.  Each thread keeps its own
    // best and looks for the next one only when its best was taken.
    uint64_t prev = ~uint64_t(0), best = 0;
    bool stale = true;
    for (int k = 0; k < K && prev != 0; ++k) {
        if (stale) {
            best = 0;
            for_elements<DT>(row, s, threadIdx.x, 0, 1, [&](float x, int j) {
                const uint64_t key = rank_key(value_order(x), j);
                if (key < prev && key > best) best = key;
            });
        }
        const uint64_t wb = warp_max64(best);
        if (lane == 0) sh.best[wid] = wb;
        __syncthreads();
        prev = warp_max64(lane < kRowWarps ? sh.best[lane] : 0);
        __syncthreads();
        stale = best == prev;
        if (threadIdx.x == 0) out[k] = prev;
    }
}

// ------------------------------------------------------------ log probabilities

// fp32 rows have half the elements per byte and so leave registers and issue
// slots for more blocks on an SM.
template <int DT, bool ENT, bool TOP>
__global__ void __launch_bounds__(kRowThreads, DT == DPZ_F32 ? 7 : 6) k_logprobs(LogprobArgs a)
{
    __shared__ StatShared ssh;
    __shared__ TopShared tsh;
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
    ThreadTop best;
    const Stat s = row_stat(thread_stat<DT, ENT, TOP>(row, sl, k, &best, tsh.kept), k, ssh,
                            rank, n);
    RowResult r;
    if (threadIdx.x < 32) r = row_result(s, a.scale, k);   // one warp writes the results
    if (rank == 0 && threadIdx.x == 0) {
        if (a.logprob != nullptr)
            a.logprob[t] = y < 0 ? 0.0f : logprob_of(target, s, r, a.scale, k);
        if (a.lse != nullptr) a.lse[t] = r.lse;
        if (ENT) a.entropy[t] = r.entropy;
    }
    if (!TOP) return;
    uint64_t* top = tsh.merged;
    block_top<DT>(row, sl, best, a.K, tsh, top);
    __syncthreads();
    if (n > 1) {
        // every block's best to the first block, which ranks them
        uint64_t key = 0;
        if ((int)threadIdx.x < a.K) key = top[threadIdx.x];
        cluster_arrive_release();
        cluster_wait();
        if ((int)threadIdx.x < a.K) store_rank_u64(&tsh.merged[rank * a.K + threadIdx.x], 0, key);
        cluster_arrive_release();
        cluster_wait();
        if (rank != 0) return;
        if (threadIdx.x < n * a.K) {
            const uint64_t mine = tsh.merged[threadIdx.x];
            int above = 0;
            for (unsigned q = 0; q < n * a.K; ++q) above += tsh.merged[q] > mine;
            if (mine != 0 && above < a.K) tsh.cand[above] = mine;
        }
        __syncthreads();
        top = tsh.cand;
    }
    if ((int)threadIdx.x < a.K) {
        const uint64_t key = top[threadIdx.x];
        const int j = (int)(0xffffffffu - (uint32_t)key);
        const int64_t at = t * a.K + threadIdx.x;
        if (a.targets.it == DPZ_I64) static_cast<int64_t*>(a.top_ids)[at] = j;
        else static_cast<int*>(a.top_ids)[at] = j;
        a.top_logprobs[at] = logprob_of(value_of_order((uint32_t)(key >> 32)), s, r, a.scale, k);
    }
}

// ------------------------------------------------------------ gradients
//
// f(x, j) gives the gradient of element x of index j; a row is read and
// written by the same thread, so the output may be the input.
template <int DT, class F>
__device__ __forceinline__ void map_row(const char* row, char* out, const Slice& s, F&& f)
{
    constexpr int kB = El<DT>::kBytes, kV = El<DT>::kVec;
    const int t = threadIdx.x;
    // the output's rows may be aligned otherwise than the input's
    const bool same = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    const int64_t body = s.vec0 * kB;
    for (int i = s.lo + t; i < s.hi; i += kRowThreads) {
        float x[kV];
        El<DT>::unpack(ld16(row + body + (int64_t)i * 16), x);
#pragma unroll
        for (int j = 0; j < kV; ++j) x[j] = f(x[j], s.vec0 + i * kV + j);
        char* q = out + body + (int64_t)i * 16;
        if (same) st16(q, El<DT>::pack(x));
        else
#pragma unroll
            for (int j = 0; j < kV; ++j) El<DT>::store(q + j * kB, x[j]);
    }
    if (t < s.head) El<DT>::store(out + t * kB, f(El<DT>::load(row + t * kB), t));
    if (t < s.tail) {
        const int j = s.tail0 + t;
        El<DT>::store(out + (int64_t)j * kB, f(El<DT>::load(row + (int64_t)j * kB), j));
    }
}

// Zeros in this block's part of a row.
template <int DT>
__device__ __forceinline__ void zero_row(char* out, int V, unsigned rank, unsigned n)
{
    const Slice s = row_slice<DT>(out, V, rank, n);
    constexpr int kB = El<DT>::kBytes;
    const int t = threadIdx.x;
    for (int i = s.lo + t; i < s.hi; i += kRowThreads)
        st16(out + s.vec0 * kB + (int64_t)i * 16, make_uint4(0, 0, 0, 0));
    if (t < s.head) El<DT>::store(out + t * kB, 0.0f);
    if (t < s.tail) El<DT>::store(out + (int64_t)(s.tail0 + t) * kB, 0.0f);
}

template <int DT>
__global__ void __launch_bounds__(kRowThreads) k_logprobs_grad(LogprobGradArgs a)
{
    pdl_enter();
    const unsigned rank = blockIdx.y, n = gridDim.y;     // slices of a row
    const int64_t t = blockIdx.x;
    const char* row = a.x.p + t * a.x.ld * El<DT>::kBytes;
    char* out = a.dx.p + t * a.dx.ld * El<DT>::kBytes;
    const int y = load_token(a.targets, t, a.V);
    const float g = y < 0 ? 0.0f : a.dlogprob[t];
    const float h = a.dentropy != nullptr ? a.dentropy[t] : 0.0f;
    const float lse = a.lse[t];
    if ((g == 0.0f && h == 0.0f) || lse == -INFINITY) {
        zero_row<DT>(out, a.V, rank, n);
        return;
    }
    const float H = h != 0.0f ? a.entropy[t] : 0.0f;
    // -p (g + h (log p + H)) = p (A + B log2 p)
    const float A = -__fmaf_rn(h, H, g) * a.scale, B = -h * kLn2 * a.scale;
    const float gs = g * a.scale;
    map_row<DT>(row, out, row_slice<DT>(row, a.V, rank, n), [&](float x, int j) {
        const float u = max_nan(__fmaf_rn(x, a.scale, -lse) * kLog2e, kMinExp);
        const float d = ex2(u) * __fmaf_rn(B, u, A);
        return j == y ? d + gs : d;
    });
}

// ------------------------------------------------------------ distillation

// The teacher's entries of one row in shared memory: tokens (-1: absent), the
// student's logits there, probabilities and their logarithms.
struct Teacher {
    int id[DPZ_LM_MAX_TEACHER];
    float x[DPZ_LM_MAX_TEACHER], q[DPZ_LM_MAX_TEACHER], logq[DPZ_LM_MAX_TEACHER];
    int any;
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

// One warp loads a row's entries and their softmax; the student's logits of
// those in [lo, hi).
template <int DT>
__device__ __forceinline__ void load_teacher(const DistillArgs& a, int64_t t, const char* row,
                                             int64_t lo, int64_t hi, Teacher& w)
{
    const int lane = threadIdx.x & 31;
    float m = -INFINITY;
    for (int k = lane; k < a.K; k += 32) {
        const int64_t at = t * a.K + k;
        int id = load_token(a.ids, at, a.V);
        float v = a.teacher.dt == DPZ_F32 ? El<DPZ_F32>::load(a.teacher.p + at * 4)
                                          : El<DPZ_BF16>::load(a.teacher.p + at * 2);
        if (v == -INFINITY) id = -1;
        if (id < 0) v = -INFINITY;
        w.id[k] = id;
        w.x[k] = id < lo || id >= hi ? 0.0f : El<DT>::load(row + (int64_t)id * El<DT>::kBytes);
        w.logq[k] = v;
        m = max_nan(m, v);
    }
    m = warp_max_nan(m);
    float S = 0.0f;
    for (int k = lane; k < a.K; k += 32) {
        // the difference before the product, as for the student
        const float v = w.id[k] < 0 ? -INFINITY : (w.logq[k] - m) * a.inv_tau;
        w.logq[k] = v;
        S += w.id[k] < 0 ? 0.0f : expf(v);
    }
    S = warp_sum_all(S);
    const float logS = logf(S);
    for (int k = lane; k < a.K; k += 32) {
        const float v = w.logq[k] - logS;
        w.logq[k] = v;
        w.q[k] = w.id[k] < 0 ? 0.0f : expf(v);
    }
    if (lane == 0) w.any = m != -INFINITY;
}

template <int DT, bool LOSS, bool GRAD>
__global__ void __launch_bounds__(kRowThreads, 6) k_distill(DistillArgs a)
{
    __shared__ Teacher w;
    __shared__ StatShared ssh;
    const unsigned rank = cluster_rank(), n = cluster_size();
    if (LOSS && n > 1) cluster_arrive_relaxed();
    pdl_enter();
    const int64_t t = blockIdx.x >> (31 - __clz(n));
    const char* row = a.x.p + t * a.x.ld * El<DT>::kBytes;
    char* out = GRAD ? a.dx.p + t * a.dx.ld * El<DT>::kBytes : nullptr;
    const float wt = GRAD ? a.dloss[t] : 0.0f;
    if (!LOSS && wt == 0.0f) {
        zero_row<DT>(out, a.V, rank, n);
        return;
    }
    const Slice sl = row_slice<DT>(row, a.V, rank, n);
    const int lane = threadIdx.x & 31;
    // every block of a cluster needs the entries of its slice, the first one
    // all of them for the loss; the last warp loads them (the first one joins
    // the statistics).  In place, another block's slice may be overwritten
    // already unless a cluster barrier comes between, as with LOSS.
    const int first = rank == 0 ? 0 : sl.vec0 + sl.lo * El<DT>::kVec;
    const int last = rank == n - 1 ? sl.tail0 + sl.tail : sl.vec0 + sl.hi * El<DT>::kVec;
    if (threadIdx.x >= kRowThreads - 32)
        load_teacher<DT>(a, t, row, LOSS ? 0 : first, LOSS ? a.V : last, w);
    float lse;
    if (LOSS) {
        const StatScale k(a.inv_tau);
        const Stat s = row_stat(thread_stat<DT, false, false>(row, sl, k, nullptr, nullptr), k, ssh, rank, n);
        const RowResult r = row_result(s, a.inv_tau, k);
        lse = r.lse;
        if (rank == 0 && threadIdx.x < 32) {
            float sum = 0.0f;
            for (int i = lane; i < a.K; i += 32)
                if (w.q[i] != 0.0f)
                    sum += w.q[i] * (w.logq[i] - logprob_of(w.x[i], s, r, a.inv_tau, k));
            sum = warp_sum_all(sum);
            if (lane == 0) {
                a.loss[t] = w.any ? sum : 0.0f;
                if (a.lse != nullptr) a.lse[t] = lse;
            }
        }
    } else {
        lse = a.lse_in[t];
        __syncthreads();
    }
    if (!GRAD) return;
    if (wt == 0.0f || !w.any || lse == -INFINITY) {
        zero_row<DT>(out, a.V, rank, n);
        return;
    }
    const float ws = wt * a.inv_tau;
    const auto p = [&](float x) {
        return ex2(max_nan(__fmaf_rn(x, a.inv_tau, -lse) * kLog2e, kMinExp));
    };
    map_row<DT>(row, out, sl, [&](float x, int) { return ws * p(x); });
    __syncthreads();
    // the entries' tokens again where they are in the slice, now with their q
    for (int i = threadIdx.x; i < a.K; i += kRowThreads) {
        const int id = w.id[i];
        if (id < first || id >= last) continue;
        float q = 0.0f;
        bool once = true;
        for (int j = 0; j < a.K; ++j)
            if (w.id[j] == id) {
                if (j < i) once = false;
                q += w.q[j];
            }
        if (once) El<DT>::store(out + (int64_t)id * El<DT>::kBytes, ws * (p(w.x[i]) - q));
    }
}

// Blocks per row: as many as keep one wave of blocks on the GPU when there are
// few rows, at most 8, each with at least one vector per thread.
unsigned row_cluster(int64_t T, int64_t V, int dt)
{
    const int64_t nvec = V * (dt == DPZ_F32 ? 4 : 2) / 16;
    unsigned n = 1;
    while (n < kMaxCluster && T * n * 2 <= 304 && nvec >= 2 * n * kRowThreads) n *= 2;
    return n;
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t s)
{
    set_last_kernel_name("lm_logprobs");
    const bool ent = a.entropy != nullptr, top = a.K > 0;
    auto fn = a.x.dt == DPZ_BF16
                  ? (ent ? (top ? k_logprobs<DPZ_BF16, true, true> : k_logprobs<DPZ_BF16, true, false>)
                         : (top ? k_logprobs<DPZ_BF16, false, true>
                                : k_logprobs<DPZ_BF16, false, false>))
                  : (ent ? (top ? k_logprobs<DPZ_F32, true, true> : k_logprobs<DPZ_F32, true, false>)
                         : (top ? k_logprobs<DPZ_F32, false, true>
                                : k_logprobs<DPZ_F32, false, false>));
    const unsigned n = row_cluster(a.T, a.V, a.x.dt);
    return launch_kernel(fn, dim3((unsigned)a.T * n), dim3(kRowThreads), 0, s, true, n > 1 ? n : 0u,
                         a);
}

cudaError_t launch_logprobs_grad(const LogprobGradArgs& a, cudaStream_t s)
{
    set_last_kernel_name("lm_logprobs_grad");
    auto fn = a.x.dt == DPZ_BF16 ? k_logprobs_grad<DPZ_BF16> : k_logprobs_grad<DPZ_F32>;
    const unsigned n = row_cluster(a.T, a.V, a.x.dt);
    return launch_kernel(fn, dim3((unsigned)a.T, n), dim3(kRowThreads), 0, s, true, 0u, a);
}

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t s)
{
    const bool b = a.x.dt == DPZ_BF16;
    void (*fn)(DistillArgs);
    if (a.loss != nullptr && a.dx.p != nullptr) {
        set_last_kernel_name("lm_distill_step");
        fn = b ? k_distill<DPZ_BF16, true, true> : k_distill<DPZ_F32, true, true>;
    } else if (a.loss != nullptr) {
        set_last_kernel_name("lm_distill");
        fn = b ? k_distill<DPZ_BF16, true, false> : k_distill<DPZ_F32, true, false>;
    } else {
        set_last_kernel_name("lm_distill_grad");
        fn = b ? k_distill<DPZ_BF16, false, true> : k_distill<DPZ_F32, false, true>;
    }
    const unsigned n = row_cluster(a.T, a.V, a.x.dt);
    return launch_kernel(fn, dim3((unsigned)a.T * n), dim3(kRowThreads), 0, s, true, n > 1 ? n : 0u,
                         a);
}

}  // namespace dpz
