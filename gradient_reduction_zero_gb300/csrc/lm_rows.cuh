// Rows of logits over a vocabulary, shared by lm_logprobs.cu and
// lm_distill.cu: how a row's elements are read and split between blocks, the
// running softmax statistics, and the writing of a row of gradients.  Kernels
// are compiled for blocks of NT threads.
#pragma once

#include <algorithm>
#include <cmath>

#include "bulk.cuh"
#include "device.cuh"
#include "internal.h"
#include "lm.h"
#include "lm_shape.h"

namespace dpz {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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

__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ F2 ex2x2(F2 u) { return pack2(ex2(lo2(u)), ex2(hi2(u))); }

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

// ------------------------------------------------------------ a row's elements
//
// A row may begin at any element (a vocabulary of 50,257 shifts each row), so
// it is a head of single elements up to the first 16-byte boundary, a body of
// 16-byte vectors, and a tail.

template <int DT>
struct El;   // kVec: elements of a 16-byte vector

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
    static __device__ __forceinline__ void pairs(const uint4& w, F2 (&x)[kVec / 2])
    {
        x[0] = (F2)w.y << 32 | w.x;
        x[1] = (F2)w.w << 32 | w.z;
    }
    static __device__ __forceinline__ uint4 pack(const F2 (&x)[kVec / 2])
    {
        return make_uint4((uint32_t)x[0], (uint32_t)(x[0] >> 32), (uint32_t)x[1],
                          (uint32_t)(x[1] >> 32));
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
    static __device__ __forceinline__ void pairs(const uint4& w, F2 (&x)[kVec / 2])
    {
        x[0] = pack2(bf16_lo(w.x), bf16_hi(w.x));
        x[1] = pack2(bf16_lo(w.y), bf16_hi(w.y));
        x[2] = pack2(bf16_lo(w.z), bf16_hi(w.z));
        x[3] = pack2(bf16_lo(w.w), bf16_hi(w.w));
    }
    static __device__ __forceinline__ uint4 pack(const F2 (&x)[kVec / 2])
    {
        return make_uint4(pack_bf16x2(lo2(x[0]), hi2(x[0])), pack_bf16x2(lo2(x[1]), hi2(x[1])),
                          pack_bf16x2(lo2(x[2]), hi2(x[2])), pack_bf16x2(lo2(x[3]), hi2(x[3])));
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
// vectors lo + i, lo + i + NT, ...

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

struct Slice {
    int head, lo, hi, tail;   // single elements, vectors [lo, hi), single elements
    int vec0, tail0;          // index of the body's first element, of the tail's first
    int first, last;          // the slice's elements: [first, last)
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
    s.first = rank == 0 ? 0 : s.vec0 + s.lo * El<DT>::kVec;
    s.last = rank == n - 1 ? V : s.vec0 + s.hi * El<DT>::kVec;
    return s;
}

// ------------------------------------------------------------ softmax statistics
//
// Running maximum m, S = sum 2^u and U = sum u 2^u (where ENT) over a part of
// a row, with u = (x - m) c and c = scale * log2(e): one pass over the logits,
// whatever came before a larger maximum being rescaled.
struct Stat {
    float m, S, U;
};

constexpr float kMinExp = -16384.0f;   // 2^u is 0 there, and u 2^u too
constexpr float kLowest = -1e20f;

// Within a thread u is x c - (m c) in one fused operation where it may be:
// m c is rounded once and the same value is used wherever m is, so that its
// rounding shifts every u of the thread alike, by at most half a unit in the
// last place of m c, and unshifted() takes the shift out at the end.  That
// holds for |m c| up to kFusedMost, where the shift is 2^-10; at a row of -1e10
// it would be 512, beyond the range of 2^u.  Elements below kLowest count as
// kLowest, whose 2^u is 0, so that a masked element (-inf) gives 0 * u = 0 to
// U.  Larger maxima (a row wholly masked by a finite value) and extreme scales
// take the product of the difference, which has one operation more.
constexpr float kFusedMost = 0x1p15f;

struct StatScale {
    float c, most;   // most: the largest |m c| for the fused form; -1: none
    __device__ __forceinline__ explicit StatScale(float scale)
        : c(scale * kLog2e), most(c > 1e-12f && c < 1e17f ? kFusedMost : -1.0f)
    {
    }
    __device__ __forceinline__ bool fused(float mc) const { return fabsf(mc) <= most; }
};

// (x - m) c, at least kMinExp; of halves, since the difference of two of the
// type's values may overflow.
__device__ __forceinline__ float exponent(float x, float m, float c)
{
    return fmaxf(__fmaf_rn(0.5f, x, -0.5f * m) * (2.0f * c), kMinExp);
}

// A thread's S and U against rnd(m c), if that is the fused form's, against m c.
__device__ __forceinline__ Stat unshifted(Stat s, const StatScale& k)
{
    const float mc = s.m * k.c;
    if (!k.fused(mc)) return s;
    const float d = __fmaf_rn(s.m, k.c, -mc);            // exact; u is too large by d
    const float g = -d * kLn2, f = __fmaf_rn(0.5f * g, g, g);   // 2^-d - 1, d^3 left out
    const float U = __fmaf_rn(-d, s.S, s.U);
    return {s.m, __fmaf_rn(s.S, f, s.S), __fmaf_rn(U, f, U)};
}

__device__ __forceinline__ void stat_rebase(Stat& s, float m, const StatScale& k)
{
    // u against the new maximum is u + d, so 2^u gets the factor 2^d
    const float d = exponent(s.m, m, k.c);
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
    const float u = exponent(x, s.m, k.c);
    const float e = ex2(u);
    s.S += e;
    s.U = __fmaf_rn(e, u, s.U);
}

// A thread's running statistics, S and U in two halves.  With TOP also the
// first of the vectors that were added together with the largest element, a
// copy of these in `kept` (shared memory), and the largest element elsewhere.
template <int DT, int NT, bool ENT, bool TOP>
struct ThreadStat {
    float m = -INFINITY;
    F2 S = 0, U = 0;
    int best = 0;
    float second = -INFINITY;

    // The exponent of what is summed so far against a new maximum mm >= m; an
    // infinite m c has nothing that counts.
    __device__ __forceinline__ float step(float mm, const StatScale& k) const
    {
        const float a = m * k.c, b = mm * k.c;
        if (b <= k.most && (a >= -k.most || a == -INFINITY)) return fmaxf(a - b, kMinExp);
        if (k.fused(b)) return fmaxf(__fmaf_rn(m, k.c, -b), kMinExp);
        return k.fused(a) ? fmaxf(-__fmaf_rn(mm, k.c, -a), kMinExp) : exponent(m, mm, k.c);
    }

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
                for (int l = 0; l < N; ++l) kept[l * NT + threadIdx.x] = w[l];
            }
            const float mm = max_nan(m, vm);
            const float d = step(mm, k);
            const F2 f = pack2(ex2(d), ex2(d));
            if (ENT) U = fma2(f, fma2(pack2(d, d), S, U), 0);
            S = fma2(f, S, 0);
            m = mm;
        }
        const float mc = m * k.c;
        const auto term = [&](F2 u) {
            const F2 e = ex2x2(u);
            S = add2(S, e);
            if (ENT) U = fma2(e, u, U);
        };
        if (k.fused(mc)) {
            const F2 c2 = pack2(k.c, k.c), b2 = pack2(-mc, -mc);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                F2 x[kV / 2];
                El<DT>::pairs_above(w[i], kLowest, x);
#pragma unroll
                for (int j = 0; j < kV / 2; ++j) term(fma2(x[j], c2, b2));
            }
        } else if (m != -INFINITY) {          // else nothing but masked elements so far
            // such rows are rare: with alternatives in bf16 a loop, whose instructions,
            // unrolled, cost short rows 5 % in fetching the others (8,192 of 2,000:
            // 30.6 us, 29.2 so); in fp32 the loop's registers cost 4 %
            const F2 h2 = pack2(0.5f, 0.5f), b2 = pack2(-0.5f * m, -0.5f * m);
            const F2 c2 = pack2(2.0f * k.c, 2.0f * k.c);
            constexpr int kUnroll = TOP && DT == DPZ_BF16 ? 1 : N;
#pragma unroll kUnroll
            for (int i = 0; i < N; ++i) {
                uint4 v = w[0];
#pragma unroll
                for (int l = 1; l < N; ++l)
                    if (i == l) v = w[l];
                F2 x[kV / 2];
                El<DT>::pairs(v, x);
#pragma unroll
                for (int j = 0; j < kV / 2; ++j) {
                    const F2 u = mul2(fma2(x[j], h2, b2), c2);
                    term(pack2(fmaxf(lo2(u), kMinExp), fmaxf(hi2(u), kMinExp)));
                }
            }
        }
    }

    __device__ __forceinline__ Stat get(const StatScale& k) const
    {
        return unshifted({m, lo2(S) + hi2(S), ENT ? lo2(U) + hi2(U) : 0.0f}, k);
    }
};

// A thread's S alone (U is left out), against the largest element of its first
// vectors instead of the running maximum: the reference cancels in the result,
// and nothing has to be compared or rescaled, a third fewer instructions.
// Elements so far above the reference that S passes kRefSumMax, NaN and +inf
// show in good(); the thread's vectors then go through ThreadStat.  With S below 2^60 no join of up to 2^11
// threads' sums overflows, and a sum that a join's factor 2^d flushes to zero
// (d < -126) was at most 2^-66 of the others.
constexpr float kRefSumMax = 0x1p60f;

template <int DT>
struct RefStat {
    float ref = -INFINITY;
    F2 S = 0;

    template <int N>
    __device__ __forceinline__ void add(const uint4 (&w)[N], int, const StatScale& k, uint4*)
    {
        constexpr int kV = El<DT>::kVec;
        if (ref == -INFINITY) {
            ref = El<DT>::vec_max(w);
            if (ref == -INFINITY) return;     // nothing but masked elements so far
        }
        const float rc = ref * k.c;
        if (k.fused(rc)) {
            const F2 c2 = pack2(k.c, k.c), b2 = pack2(-rc, -rc);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                F2 x[kV / 2];
                El<DT>::pairs(w[i], x);
#pragma unroll
                for (int j = 0; j < kV / 2; ++j) S = add2(S, ex2x2(fma2(x[j], c2, b2)));
            }
        } else {
            const F2 h2 = pack2(0.5f, 0.5f), b2 = pack2(-0.5f * ref, -0.5f * ref);
            const F2 c2 = pack2(2.0f * k.c, 2.0f * k.c);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                F2 x[kV / 2];
                El<DT>::pairs(w[i], x);
#pragma unroll
                for (int j = 0; j < kV / 2; ++j) S = add2(S, ex2x2(mul2(fma2(x[j], h2, b2), c2)));
            }
        }
    }

    __device__ __forceinline__ bool good() const
    {
        return ref < INFINITY && lo2(S) + hi2(S) < kRefSumMax;
    }

    __device__ __forceinline__ Stat get(const StatScale& k) const
    {
        return unshifted({ref, lo2(S) + hi2(S), 0.0f}, k);
    }
};

// Adds this thread's vectors of a slice from number i on: full batches of
// kLoads, then one of two, then a single one.
template <int DT, int NT, int kLoads = 4, class TS>
__device__ __forceinline__ void thread_rows(TS& ts, const char* row, const Slice& s, int i,
                                            const StatScale& k, uint4* kept = nullptr)
{
    const char* body = row + s.vec0 * El<DT>::kBytes;
    for (; i < s.hi - (kLoads - 1) * NT; i += kLoads * NT) {
        uint4 w[kLoads];
#pragma unroll
        for (int l = 0; l < kLoads; ++l) w[l] = ld16(body + (int64_t)(i + l * NT) * 16);
        ts.add(w, i, k, kept);
    }
    if (kLoads > 2 && i < s.hi - NT) {
        const uint4 w[2] = {ld16(body + (int64_t)i * 16), ld16(body + (int64_t)(i + NT) * 16)};
        ts.add(w, i, k, kept);
        i += 2 * NT;
    }
    if (i < s.hi) {
        const uint4 w[1] = {ld16(body + (int64_t)i * 16)};
        ts.add(w, i, k, kept);
    }
}

// And its single elements.
template <int DT>
__device__ __forceinline__ Stat thread_rest(Stat st, const char* row, const Slice& s,
                                            const StatScale& k)
{
    constexpr int kB = El<DT>::kBytes;
    const int t = threadIdx.x;
    if (t < s.head) stat_add(st, El<DT>::load(row + t * kB), k);
    if (t < s.tail) stat_add(st, El<DT>::load(row + (int64_t)(s.tail0 + t) * kB), k);
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

template <int NT>
struct StatShared {
    Stat warp[NT / 32];
    Stat block[kMaxCluster];   // by cluster rank
};

// What the blocks of a row's cluster have found, joined.
template <int NT>
__device__ __forceinline__ Stat blocks_stat(const StatScale& k, const StatShared<NT>& sh, unsigned n)
{
    Stat s = sh.block[0];
    for (unsigned r = 1; r < n; ++r) s = stat_join(s, sh.block[r], k);
    return s;
}

// The statistics of the whole row, in every thread, from each thread's own.
// In a cluster every block must have announced itself with
// cluster_arrive_relaxed before.  The block's barriers are two __syncthreads,
// or one and the cluster's: what a thread stores to shared memory before the
// call is visible to other(), which one other warp runs while the first joins
// the warps' parts, and what other() stores is visible after the call.
template <int NT, class F>
__device__ __forceinline__ Stat row_stat(Stat s, const StatScale& k, StatShared<NT>& sh,
                                         unsigned rank, unsigned n, F&& other)
{
    constexpr int kWarps = NT / 32;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    s = warp_stat(s, k);
    if (lane == 0) sh.warp[wid] = s;
    __syncthreads();
    if (n > 1) cluster_wait();
    if (wid == 0) {
        s = warp_stat(lane < kWarps ? sh.warp[lane] : Stat{-INFINITY, 0.0f, 0.0f}, k);
        if (n == 1) {
            if (lane == 0) sh.block[0] = s;
        } else if (lane < (int)n) {
            store_rank_f32(&sh.block[rank].m, lane, s.m);
            store_rank_f32(&sh.block[rank].S, lane, s.S);
            store_rank_f32(&sh.block[rank].U, lane, s.U);
        }
    }
    if (wid == kWarps - 1) other();
    if (n == 1) __syncthreads();
    else {
        cluster_arrive_release();
        cluster_wait();
    }
    return blocks_stat(k, sh, n);
}

// row_stat for a warp beside the NT threads, which works until then and has
// nothing to add.
template <int NT>
__device__ __forceinline__ Stat row_stat_beside(const StatScale& k, StatShared<NT>& sh, unsigned n)
{
    __syncthreads();
    if (n == 1) __syncthreads();
    else {
        cluster_wait();
        cluster_arrive_release();
        cluster_wait();
    }
    return blocks_stat(k, sh, n);
}

// log2 of S, lse and entropy of a row's statistics; m NaN or +inf: NaN, m -inf:
// lse -inf and entropy 0.
struct RowResult {
    float lse, log2S, entropy;
    bool empty, bad;
};

__device__ __forceinline__ RowResult row_result(const Stat& s, float scale)
{
    RowResult r;
    r.empty = s.m == -INFINITY;
    r.bad = !(s.m < INFINITY);
    r.log2S = r.bad ? quiet_nan() : log2f(s.S);
    r.lse = r.bad ? quiet_nan() : r.empty ? -INFINITY : __fmaf_rn(s.m, scale, r.log2S * kLn2);
    r.entropy = r.bad ? quiet_nan() : r.empty ? 0.0f : (r.log2S - s.U / s.S) * kLn2;
    return r;
}

__device__ __forceinline__ float logprob_of(float x, const Stat& s, const RowResult& r, float scale)
{
    if (r.bad) return quiet_nan();
    if (r.empty) return -INFINITY;
    // of halves, as in exponent()
    return __fmaf_rn(__fmaf_rn(0.5f, x, -0.5f * s.m), 2.0f * scale, -r.log2S * kLn2);
}

// ------------------------------------------------------------ gradients
//
// map_row writes f(x) for the elements of a slice, where f takes and gives
// pairs.  An element is read and written by the same thread, so the output
// may be the input.  STREAM: stores that leave L2 first.
template <int DT, bool STREAM = true, class F>
__device__ __forceinline__ void map_vector(const uint4& w, char* q, bool same, F&& f)
{
    constexpr int kB = El<DT>::kBytes, kV = El<DT>::kVec;
    F2 x[kV / 2];
    El<DT>::pairs(w, x);
#pragma unroll
    for (int j = 0; j < kV / 2; ++j) x[j] = f(x[j]);
    if (same) {
        if (STREAM) st16(q, El<DT>::pack(x));
        else *reinterpret_cast<uint4*>(q) = El<DT>::pack(x);
    } else {
#pragma unroll
        for (int j = 0; j < kV / 2; ++j) {
            El<DT>::store(q + 2 * j * kB, lo2(x[j]));
            El<DT>::store(q + (2 * j + 1) * kB, hi2(x[j]));
        }
    }
}

// Whether the output's rows are aligned as the input's are.
__device__ __forceinline__ bool same_alignment(const char* row, const char* out)
{
    return ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
}

// A thread's next vectors, loaded ahead of their use.
constexpr int kMapLoads = 4;

template <int DT, int NT>
__device__ __forceinline__ void map_load(const char* row, const Slice& s, int i,
                                         uint4 (&w)[kMapLoads])
{
    const char* body = row + s.vec0 * El<DT>::kBytes;
#pragma unroll
    for (int l = 0; l < kMapLoads; ++l)
        if (i + l * NT < s.hi) w[l] = ld16(body + (int64_t)(i + l * NT) * 16);
}

// The vectors from number i on, of which w are the first, then the slice's
// single elements.
template <int DT, int NT, class F>
__device__ __forceinline__ void map_row(const char* row, char* out, const Slice& s, int i,
                                        uint4 (&w)[kMapLoads], F&& f)
{
    constexpr int kB = El<DT>::kBytes;
    const int t = threadIdx.x;
    const bool same = same_alignment(row, out);
    const int body = s.vec0 * kB;
    while (i < s.hi) {
#pragma unroll
        for (int l = 0; l < kMapLoads; ++l)
            if (i + l * NT < s.hi)
                map_vector<DT>(w[l], out + body + (int64_t)(i + l * NT) * 16, same, f);
        i += kMapLoads * NT;
        map_load<DT, NT>(row, s, i, w);
    }
    if (t < s.head) El<DT>::store(out + t * kB, lo2(f(pack2(El<DT>::load(row + t * kB), 0.0f))));
    if (t < s.tail) {
        const int64_t at = (int64_t)(s.tail0 + t) * kB;
        El<DT>::store(out + at, lo2(f(pack2(El<DT>::load(row + at), 0.0f))));
    }
}

// Zeros in the elements of a slice, which is the logits' also where the output
// is aligned otherwise: a block never writes to another one's elements.
template <int DT, int NT>
__device__ __forceinline__ void zero_slice(char* out, const Slice& s)
{
    constexpr int kB = El<DT>::kBytes;
    char* p = out + (int64_t)s.first * kB;
    const RowSpan r = row_span<DT>(p, s.last - s.first);
    const int t = threadIdx.x;
    for (int i = t; i < r.nvec; i += NT)
        st16(p + r.head * kB + (int64_t)i * 16, make_uint4(0, 0, 0, 0));
    if (t < r.head) El<DT>::store(p + t * kB, 0.0f);
    if (t < r.tail) El<DT>::store(p + (int64_t)(r.head + r.nvec * El<DT>::kVec + t) * kB, 0.0f);
}

// ------------------------------------------------------------ launch shapes

// The distillation step's blocks for rows longer than kMidRow, and the most
// shared memory each stages.  Shorter ones are read twice instead: 8,192 rows
// of 16,000 bf16 take 92 us (staged 128; with blocks of 256 threads 99), of
// 24,000 149 and 151, of 32,000 224 and 176.  All resident blocks' rows have to
// stay in L2 until they are read again: with 12 blocks on an SM instead of 9,
// 16,000 take 106 us.
constexpr int kStepThreads = kRowThreads;
constexpr int kStageMax = 100 * 1024;

// Blocks on an SM that the compiler leaves registers for, the teacher's warp
// counted in.  The loss of 8,192 x 50,257 bf16 takes 137.6 us with 4, 129.6 with
// 5 and 133.6 with 6; fp32 rows need fewer registers.  The gradient with 5 takes
// 125 us at 4,096 x 50,257 bf16 against 127.6 with 7, but 37 to 38 at rows of 16
// to 32 KB against 33.  The step's two blocks are what shared memory holds; in
// blocks of 64 threads that read the row twice, 14, 16 and 20 take 23.4, 22.1 and
// 22.6 us at 8,192 x 2,000 bf16, 54.6, 54.1 and 58.9 at 8,192 x 8,000.
template <int DT, int NT>
constexpr int kLossBlocks = NT == kRowThreads ? (DT == DPZ_F32 ? 6 : 5) : NT == kMidThreads ? 10 : 20;
template <int NT>
constexpr int kGradBlocks = NT == kRowThreads ? 7 : NT == kMidThreads ? 8 : 20;
template <int NT>
constexpr int kRereadBlocks = NT == kRowThreads ? 4 : NT == kMidThreads ? 9 : 16;
constexpr int kStepBlocks = 2;

}  // namespace

}  // namespace dpz
