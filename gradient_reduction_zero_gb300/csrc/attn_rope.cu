// The norm of every head of queries and keys with the position rotation, in
// one pass, and its gradient.
//
//   n = x * rsqrt(mean(x^2) + eps),  y = R(angle) (w * n),  angle_i = position * inv_freq_i
//   g = R(-angle) dy,  dw = sum g * n,  dx = rsqrt(..) * (w g - n mean(w g n))
//
// Bound by HBM: every element is read once and written once, everything else
// stays in registers.  A lane holds one slot of a head: two vectors of V
// elements, chosen so that both elements of each rotated pair are the lane's
// own (vectors v and v + R/2/V when pairs are half a rotation apart, neighbours
// otherwise), so that the rotation needs no exchange; 2^k lanes share a
// head.  A group of lanes takes one token and several of its heads, and
// computes the token's sines and cosines once for all of them.
//
// Measured: 16,384 tokens of 32 + 8 heads of 128 in bf16 67 us (5.0 TB/s); the gradient of
// 32,768 tokens of 25 + 25 heads of 64 159 us (4.0 TB/s).
//
// Angles: a frequency is taken as a fraction of a turn in 128-bit fixed point, whose
// product with a 64-bit position wraps exactly: far positions lose nothing, where a
// product in fp32 is off by whole radians at 10^7.  The top 32 bits go to sincospi.
#include <cmath>
#include <type_traits>

#include "attn.h"
#include "bulk.cuh"
#include "device.cuh"
#include "pairs.cuh"

namespace dpz {

namespace {

// Threads of a block, rows that a lane has under way, and blocks that stay: what the registers
// hold decides the speed (bytes in flight), not the arithmetic.  One row under way 87 us, four
// 83 (67 with blocks that stay and heads shared out evenly); the gradient 159 us with two
// blocks of 256 threads an SM and one row, 226 with three of vectors half as long and
// two rows, and before the heads were shared out evenly 173 against 254 with one block of 384
// and two rows.
constexpr int kRopeThreads = 256, kRopeAhead = 4, kRopeBlocks = 304;
constexpr int kRopeGradThreads = 256, kRopeGradAhead = 1;

// A vector of V elements of type DT: as it lies in memory, and as fp32 in pairs (a single
// element as a float).
template <int DT, int V>
struct Vec;

template <>
struct Vec<DPZ_F32, 1> {
    using Raw = float;
    static __device__ __forceinline__ float one(Raw r) { return r; }
    static __device__ __forceinline__ Raw back(float x) { return x; }
};
template <>
struct Vec<DPZ_BF16, 1> {
    using Raw = uint16_t;
    static __device__ __forceinline__ float one(Raw r) { return __uint_as_float((uint32_t)r << 16); }
    static __device__ __forceinline__ Raw back(float x) { return (uint16_t)pack_bf16x2(x, 0.0f); }
};
template <>
struct Vec<DPZ_F32, 4> {
    using Raw = float4;
    static __device__ __forceinline__ void unpack(const Raw& r, F2 x[2])
    {
        x[0] = pack2(r.x, r.y);
        x[1] = pack2(r.z, r.w);
    }
    static __device__ __forceinline__ Raw pack(const F2 x[2])
    {
        return make_float4(lo2(x[0]), hi2(x[0]), lo2(x[1]), hi2(x[1]));
    }
};
template <>
struct Vec<DPZ_BF16, 4> {
    using Raw = uint2;
    static __device__ __forceinline__ void unpack(const Raw& r, F2 x[2])
    {
        x[0] = pack2(bf16_lo(r.x), bf16_hi(r.x));
        x[1] = pack2(bf16_lo(r.y), bf16_hi(r.y));
    }
    static __device__ __forceinline__ Raw pack(const F2 x[2])
    {
        return make_uint2(pack_bf16x2(lo2(x[0]), hi2(x[0])), pack_bf16x2(lo2(x[1]), hi2(x[1])));
    }
};
template <>
struct Vec<DPZ_BF16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(const Raw& r, F2 x[4])
    {
        x[0] = pack2(bf16_lo(r.x), bf16_hi(r.x));
        x[1] = pack2(bf16_lo(r.y), bf16_hi(r.y));
        x[2] = pack2(bf16_lo(r.z), bf16_hi(r.z));
        x[3] = pack2(bf16_lo(r.w), bf16_hi(r.w));
    }
    static __device__ __forceinline__ Raw pack(const F2 x[4])
    {
        return make_uint4(pack_bf16x2(lo2(x[0]), hi2(x[0])), pack_bf16x2(lo2(x[1]), hi2(x[1])),
                          pack_bf16x2(lo2(x[2]), hi2(x[2])), pack_bf16x2(lo2(x[3]), hi2(x[3])));
    }
};

// Register pairs of a slot: those of its first vector, then of its second; with single
// elements, one pair of the two.
template <int V>
constexpr int kPairs = V == 1 ? 1 : V;

// How a head is cut: `pairs` slots hold rotated pairs of vectors, the rest two
// vectors each of what is not rotated (the last may hold one).
struct Cut {
    int pairs, slots, lanes;   // lanes: of a head, a power of two
    int half;                  // R / 2
    int vecs;                  // vectors of a head
};

template <int V>
DPZ_HD inline Cut make_cut(int D, int R, bool interleaved)
{
    Cut c;
    c.half = R / 2;
    c.vecs = D / V;
    // neighbours form a pair: any two vectors make a slot
    c.pairs = interleaved && V > 1 ? 0 : c.half / V;
    const int rest = interleaved && V > 1 ? c.vecs : c.vecs - 2 * c.pairs;
    c.slots = c.pairs + (rest + 1) / 2;
    c.lanes = 1;
    while (c.lanes < 32 && c.lanes < c.slots) c.lanes *= 2;
    return c;
}

// The two first elements of a slot; -1: no such vector.
template <int V>
__device__ __forceinline__ void slot_elems(const Cut& c, int slot, int D, bool interleaved, int e[2])
{
    if (slot >= c.slots) {
        e[0] = e[1] = -1;
    } else if (slot < c.pairs) {
        e[0] = interleaved ? 2 * slot : slot * V;          // interleaved here: V = 1
        e[1] = interleaved ? 2 * slot + 1 : slot * V + c.half;
    } else {
        const int base = 2 * c.pairs * V, n = c.slots - c.pairs, i = slot - c.pairs;
        e[0] = base + i * V;
        e[1] = base + (i + n) * V;
        if (e[1] >= D) e[1] = -1;
    }
}

// A fraction of a turn in units of 2^-128.
struct Fraction {
    uint64_t hi, lo;
};

// 64 bits of the number p from bit b on, 0 <= b.
__device__ __forceinline__ uint64_t bits_from(const uint64_t p[4], int b)
{
    const int i = b >> 6, r = b & 63;
    const uint64_t x = i == 0 ? p[0] : i == 1 ? p[1] : i == 2 ? p[2] : i == 3 ? p[3] : 0;
    const uint64_t y = i == 0 ? p[1] : i == 1 ? p[2] : i == 2 ? p[3] : 0;
    return r == 0 ? x : x >> r | y << (64 - r);
}

// f / (2 pi) modulo 1, rounded towards 0: the mantissa times 1 / (2 pi) in 192 bits, shifted
// by the exponent.
__device__ __forceinline__ Fraction turn_fraction(float f)
{
    // floor(2^192 / (2 pi)), high word first
    const uint64_t c2 = 0x28be60db9391054aull, c1 = 0x7f09d5f47d4d3770ull, c0 = 0x36d8a5664f10e410ull;
    const uint32_t b = __float_as_uint(f);
    const int ex = (int)(b >> 23 & 255);
    const uint64_t m = ex ? (b & 0x7fffff) | 0x800000 : b & 0x7fffff;
    const int e = (ex ? ex : 1) - 150;              // |f| = m 2^e
    uint64_t p[4];
    p[0] = m * c0;
    const uint64_t h0 = __umul64hi(m, c0);
    p[1] = m * c1 + h0;
    const uint64_t h1 = __umul64hi(m, c1) + (p[1] < h0);
    p[2] = m * c2 + h1;
    p[3] = __umul64hi(m, c2) + (p[2] < h1);
    const int sh = max(64 - e, 0);                  // |f| < 2^88 is exact
    const uint64_t hi = bits_from(p, sh + 64), lo = bits_from(p, sh);
    if (b >> 31) return {~hi + (lo == 0), 0 - lo};
    return {hi, lo};
}

__device__ __forceinline__ int64_t position_of(const RopeArgs& a, int64_t t)
{
    return a.itype == DPZ_I64 ? static_cast<const int64_t*>(a.positions)[t]
                              : (int64_t) static_cast<const int*>(a.positions)[t];
}

// Sine and cosine of position * frequency: the product's top 64 bits of the turn's fraction.
__device__ __forceinline__ void turn_by(int64_t pos, const Fraction& f, float* s, float* c)
{
    const uint64_t u = (uint64_t)pos * f.hi + __umul64hi((uint64_t)pos, f.lo) -
                       (pos < 0 ? f.lo : 0);
    const float half_turns = (float)(int32_t)(u >> 32) * 0x1p-31f;   // in [-1, 1]
    sincospif(half_turns, s, c);
}

// The whole of a lane's part of a head.
template <int V, int NS>
struct Part {
    int e[NS][2];        // first elements of its vectors
    bool rotated[NS];
};

template <int V, int NS>
__device__ __forceinline__ Part<V, NS> my_part(const Cut& c, int lane, const RopeArgs& a)
{
    Part<V, NS> p;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        slot_elems<V>(c, lane + s * c.lanes, a.D, a.interleaved, p.e[s]);
        p.rotated[s] = lane + s * c.lanes < c.pairs;
    }
    return p;
}

// The element that half h (0 or 1) of register pair q of a slot holds.
template <int V, int NS>
__device__ __forceinline__ int elem_of(const Part<V, NS>& p, int s, int q, int h)
{
    if (V == 1) return p.e[s][h];
    const int first = p.e[s][q / (V / 2 > 0 ? V / 2 : 1)];
    return first < 0 ? -1 : first + 2 * (q % (V / 2 > 0 ? V / 2 : 1)) + h;
}

// A lane's sines and cosines.  SWAP (both elements of a rotated pair in one register pair:
// neighbours, or single elements): (cos, sin) of each register pair.  Otherwise a pair's
// elements are in the same place of the two vectors: cosines of a vector's places, then sines.
template <int V, int NS>
struct Turns {
    F2 t[NS][kPairs<V>];
};

template <bool SWAP, int V, int NS>
__device__ __forceinline__ Turns<V, NS> turns_of(const Part<V, NS>& p, const RopeArgs& a,
                                                 const Fraction* frac, int64_t t)
{
    const int64_t pos = a.positions ? position_of(a, t) : 0;
    const auto turn = [&](int f, float* sn, float* cs) {
        *sn = 0.0f;
        *cs = 1.0f;
        if (f >= 0 && a.positions) turn_by(pos, frac[f], sn, cs);
    };
    Turns<V, NS> r;
#pragma unroll
    for (int s = 0; s < NS; ++s)
        if (SWAP) {
#pragma unroll
            for (int q = 0; q < kPairs<V>; ++q) {
                const int el = elem_of<V, NS>(p, s, q, 0);
                int f = -1;
                if (V == 1) {
                    if (p.rotated[s]) f = a.interleaved ? el / 2 : el;
                } else if (el >= 0 && el < a.R) {
                    f = el / 2;
                }
                float sn, cs;
                turn(f, &sn, &cs);
                r.t[s][q] = pack2(cs, sn);
            }
        } else {
#pragma unroll
            for (int q = 0; q < V / 2; ++q) {
                const int f = p.rotated[s] ? p.e[s][0] + 2 * q : -1;
                float sn[2], cs[2];
                turn(f, &sn[0], &cs[0]);
                turn(f < 0 ? -1 : f + 1, &sn[1], &cs[1]);
                r.t[s][q] = pack2(cs[0], cs[1]);
                r.t[s][(q + V / 2) % kPairs<V>] = pack2(sn[0], sn[1]);
            }
        }
    return r;
}

// With a pair's partner in y, x * m[0] + y * m[1] is its rotation by the lane's angles
// (back: by their negatives).
template <bool SWAP, int V, int NS>
__device__ __forceinline__ void matrix_of(const Turns<V, NS>& r, int s, int q, bool back, F2 m[2])
{
    if (SWAP) {
        const float cs = lo2(r.t[s][q]), sn = back ? -hi2(r.t[s][q]) : hi2(r.t[s][q]);
        m[0] = pack2(cs, cs);
        m[1] = pack2(-sn, sn);
    } else {
        const int k = q % (V / 2 > 0 ? V / 2 : 1);
        const F2 sn = r.t[s][(k + V / 2) % kPairs<V>];
        const bool minus = (q < V / 2) != back;
        m[0] = r.t[s][k];
        m[1] = minus ? sn ^ 0x8000000080000000ull : sn;
    }
}

template <bool SWAP, int V>
__device__ __forceinline__ F2 partner(const F2 x[kPairs<V>], int q)
{
    return SWAP ? swap2(x[q]) : x[(q + V / 2) % kPairs<V>];
}

// A lane's part of a row as it lies in memory; zeros where it has none or `on` is false.
template <int DT, int V, int NS>
struct RawSlots {
    typename Vec<DT, V>::Raw r[NS][2];

    __device__ __forceinline__ void load(const Part<V, NS>& p, const char* row, bool on)
    {
        constexpr int ES = DT == DPZ_BF16 ? 2 : 4;
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                r[s][v] = {};
                if (on && p.e[s][v] >= 0)
                    r[s][v] = *reinterpret_cast<const typename Vec<DT, V>::Raw*>(
                        row + (int64_t)p.e[s][v] * ES);
            }
    }
    __device__ __forceinline__ void unpack(F2 x[NS][kPairs<V>]) const
    {
#pragma unroll
        for (int s = 0; s < NS; ++s)
            if constexpr (V == 1) {
                x[s][0] = pack2(Vec<DT, 1>::one(r[s][0]), Vec<DT, 1>::one(r[s][1]));
            } else {
                Vec<DT, V>::unpack(r[s][0], x[s]);
                Vec<DT, V>::unpack(r[s][1], x[s] + V / 2);
            }
    }
};

template <int DT, int V, int NS>
__device__ __forceinline__ void store_slots(const Part<V, NS>& p, char* row,
                                            const F2 x[NS][kPairs<V>])
{
    constexpr int ES = DT == DPZ_BF16 ? 2 : 4;
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            typename Vec<DT, V>::Raw r;
            if constexpr (V == 1) r = Vec<DT, 1>::back(v ? hi2(x[s][0]) : lo2(x[s][0]));
            else r = Vec<DT, V>::pack(x[s] + v * (V / 2));
            if (p.e[s][v] >= 0)
                *reinterpret_cast<typename Vec<DT, V>::Raw*>(row + (int64_t)p.e[s][v] * ES) = r;
        }
}

template <int V, int NS>
__device__ __forceinline__ void load_weights(const Part<V, NS>& p, const void* w, int wdt,
                                             F2 x[NS][kPairs<V>])
{
    const auto weight = [&](int at) {
        return w == nullptr || at < 0 ? 1.0f
               : wdt == DPZ_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[at])
                                 : static_cast<const float*>(w)[at];
    };
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int q = 0; q < kPairs<V>; ++q)
            x[s][q] = pack2(weight(elem_of<V, NS>(p, s, q, 0)), weight(elem_of<V, NS>(p, s, q, 1)));
}

// The sum of products over a head, whole in each of its lanes.
template <int V, int NS>
__device__ __forceinline__ float dot(const F2 a[NS][kPairs<V>], const F2 b[NS][kPairs<V>], int lanes)
{
    F2 t[2] = {0, 0};
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int q = 0; q < kPairs<V>; ++q)
            t[(s + q) & 1] = fma2(a[s][q], b[s][q], t[(s + q) & 1]);
    t[0] = add2(t[0], t[1]);
    float y = lo2(t[0]) + hi2(t[0]);
    for (int o = 1; o < lanes; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    return y;
}

// Row of head h of token t.
__device__ __forceinline__ char* head_row(const Heads& x, int64_t t, int h, int es)
{
    return x.p + (t * x.ld + (int64_t)h * x.hs) * es;
}

__device__ __forceinline__ void fill_fractions(const RopeArgs& a, Fraction* frac)
{
    for (int i = threadIdx.x; i < (a.positions ? a.R / 2 : 0); i += blockDim.x)
        frac[i] = turn_fraction(a.inv_freq[i]);
    __syncthreads();
}

// An item is a token and `per` of the queries' (blockIdx.y = 0) or of the keys' heads, which
// share the token's sines and cosines; the next head's row is loaded while one is at work.

template <int DT, int V, int NS, bool SWAP>
__global__ void __launch_bounds__(kRopeThreads, 2) k_rope(const __grid_constant__ RopeArgs a, int per)
{
    pdl_enter();
    constexpr int ES = DT == DPZ_BF16 ? 2 : 4;
    __shared__ Fraction frac[kRopeMaxD / 2];
    fill_fractions(a, frac);
    const int k = blockIdx.y, H = a.H[k];
    const Cut c = make_cut<V>(a.D, a.R, a.interleaved);
    const int lane = threadIdx.x & (c.lanes - 1);
    const Part<V, NS> p = my_part<V, NS>(c, lane, a);
    const unsigned each = (unsigned)(H + per - 1) / (unsigned)per;
    const int64_t items = a.T * each, step = (int64_t)gridDim.x * (kRopeThreads / c.lanes);
    const float inv = 1.0f / (float)a.D;
    F2 w[NS][kPairs<V>];
    load_weights<V, NS>(p, a.w[k], a.wdt, w);
    // whole warps go round the loop together: every lane takes part in the exchanges
    for (int64_t base = (int64_t)blockIdx.x * (kRopeThreads / c.lanes); base < items; base += step) {
        const int64_t item = base + threadIdx.x / c.lanes;
        const bool live = item < items;
        const int64_t t = live ? item / each : 0;
        const int h0 = live ? (int)(item - t * each) * per : 0;
        const int n = live ? min(per, H - h0) : 0;
        RawSlots<DT, V, NS> raw[kRopeAhead];
#pragma unroll
        for (int j = 0; j < kRopeAhead; ++j) raw[j].load(p, head_row(a.in[k], t, h0 + j, ES), j < n);
        // the weights are in the rotation's factors
        F2 own[NS][kPairs<V>], other[NS][kPairs<V>];
        {
            const Turns<V, NS> turns = turns_of<SWAP, V, NS>(p, a, frac, t);
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int q = 0; q < kPairs<V>; ++q) {
                    F2 m[2];
                    matrix_of<SWAP, V, NS>(turns, s, q, false, m);
                    own[s][q] = mul2(w[s][q], m[0]);
                    other[s][q] = mul2(partner<SWAP, V>(w[s], q), m[1]);
                }
        }
        for (int b0 = 0; b0 < min(per, H); b0 += kRopeAhead)
#pragma unroll
            for (int j = 0; j < kRopeAhead; ++j) {
                const int b = b0 + j;
                F2 x[NS][kPairs<V>], y[NS][kPairs<V>];
                raw[j].unpack(x);
                raw[j].load(p, head_row(a.in[k], t, h0 + b + kRopeAhead, ES), b + kRopeAhead < n);
                const float r = rsqrtf(fmaf(dot<V, NS>(x, x, c.lanes), inv, a.eps));
                const F2 rr = pack2(r, r);
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int q = 0; q < kPairs<V>; ++q)
                        y[s][q] = mul2(rr, fma2(x[s][q], own[s][q],
                                                mul2(partner<SWAP, V>(x[s], q), other[s][q])));
                if (b < n) store_slots<DT, V, NS>(p, head_row(a.out[k], t, h0 + b, ES), y);
            }
    }
}

// One block per part of the tokens, for the queries and for the keys; each group of lanes
// walks the part's items and keeps the weights' gradient of its slot, which are
// joined in the order of the groups at the end.
template <int DT, int V, int NS, bool SWAP>
__global__ void __launch_bounds__(kRopeGradThreads, 2)
k_rope_grad(const __grid_constant__ RopeArgs a, int per)
{
    pdl_enter();
    constexpr int ES = DT == DPZ_BF16 ? 2 : 4;
    __shared__ Fraction frac[kRopeMaxD / 2];
    __shared__ float joined[kRopeGradThreads / 32][kRopeMaxD];
    fill_fractions(a, frac);
    const int k = blockIdx.y, H = a.H[k];
    const Cut c = make_cut<V>(a.D, a.R, a.interleaved);
    const int lane = threadIdx.x & (c.lanes - 1), groups = kRopeGradThreads / c.lanes;
    const Part<V, NS> p = my_part<V, NS>(c, lane, a);
    const int64_t tokens = rope_part_tokens(a.T), t0 = blockIdx.x * tokens;
    const unsigned each = (unsigned)(H + per - 1) / (unsigned)per;
    const int items = (int)min(tokens, a.T - t0) * (int)each;
    const float inv = 1.0f / (float)a.D;
    F2 w[NS][kPairs<V>], dw[NS][kPairs<V>] = {};
    load_weights<V, NS>(p, a.w[k], a.wdt, w);
    // whole warps go round the loop together
    for (int base = 0; base < items; base += groups) {
        const int item = base + (int)threadIdx.x / c.lanes;
        const bool live = item < items;
        const int64_t t = t0 + (live ? (int)((unsigned)item / each) : 0);
        const int h0 = live ? (int)((unsigned)item % each) * per : 0;
        const int n = live ? min(per, H - h0) : 0;
        RawSlots<DT, V, NS> rx[kRopeGradAhead], rd[kRopeGradAhead];
#pragma unroll
        for (int j = 0; j < kRopeGradAhead; ++j) {
            rx[j].load(p, head_row(a.in[k], t, h0 + j, ES), j < n);
            rd[j].load(p, head_row(a.dout[k], t, h0 + j, ES), j < n);
        }
        const Turns<V, NS> turns = turns_of<SWAP, V, NS>(p, a, frac, t);
        for (int b0 = 0; b0 < min(per, H); b0 += kRopeGradAhead)
#pragma unroll
        for (int j = 0; j < kRopeGradAhead; ++j) {
            const int b = b0 + j;
            F2 x[NS][kPairs<V>], d[NS][kPairs<V>];
            rx[j].unpack(x);
            rd[j].unpack(d);
            rx[j].load(p, head_row(a.in[k], t, h0 + b + kRopeGradAhead, ES), b + kRopeGradAhead < n);
            rd[j].load(p, head_row(a.dout[k], t, h0 + b + kRopeGradAhead, ES),
                       b + kRopeGradAhead < n);
            const float r = rsqrtf(fmaf(dot<V, NS>(x, x, c.lanes), inv, a.eps));
            const F2 rr = pack2(r, r);
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                F2 g[kPairs<V>];
#pragma unroll
                for (int q = 0; q < kPairs<V>; ++q) {
                    F2 m[2];
                    matrix_of<SWAP, V, NS>(turns, s, q, true, m);
                    g[q] = fma2(d[s][q], m[0], mul2(partner<SWAP, V>(d[s], q), m[1]));
                }
#pragma unroll
                for (int q = 0; q < kPairs<V>; ++q) {
                    x[s][q] = mul2(x[s][q], rr);
                    dw[s][q] = fma2(g[q], x[s][q], dw[s][q]);
                    d[s][q] = mul2(g[q], w[s][q]);
                }
            }
            const float mean = dot<V, NS>(x, d, c.lanes) * inv;
            const F2 mm = pack2(-mean, -mean);
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int q = 0; q < kPairs<V>; ++q)
                    d[s][q] = mul2(rr, fma2(mm, x[s][q], d[s][q]));
            if (b < n) store_slots<DT, V, NS>(p, head_row(a.out[k], t, h0 + b, ES), d);
        }
    }
    if (a.dw[0] == nullptr && a.dw[1] == nullptr) return;
    // the groups of a warp, then the warps, in a fixed order
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int q = 0; q < kPairs<V>; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float y = h ? hi2(dw[s][q]) : lo2(dw[s][q]);
                for (int o = c.lanes; o < 32; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                const int at = elem_of<V, NS>(p, s, q, h);
                if ((threadIdx.x & 31) < c.lanes && at >= 0) joined[threadIdx.x >> 5][at] = y;
            }
    __syncthreads();
    for (int i = threadIdx.x; i < a.D; i += kRopeGradThreads) {
        float y = 0.0f;
#pragma unroll
        for (int w = 0; w < kRopeGradThreads / 32; ++w) y += joined[w][i];
        a.partial[((int64_t)blockIdx.x * 2 + k) * a.D + i] = y;
    }
}

// The weights' gradients: 8 columns of the partial rows per block, 128 threads to a column,
// each with every 128th row, joined in order.
constexpr int kDwThreads = 1024, kDwCols = 8, kDwRows = kDwThreads / kDwCols;

__global__ void __launch_bounds__(kDwThreads) k_rope_dw(const __grid_constant__ RopeArgs a)
{
    pdl_enter();
    __shared__ double sums[kDwThreads / 32][kDwCols];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * kDwCols + (lane & 7), cols = 2 * a.D;
    const int64_t rows = rope_parts(a.T);
    double y = 0.0;
    if (col < cols) {
        float s[8] = {};
        for (int64_t r = threadIdx.x / kDwCols; r < rows; r += 8 * kDwRows)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (r + k * kDwRows < rows) s[k] += a.partial[(r + k * kDwRows) * cols + col];
        y = (((double)s[0] + s[1]) + ((double)s[2] + s[3])) +
            (((double)s[4] + s[5]) + ((double)s[6] + s[7]));
    }
    y += __shfl_xor_sync(0xffffffffu, y, 8);
    y += __shfl_xor_sync(0xffffffffu, y, 16);
    if (lane < kDwCols) sums[warp][lane] = y;
    __syncthreads();
    if (threadIdx.x >= kDwCols || col >= cols) return;
    double t[4] = {};
#pragma unroll
    for (int w = 0; w < kDwThreads / 32; ++w) t[w & 3] += sums[w][lane];
    const float total = (float)((t[0] + t[1]) + (t[2] + t[3]));
    const int k = col >= a.D, d = k ? col - a.D : col;
    if (a.dw[k] == nullptr) return;
    if (a.wdt == DPZ_BF16) static_cast<__nv_bfloat16*>(a.dw[k])[d] = __float2bfloat16_rn(total);
    else static_cast<float*>(a.dw[k])[d] = total;
}

// Elements of a vector that every row of every tensor of the call allows.
int vector_of(const RopeArgs& a, bool grad)
{
    const int es = a.dt == DPZ_BF16 ? 2 : 4;
    uintptr_t bits = 0;
    const auto look = [&](const Heads& h) {
        bits |= reinterpret_cast<uintptr_t>(h.p) | (uintptr_t)(h.ld * es) | (uintptr_t)(h.hs * es);
    };
    for (int k = 0; k < 2; ++k) {
        if (a.H[k] == 0) continue;
        look(a.in[k]);
        look(a.out[k]);
        if (grad) look(a.dout[k]);
    }
    for (int v = 16 / es; v >= 4; v /= 2) {
        const bool whole = a.D % v == 0 && (a.interleaved ? true : (a.R / 2) % v == 0);
        if (whole && bits % (v * es) == 0) return v;
    }
    return 1;
}

// Calls f with the type, the vector, the slots of a lane and whether a rotated pair is in one
// register pair as constants.
template <class F>
cudaError_t by_vector(const RopeArgs& a, bool grad, F&& f)
{
    using std::integral_constant;
    const int v = vector_of(a, grad);
    const auto style = [&](auto dt, auto vec) {
        constexpr integral_constant<int, 1> ns{};
        return a.interleaved ? f(dt, vec, ns, std::true_type{}) : f(dt, vec, ns, std::false_type{});
    };
    if (a.dt == DPZ_BF16) {
        constexpr integral_constant<int, DPZ_BF16> dt{};
        if (v == 8) return style(dt, integral_constant<int, 8>{});
        if (v == 4) return style(dt, integral_constant<int, 4>{});
        return f(dt, integral_constant<int, 1>{}, integral_constant<int, 4>{}, std::true_type{});
    }
    constexpr integral_constant<int, DPZ_F32> dt{};
    if (v == 4) return style(dt, integral_constant<int, 4>{});
    return f(dt, integral_constant<int, 1>{}, integral_constant<int, 4>{}, std::true_type{});
}

}  // namespace

// Heads of an item, by sizes alone (the sums' order follows it): up to `most`, fewer while
// the items would leave most of the threads without work, and about equally many in each item
// (25 heads as 4 x 7, not 16 + 9).
int heads_of_item(int64_t tokens, int H, int lanes, int64_t threads, int most)
{
    int per = most;
    while (per > 1 && tokens * ((H + per - 1) / per) * lanes < threads) per /= 2;
    const int each = (H + per - 1) / per;
    return each > 0 ? (H + each - 1) / each : 1;
}

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s)
{
    set_last_kernel_name("attn_qk_norm_rope");
    return by_vector(a, false, [&](auto dt, auto v, auto ns, auto swap) {
        const Cut c = make_cut<v>(a.D, a.R, a.interleaved);
        const int H = a.H[0] > a.H[1] ? a.H[0] : a.H[1];
        const int per = heads_of_item(a.T, H, c.lanes, 152 * 768, 16);
        const int64_t threads = a.T * ((H + per - 1) / per) * c.lanes;
        const int64_t need = (threads + kRopeThreads - 1) / kRopeThreads;
        const unsigned blocks = (unsigned)(need < kRopeBlocks ? need : kRopeBlocks);
        return launch_kernel(k_rope<dt, v, ns, swap>, dim3(blocks, a.H[1] > 0 ? 2 : 1), dim3(kRopeThreads),
                             0, s, true, 0u, a, per);
    });
}

cudaError_t launch_rope_grad(const RopeArgs& a, cudaStream_t s)
{
    set_last_kernel_name("attn_qk_norm_rope_grad");
    return by_vector(a, true, [&](auto dt, auto v, auto ns, auto swap) {
        const Cut c = make_cut<v>(a.D, a.R, a.interleaved);
        const int H = a.H[0] > a.H[1] ? a.H[0] : a.H[1];
        const int per = heads_of_item(rope_part_tokens(a.T), H, c.lanes, kRopeGradThreads, 8);
        return launch_kernel(k_rope_grad<dt, v, ns, swap>, dim3((unsigned)rope_parts(a.T), 2),
                             dim3(kRopeGradThreads), 0, s, true, 0u, a, per);
    });
}

cudaError_t launch_rope_dw(const RopeArgs& a, cudaStream_t s)
{
    set_last_kernel_name("attn_qk_norm_rope_dw");
    return launch_kernel(k_rope_dw, dim3((unsigned)((2 * a.D + kDwCols - 1) / kDwCols)), dim3(kDwThreads), 0, s,
                         true, 0u, a);
}

}  // namespace dpz
