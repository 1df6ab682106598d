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
// Angles: a frequency is taken as a fraction of a turn in 128-bit fixed point, whose
// product with a 64-bit position wraps exactly: far positions lose nothing, where a
// product in fp32 is off by whole radians at 10^7.  The top 32 bits go to sincospi.
#include <cmath>
#include <type_traits>

#include "attn.h"
#include "bulk.cuh"
#include "device.cuh"
#include "lm_shape.h"

namespace dpz {

namespace {

constexpr int kRopeThreads = 256;

// A vector of V elements of type DT: as it lies in memory, and as fp32.
template <int DT, int V>
struct Vec;

template <>
struct Vec<DPZ_F32, 1> {
    using Raw = float;
    static __device__ __forceinline__ void unpack(const Raw& r, float x[1]) { x[0] = r; }
    static __device__ __forceinline__ Raw pack(const float x[1]) { return x[0]; }
};
template <>
struct Vec<DPZ_F32, 4> {
    using Raw = float4;
    static __device__ __forceinline__ void unpack(const Raw& r, float x[4])
    {
        x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
    }
    static __device__ __forceinline__ Raw pack(const float x[4])
    {
        return make_float4(x[0], x[1], x[2], x[3]);
    }
};
template <>
struct Vec<DPZ_BF16, 1> {
    using Raw = uint16_t;
    static __device__ __forceinline__ void unpack(const Raw& r, float x[1])
    {
        x[0] = __uint_as_float((uint32_t)r << 16);
    }
    static __device__ __forceinline__ Raw pack(const float x[1])
    {
        return (uint16_t)pack_bf16x2(x[0], 0.0f);
    }
};
template <>
struct Vec<DPZ_BF16, 4> {
    using Raw = uint2;
    static __device__ __forceinline__ void unpack(const Raw& r, float x[4])
    {
        x[0] = bf16_lo(r.x); x[1] = bf16_hi(r.x);
        x[2] = bf16_lo(r.y); x[3] = bf16_hi(r.y);
    }
    static __device__ __forceinline__ Raw pack(const float x[4])
    {
        return make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    }
};
template <>
struct Vec<DPZ_BF16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(const Raw& r, float x[8])
    {
        x[0] = bf16_lo(r.x); x[1] = bf16_hi(r.x);
        x[2] = bf16_lo(r.y); x[3] = bf16_hi(r.y);
        x[4] = bf16_lo(r.z); x[5] = bf16_hi(r.z);
        x[6] = bf16_lo(r.w); x[7] = bf16_hi(r.w);
    }
    static __device__ __forceinline__ Raw pack(const float x[8])
    {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                          pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
};

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

// Sines and cosines of a slot's pairs.  Pairs of two vectors: V of them.
// Neighbours: V / 2 in each vector, the identity past the rotated elements.
template <int V, int NS>
__device__ __forceinline__ void slot_turns(const Part<V, NS>& p, const RopeArgs& a,
                                           const Fraction* frac, int64_t t, float sn[NS][V],
                                           float cs[NS][V])
{
    const int64_t pos = a.positions ? position_of(a, t) : 0;
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sn[s][i] = 0.0f;
            cs[s][i] = 1.0f;
            int f = -1;
            if (a.interleaved && V > 1) {
                const int first = p.e[s][i < V / 2 ? 0 : 1];
                const int el = first + 2 * (i % (V / 2 > 0 ? V / 2 : 1));
                if (first >= 0 && el < a.R) f = el / 2;
            } else if (p.rotated[s]) {
                f = (a.interleaved ? p.e[s][0] / 2 : p.e[s][0]) + i;
            }
            if (f >= 0 && a.positions) turn_by(pos, frac[f], &sn[s][i], &cs[s][i]);
        }
}

// Rotates a slot by sign * angle.
template <int V>
__device__ __forceinline__ void rotate(float x[2][V], const float sn[V], const float cs[V],
                                       bool interleaved, float sign)
{
    if (interleaved && V > 1) {
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float c = cs[v * (V / 2) + i], s = sign * sn[v * (V / 2) + i];
                const float u = x[v][2 * i], w = x[v][(2 * i + 1) % V];
                x[v][2 * i] = fmaf(u, c, -w * s);
                x[v][(2 * i + 1) % V] = fmaf(w, c, u * s);
            }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float c = cs[i], s = sign * sn[i], u = x[0][i], w = x[1][i];
            x[0][i] = fmaf(u, c, -w * s);
            x[1][i] = fmaf(w, c, u * s);
        }
    }
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
    __device__ __forceinline__ void unpack(float x[NS][2][V]) const
    {
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int v = 0; v < 2; ++v) Vec<DT, V>::unpack(r[s][v], x[s][v]);
    }
};

template <int DT, int V, int NS>
__device__ __forceinline__ void store_slots(const Part<V, NS>& p, char* row, const float x[NS][2][V])
{
    constexpr int ES = DT == DPZ_BF16 ? 2 : 4;
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int v = 0; v < 2; ++v)
            if (p.e[s][v] >= 0)
                *reinterpret_cast<typename Vec<DT, V>::Raw*>(row + (int64_t)p.e[s][v] * ES) =
                    Vec<DT, V>::pack(x[s][v]);
}

template <int V, int NS>
__device__ __forceinline__ void load_weights(const Part<V, NS>& p, const void* w, int wdt,
                                             float x[NS][2][V])
{
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int at = p.e[s][v] + i;
                x[s][v][i] = w == nullptr || p.e[s][v] < 0 ? 1.0f
                             : wdt == DPZ_BF16
                                 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[at])
                                 : static_cast<const float*>(w)[at];
            }
}

template <int V, int NS>
__device__ __forceinline__ float dot(const float a[NS][2][V], const float b[NS][2][V], int lanes)
{
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int i = 0; i < V; ++i) s = fmaf(a[k][v][i], b[k][v][i], s);
    for (int o = 1; o < lanes; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// Row of head h of token t.
__device__ __forceinline__ char* head_row(const Heads& x, int64_t t, int h, int es)
{
    return x.p + (t * x.ld + (int64_t)h * x.hs) * es;
}

__device__ __forceinline__ void fill_fractions(const RopeArgs& a, Fraction* frac)
{
    for (int i = threadIdx.x; i < (a.positions ? a.R / 2 : 0); i += kRopeThreads)
        frac[i] = turn_fraction(a.inv_freq[i]);
    __syncthreads();
}

// An item is a token and `per` of the queries' (blockIdx.y = 0) or of the keys' heads, which
// share the token's sines and cosines; the next head's row is loaded while one is at work.

template <int DT, int V, int NS>
__global__ void __launch_bounds__(kRopeThreads, 3) k_rope(const __grid_constant__ RopeArgs a, int per)
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
    const int64_t item = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) / c.lanes;
    const bool live = item < a.T * each;     // every lane takes part in the exchanges
    const int64_t t = live ? item / each : 0;
    const int h0 = live ? (int)(item - t * each) * per : 0;
    const int n = live ? min(per, H - h0) : 0;
    RawSlots<DT, V, NS> raw;
    raw.load(p, head_row(a.in[k], t, h0, ES), n > 0);
    float sn[NS][V], cs[NS][V], w[NS][2][V];
    load_weights<V, NS>(p, a.w[k], a.wdt, w);
    slot_turns<V, NS>(p, a, frac, t, sn, cs);
    const float inv = 1.0f / (float)a.D;
    for (int b = 0; b < per; ++b) {
        float x[NS][2][V];
        raw.unpack(x);
        raw.load(p, head_row(a.in[k], t, h0 + b + 1, ES), b + 1 < n);
        const float r = rsqrtf(fmaf(dot<V, NS>(x, x, c.lanes), inv, a.eps));
#pragma unroll
        for (int s = 0; s < NS; ++s) {
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) (&x[s][0][0])[i] *= r * (&w[s][0][0])[i];
            rotate<V>(x[s], sn[s], cs[s], a.interleaved, 1.0f);
        }
        if (b < n) store_slots<DT, V, NS>(p, head_row(a.out[k], t, h0 + b, ES), x);
    }
}

// One block per part of the tokens, for the queries and for the keys; each group of lanes
// walks the part's items and keeps the weights' gradient of its slot, which are
// joined in the order of the groups at the end.
template <int DT, int V, int NS>
__global__ void __launch_bounds__(kRopeThreads, 2)
k_rope_grad(const __grid_constant__ RopeArgs a, int per)
{
    pdl_enter();
    constexpr int ES = DT == DPZ_BF16 ? 2 : 4;
    __shared__ Fraction frac[kRopeMaxD / 2];
    __shared__ float joined[kRopeThreads / 32][kRopeMaxD];
    fill_fractions(a, frac);
    const int k = blockIdx.y, H = a.H[k];
    const Cut c = make_cut<V>(a.D, a.R, a.interleaved);
    const int lane = threadIdx.x & (c.lanes - 1), groups = kRopeThreads / c.lanes;
    const Part<V, NS> p = my_part<V, NS>(c, lane, a);
    const int64_t tokens = rope_part_tokens(a.T), t0 = blockIdx.x * tokens;
    const unsigned each = (unsigned)(H + per - 1) / (unsigned)per;
    const int items = (int)min(tokens, a.T - t0) * (int)each;
    const float inv = 1.0f / (float)a.D;
    float w[NS][2][V], dw[NS][2][V] = {};
    load_weights<V, NS>(p, a.w[k], a.wdt, w);
    // whole warps go round the loop together
    for (int base = 0; base < items; base += groups) {
        const int item = base + (int)threadIdx.x / c.lanes;
        const bool live = item < items;
        const int64_t t = t0 + (live ? (int)((unsigned)item / each) : 0);
        const int h0 = live ? (int)((unsigned)item % each) * per : 0;
        const int n = live ? min(per, H - h0) : 0;
        RawSlots<DT, V, NS> rx, rd;
        rx.load(p, head_row(a.in[k], t, h0, ES), n > 0);
        rd.load(p, head_row(a.dout[k], t, h0, ES), n > 0);
        float sn[NS][V], cs[NS][V];
        slot_turns<V, NS>(p, a, frac, t, sn, cs);
        for (int b = 0; b < per; ++b) {
            float x[NS][2][V], d[NS][2][V];
            rx.unpack(x);
            rd.unpack(d);
            rx.load(p, head_row(a.in[k], t, h0 + b + 1, ES), b + 1 < n);
            rd.load(p, head_row(a.dout[k], t, h0 + b + 1, ES), b + 1 < n);
            const float r = rsqrtf(fmaf(dot<V, NS>(x, x, c.lanes), inv, a.eps));
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                rotate<V>(d[s], sn[s], cs[s], a.interleaved, -1.0f);
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) {
                    const float y = (&x[s][0][0])[i] *= r;
                    float& g = (&d[s][0][0])[i];
                    (&dw[s][0][0])[i] = fmaf(g, y, (&dw[s][0][0])[i]);
                    g *= (&w[s][0][0])[i];
                }
            }
            const float mean = dot<V, NS>(x, d, c.lanes) * inv;
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int i = 0; i < 2 * V; ++i)
                    (&d[s][0][0])[i] = r * fmaf(-mean, (&x[s][0][0])[i], (&d[s][0][0])[i]);
            if (b < n) store_slots<DT, V, NS>(p, head_row(a.out[k], t, h0 + b, ES), d);
        }
    }
    if (a.dw[0] == nullptr && a.dw[1] == nullptr) return;
    // the groups of a warp, then the warps, in a fixed order
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float y = dw[s][v][i];
                for (int o = c.lanes; o < 32; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                if ((threadIdx.x & 31) < c.lanes && p.e[s][v] >= 0)
                    joined[threadIdx.x >> 5][p.e[s][v] + i] = y;
            }
    __syncthreads();
    for (int i = threadIdx.x; i < a.D; i += kRopeThreads) {
        float y = 0.0f;
#pragma unroll
        for (int w = 0; w < kRopeThreads / 32; ++w) y += joined[w][i];
        a.partial[((int64_t)blockIdx.x * 2 + k) * a.D + i] = y;
    }
}

// The weights' gradients: 32 columns of the partial rows per block, 8 warps
// each taking every eighth row, joined in order.
constexpr int kDwThreads = 1024;

__global__ void __launch_bounds__(kDwThreads) k_rope_dw(RopeArgs a)
{
    pdl_enter();
    __shared__ double sums[kDwThreads / 32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane, cols = 2 * a.D;
    const int64_t rows = rope_parts(a.T);
    double y = 0.0;
    if (col < cols) {
        float s[4] = {};
        int64_t r = warp;
        for (; r + 3 * (kDwThreads / 32) < rows; r += 4 * (kDwThreads / 32))
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] += a.partial[(r + k * (kDwThreads / 32)) * cols + col];
        for (; r < rows; r += kDwThreads / 32) s[0] += a.partial[r * cols + col];
        y = ((double)s[0] + s[1]) + ((double)s[2] + s[3]);
    }
    sums[warp][lane] = y;
    __syncthreads();
    if (warp != 0 || col >= cols) return;
    double total = 0.0;
    for (int w = 0; w < kDwThreads / 32; ++w) total += sums[w][lane];
    const int k = col >= a.D, d = k ? col - a.D : col;
    if (a.dw[k] == nullptr) return;
    if (a.wdt == DPZ_BF16) static_cast<__nv_bfloat16*>(a.dw[k])[d] = __float2bfloat16_rn((float)total);
    else static_cast<float*>(a.dw[k])[d] = (float)total;
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

// Calls f with the type, the vector and the slots of a lane as constants.
template <class F>
cudaError_t by_vector(const RopeArgs& a, bool grad, F&& f)
{
    using std::integral_constant;
    const int v = vector_of(a, grad);
    if (a.dt == DPZ_BF16) {
        constexpr integral_constant<int, DPZ_BF16> dt{};
        if (v == 8) return f(dt, integral_constant<int, 8>{}, integral_constant<int, 1>{});
        if (v == 4) return f(dt, integral_constant<int, 4>{}, integral_constant<int, 1>{});
        return f(dt, integral_constant<int, 1>{}, integral_constant<int, 4>{});
    }
    constexpr integral_constant<int, DPZ_F32> dt{};
    if (v == 4) return f(dt, integral_constant<int, 4>{}, integral_constant<int, 1>{});
    return f(dt, integral_constant<int, 1>{}, integral_constant<int, 4>{});
}

}  // namespace

// Heads of an item, by sizes alone (the sums' order follows it): up to 16, fewer while
// the items would leave most of the GPU without work.
int heads_of_item(int64_t tokens, int H, int lanes, int64_t threads)
{
    int per = 16;
    while (per > 1 && tokens * ((H + per - 1) / per) * lanes < threads) per /= 2;
    return per;
}

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s)
{
    set_last_kernel_name("attn_qk_norm_rope");
    return by_vector(a, false, [&](auto dt, auto v, auto ns) {
        const Cut c = make_cut<v>(a.D, a.R, a.interleaved);
        const int H = a.H[0] > a.H[1] ? a.H[0] : a.H[1];
        const int per = heads_of_item(a.T, H, c.lanes, 152 * 768);
        const int64_t threads = a.T * ((H + per - 1) / per) * c.lanes;
        const unsigned blocks = (unsigned)((threads + kRopeThreads - 1) / kRopeThreads);
        return launch_kernel(k_rope<dt, v, ns>, dim3(blocks, a.H[1] > 0 ? 2 : 1), dim3(kRopeThreads),
                             0, s, true, 0u, a, per);
    });
}

cudaError_t launch_rope_grad(const RopeArgs& a, cudaStream_t s)
{
    set_last_kernel_name("attn_qk_norm_rope_grad");
    return by_vector(a, true, [&](auto dt, auto v, auto ns) {
        const Cut c = make_cut<v>(a.D, a.R, a.interleaved);
        const int H = a.H[0] > a.H[1] ? a.H[0] : a.H[1];
        const int per = heads_of_item(rope_part_tokens(a.T), H, c.lanes, kRopeThreads);
        return launch_kernel(k_rope_grad<dt, v, ns>, dim3((unsigned)rope_parts(a.T), 2),
                             dim3(kRopeThreads), 0, s, true, 0u, a, per);
    });
}

cudaError_t launch_rope_dw(const RopeArgs& a, cudaStream_t s)
{
    set_last_kernel_name("attn_qk_norm_rope_dw");
    return launch_kernel(k_rope_dw, dim3((unsigned)((2 * a.D + 31) / 32)), dim3(kDwThreads), 0, s,
                         true, 0u, a);
}

}  // namespace dpz
