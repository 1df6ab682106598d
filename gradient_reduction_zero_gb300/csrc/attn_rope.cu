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
// Angles: a position times a frequency is taken as a fraction of a turn in 64-bit
// fixed point, whose product with an integer position wraps exactly: far
// positions lose nothing, where a product in fp32 is off by whole radians at
// 10^7.  The top 32 bits go to sincospi.
#include <cmath>
#include <type_traits>

#include "attn.h"
#include "bulk.cuh"
#include "device.cuh"
#include "lm_shape.h"

namespace dpz {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kHeadsPerItem = 8;    // heads that share a token's sines and cosines

// A vector of V elements of type DT as fp32.
template <int DT, int V>
struct Vec;

template <>
struct Vec<DPZ_F32, 1> {
    static __device__ __forceinline__ void load(const char* p, float x[1])
    {
        x[0] = *reinterpret_cast<const float*>(p);
    }
    static __device__ __forceinline__ void store(char* p, const float x[1])
    {
        *reinterpret_cast<float*>(p) = x[0];
    }
};
template <>
struct Vec<DPZ_F32, 4> {
    static __device__ __forceinline__ void load(const char* p, float x[4])
    {
        const float4 v = *reinterpret_cast<const float4*>(p);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    }
    static __device__ __forceinline__ void store(char* p, const float x[4])
    {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    }
};
template <>
struct Vec<DPZ_BF16, 1> {
    static __device__ __forceinline__ void load(const char* p, float x[1])
    {
        x[0] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
    }
    static __device__ __forceinline__ void store(char* p, const float x[1])
    {
        *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(x[0]);
    }
};
template <>
struct Vec<DPZ_BF16, 4> {
    static __device__ __forceinline__ void load(const char* p, float x[4])
    {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x);
        x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
    }
    static __device__ __forceinline__ void store(char* p, const float x[4])
    {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    }
};
template <>
struct Vec<DPZ_BF16, 8> {
    static __device__ __forceinline__ void load(const char* p, float x[8])
    {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x);
        x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
        x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z);
        x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
    }
    static __device__ __forceinline__ void store(char* p, const float x[8])
    {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                       pack_bf16x2(x[6], x[7]));
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

// inv_freq / (2 pi) modulo 1, in units of 2^-64 (rounded down): the mantissa
// times 1 / (2 pi) in 128 bits, shifted by the exponent.
__device__ __forceinline__ uint64_t turn_fraction(float f)
{
    // floor(2^128 / (2 pi)), high and low words
    const uint64_t hi = 0x28be60db9391054aull, lo = 0x7f09d5f47d4d3770ull;
    const uint32_t b = __float_as_uint(f);
    const int ex = (int)(b >> 23 & 255);
    const uint64_t m = ex ? (b & 0x7fffff) | 0x800000 : b & 0x7fffff;
    const int e = (ex ? ex : 1) - 150;              // |f| = m 2^e
    // p = m * (hi, lo): 152 bits in (p2, p1, p0)
    const uint64_t p0 = m * lo;
    const uint64_t c0 = __umul64hi(m, lo);
    const uint64_t p1 = m * hi + c0;
    const uint64_t p2 = __umul64hi(m, hi) + (p1 < c0);
    // bits 64 - e and up of p, modulo 2^64
    const int sh = 64 - e;                           // 64 - e >= 0 up to e = 64
    uint64_t r = 0;
    if (sh >= 128) r = sh < 192 ? p2 >> (sh - 128) : 0;
    else if (sh > 64) r = p1 >> (sh - 64) | p2 << (128 - sh);
    else if (sh == 64) r = p1;
    else if (sh > 0) r = p0 >> sh | p1 << (64 - sh);
    else if (sh > -64) r = p0 << -sh;
    return b >> 31 ? 0 - r : r;
}

__device__ __forceinline__ int64_t position_of(const RopeArgs& a, int64_t t)
{
    return a.itype == DPZ_I64 ? static_cast<const int64_t*>(a.positions)[t]
                              : (int64_t) static_cast<const int*>(a.positions)[t];
}

// Sine and cosine of position * frequency.
__device__ __forceinline__ void turn_by(int64_t pos, uint64_t frac, float* s, float* c)
{
    const uint64_t u = (uint64_t)pos * frac;
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
                                           const uint64_t* frac, int64_t t, float sn[NS][V],
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

template <int DT, int V, int NS>
__device__ __forceinline__ void load_slots(const Part<V, NS>& p, const char* row, float x[NS][2][V])
{
    constexpr int ES = DT == DPZ_BF16 ? 2 : 4;
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int v = 0; v < 2; ++v)
            if (p.e[s][v] >= 0) Vec<DT, V>::load(row + (int64_t)p.e[s][v] * ES, x[s][v]);
            else
#pragma unroll
                for (int i = 0; i < V; ++i) x[s][v][i] = 0.0f;
}

template <int DT, int V, int NS>
__device__ __forceinline__ void store_slots(const Part<V, NS>& p, char* row, const float x[NS][2][V])
{
    constexpr int ES = DT == DPZ_BF16 ? 2 : 4;
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int v = 0; v < 2; ++v)
            if (p.e[s][v] >= 0) Vec<DT, V>::store(row + (int64_t)p.e[s][v] * ES, x[s][v]);
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

// Row of head h (queries' heads first, then keys') of token t.
__device__ __forceinline__ char* head_row(const Heads* x, const RopeArgs& a, int64_t t, int h, int es)
{
    const int k = h >= a.H[0];
    const Heads& m = x[k];
    return m.p + (t * m.ld + (int64_t)(h - (k ? a.H[0] : 0)) * m.hs) * es;
}

__device__ __forceinline__ void fill_fractions(const RopeArgs& a, uint64_t* frac)
{
    for (int i = threadIdx.x; i < (a.positions ? a.R / 2 : 0); i += kRopeThreads)
        frac[i] = turn_fraction(a.inv_freq[i]);
    __syncthreads();
}

// An item is a token and kHeadsPerItem of the queries' or of the keys' heads.
struct Items {
    int per[2];     // items of a token among the queries' and the keys' heads
    int64_t n;
};

__device__ __forceinline__ Items items_of(const RopeArgs& a, int64_t tokens)
{
    Items m;
    m.per[0] = (a.H[0] + kHeadsPerItem - 1) / kHeadsPerItem;
    m.per[1] = (a.H[1] + kHeadsPerItem - 1) / kHeadsPerItem;
    m.n = tokens * (m.per[0] + m.per[1]);
    return m;
}

template <int DT, int V, int NS>
__global__ void __launch_bounds__(kRopeThreads) k_rope(RopeArgs a)
{
    pdl_enter();
    constexpr int ES = DT == DPZ_BF16 ? 2 : 4;
    __shared__ uint64_t frac[kRopeMaxD / 2];
    fill_fractions(a, frac);
    const Cut c = make_cut<V>(a.D, a.R, a.interleaved);
    const int lane = threadIdx.x & (c.lanes - 1);
    const Part<V, NS> p = my_part<V, NS>(c, lane, a);
    const Items m = items_of(a, a.T);
    const int64_t item = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) / c.lanes;
    const bool live = item < m.n;     // every lane takes part in the exchanges
    const int each = m.per[0] + m.per[1];
    const int64_t t = live ? item / each : 0;
    const int g = live ? (int)(item % each) : 0, k = g >= m.per[0];
    const int h0 = (k ? g - m.per[0] : g) * kHeadsPerItem + (k ? a.H[0] : 0);
    const int h1 = min(h0 + kHeadsPerItem, k ? a.H[0] + a.H[1] : a.H[0]);
    float sn[NS][V], cs[NS][V], w[NS][2][V];
    slot_turns<V, NS>(p, a, frac, t, sn, cs);
    load_weights<V, NS>(p, a.w[k], a.wdt, w);
    const float inv = 1.0f / (float)a.D;
    constexpr int kAtOnce = NS * V >= 8 ? 2 : 4;
    for (int b = 0; b < kHeadsPerItem; b += kAtOnce) {
        float x[kAtOnce][NS][2][V];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (live && h0 + b + j < h1)
                load_slots<DT, V, NS>(p, head_row(a.in, a, t, h0 + b + j, ES), x[j]);
            else
#pragma unroll
                for (int i = 0; i < NS * 2 * V; ++i) (&x[j][0][0][0])[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const float r = rsqrtf(fmaf(dot<V, NS>(x[j], x[j], c.lanes), inv, a.eps));
#pragma unroll
            for (int s = 0; s < NS; ++s) {
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) (&x[j][s][0][0])[i] *= r * (&w[s][0][0])[i];
                rotate<V>(x[j][s], sn[s], cs[s], a.interleaved, 1.0f);
            }
            if (live && h0 + b + j < h1)
                store_slots<DT, V, NS>(p, head_row(a.out, a, t, h0 + b + j, ES), x[j]);
        }
    }
}

// One block per part of the tokens; each group of lanes walks the part's items
// and keeps the weights' gradients of its slot, which are joined in the
// order of the groups at the end.
template <int DT, int V, int NS>
__global__ void __launch_bounds__(kRopeThreads) k_rope_grad(RopeArgs a)
{
    pdl_enter();
    constexpr int ES = DT == DPZ_BF16 ? 2 : 4;
    __shared__ uint64_t frac[kRopeMaxD / 2];
    __shared__ float joined[kRopeThreads / 32][2][kRopeMaxD];
    fill_fractions(a, frac);
    const Cut c = make_cut<V>(a.D, a.R, a.interleaved);
    const int lane = threadIdx.x & (c.lanes - 1);
    const Part<V, NS> p = my_part<V, NS>(c, lane, a);
    const int64_t per = rope_part_tokens(a.T), t0 = blockIdx.x * per;
    const Items m = items_of(a, min(per, a.T - t0));
    const int each = m.per[0] + m.per[1], groups = kRopeThreads / c.lanes;
    const float inv = 1.0f / (float)a.D;
    float dw[2][NS][2][V] = {};
    // whole warps go round the loop together
    for (int64_t base = 0; base < m.n; base += groups) {
        const int64_t item = base + threadIdx.x / c.lanes;
        const bool live = item < m.n;
        const int64_t t = t0 + (live ? item / each : 0);
        const int g = live ? (int)(item % each) : 0, k = g >= m.per[0];
        const int h0 = (k ? g - m.per[0] : g) * kHeadsPerItem + (k ? a.H[0] : 0);
        const int h1 = min(h0 + kHeadsPerItem, k ? a.H[0] + a.H[1] : a.H[0]);
        float sn[NS][V], cs[NS][V], w[NS][2][V];
        slot_turns<V, NS>(p, a, frac, t, sn, cs);
        load_weights<V, NS>(p, a.w[k], a.wdt, w);
        constexpr int kAtOnce = 2;
        for (int b = 0; b < kHeadsPerItem; b += kAtOnce) {
            float x[kAtOnce][NS][2][V], d[kAtOnce][NS][2][V];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
                if (live && h0 + b + j < h1) {
                    load_slots<DT, V, NS>(p, head_row(a.in, a, t, h0 + b + j, ES), x[j]);
                    load_slots<DT, V, NS>(p, head_row(a.dout, a, t, h0 + b + j, ES), d[j]);
                } else {
#pragma unroll
                    for (int i = 0; i < NS * 2 * V; ++i)
                        (&x[j][0][0][0])[i] = (&d[j][0][0][0])[i] = 0.0f;
                }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const float r = rsqrtf(fmaf(dot<V, NS>(x[j], x[j], c.lanes), inv, a.eps));
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    rotate<V>(d[j][s], sn[s], cs[s], a.interleaved, -1.0f);
#pragma unroll
                    for (int i = 0; i < 2 * V; ++i) {
                        const float n = (&x[j][s][0][0])[i] *= r;
                        float& g1 = (&d[j][s][0][0])[i];
                        float& sum0 = (&dw[0][s][0][0])[i];
                        float& sum1 = (&dw[1][s][0][0])[i];
                        sum0 = fmaf(k ? 0.0f : g1, n, sum0);
                        sum1 = fmaf(k ? g1 : 0.0f, n, sum1);
                        g1 *= (&w[s][0][0])[i];
                    }
                }
                const float mean = dot<V, NS>(x[j], d[j], c.lanes) * inv;
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int i = 0; i < 2 * V; ++i)
                        (&d[j][s][0][0])[i] = r * fmaf(-mean, (&x[j][s][0][0])[i], (&d[j][s][0][0])[i]);
                if (live && h0 + b + j < h1)
                    store_slots<DT, V, NS>(p, head_row(a.out, a, t, h0 + b + j, ES), d[j]);
            }
        }
    }
    if (a.dw[0] == nullptr && a.dw[1] == nullptr) return;
    // the groups of a warp, then the warps, in a fixed order
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float y = dw[k][s][v][i];
                    for (int o = c.lanes; o < 32; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                    if ((threadIdx.x & 31) < c.lanes && p.e[s][v] >= 0)
                        joined[threadIdx.x >> 5][k][p.e[s][v] + i] = y;
                }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.D; i += kRopeThreads) {
        const int k = i >= a.D, d = k ? i - a.D : i;
        float y = 0.0f;
#pragma unroll
        for (int w = 0; w < kRopeThreads / 32; ++w) y += joined[w][k][d];
        a.partial[(int64_t)blockIdx.x * 2 * a.D + i] = y;
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

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s)
{
    set_last_kernel_name("attn_qk_norm_rope");
    return by_vector(a, false, [&](auto dt, auto v, auto ns) {
        const Cut c = make_cut<v>(a.D, a.R, a.interleaved);
        const int64_t each = (a.H[0] + kHeadsPerItem - 1) / kHeadsPerItem +
                             (a.H[1] + kHeadsPerItem - 1) / kHeadsPerItem;
        const int64_t threads = a.T * each * c.lanes;
        const unsigned blocks = (unsigned)((threads + kRopeThreads - 1) / kRopeThreads);
        return launch_kernel(k_rope<dt, v, ns>, dim3(blocks), dim3(kRopeThreads), 0, s, true, 0u, a);
    });
}

cudaError_t launch_rope_grad(const RopeArgs& a, cudaStream_t s)
{
    set_last_kernel_name("attn_qk_norm_rope_grad");
    return by_vector(a, true, [&](auto dt, auto v, auto ns) {
        return launch_kernel(k_rope_grad<dt, v, ns>, dim3((unsigned)rope_parts(a.T)),
                             dim3(kRopeThreads), 0, s, true, 0u, a);
    });
}

cudaError_t launch_rope_dw(const RopeArgs& a, cudaStream_t s)
{
    set_last_kernel_name("attn_qk_norm_rope_dw");
    return launch_kernel(k_rope_dw, dim3((unsigned)((2 * a.D + 31) / 32)), dim3(kDwThreads), 0, s,
                         true, 0u, a);
}

}  // namespace dpz
