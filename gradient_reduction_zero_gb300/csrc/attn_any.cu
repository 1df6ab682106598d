// Attention and its gradient in fp32 arithmetic, for either type, any stride
// and any head up to 128 elements: fp32 tensors, and bf16 ones that the
// tensor-core kernels of attn_tc.cu do not take.
//
//   s_ij = scale q_i . k_j,  p_ij = exp(s_ij - lse_i),  out_i = sum_j p_ij v_j
//   delta_i = dout_i . out_i,  ds_ij = p_ij (dout_i . v_j - delta_i)
//   dv_j = sum_i p_ij dout_i,  dk_j = scale sum_i ds_ij q_i,  dq_i = scale sum_j ds_ij k_j
//
// 256 threads on tiles of 64 queries by 64 keys.  Thread (ty, tx) owns rows
// 4 ty .. 4 ty + 3 of a product and its columns tx, tx + 16, ... (of scores) or
// 4 tx + 64 c .. (of outputs); operands lie row by row in shared memory with a
// padding of four floats, so that each 16-byte read of 16 different rows
// covers all banks.  Bound by the FMA units: 64 products per 8 reads.
// The queries' gradient and the keys' and values' are separate kernels that
// each recompute the scores: every sum then has one owner and a fixed order.
// Measured in fp32: 2 x 509 tokens of 12 heads of 64, 70 us (23 TFLOP/s); the gradient of
// 3 x 255, 95 us.  With element-wise loads one after another 77 and 129.
#include <cmath>
#include <type_traits>

#include "attn.h"
#include "bulk.cuh"
#include "device.cuh"

namespace dpz {

namespace {

constexpr int kAnyThreads = 256;
constexpr int kAnyTile = 64;
constexpr int kAnyPs = kAnyTile + 4;    // row stride of the probabilities' tile

template <int DT>
__device__ __forceinline__ float elem(const char* p)
{
    return DT == DPZ_BF16 ? __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t*>(p) << 16)
                          : *reinterpret_cast<const float*>(p);
}

template <int DT>
__device__ __forceinline__ void put(char* p, float x)
{
    if (DT == DPZ_BF16) *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(x);
    else *reinterpret_cast<float*>(p) = x;
}

// Whether groups of four elements of every row lie on boundaries of their size.
template <int DT>
__device__ __forceinline__ bool quads(const Heads& x, int D)
{
    constexpr int ES = DT == DPZ_BF16 ? 2 : 4;
    return ((reinterpret_cast<uintptr_t>(x.p) / ES | (uintptr_t)x.ld | (uintptr_t)x.hs | (uintptr_t)D) & 3) == 0 &&
           reinterpret_cast<uintptr_t>(x.p) % ES == 0;
}

// A thread's part of a tile: 64 rows of DP floats, rows [row, row + 64) of head h among rows
// [first, first + n) of x, zeros beyond n and beyond D.  All of its loads are under way
// before the first is used.
template <int DT, int DP>
struct TileLoad {
    static constexpr int kQuads = kAnyTile * DP / 4 / kAnyThreads;
    float4 v[kQuads];

    __device__ __forceinline__ void load(const Heads& x, int64_t first, int row, int n, int h, int D)
    {
        constexpr int ES = DT == DPZ_BF16 ? 2 : 4;
        const char* base = x.p + ((first + row) * x.ld + (int64_t)h * x.hs) * ES;
        const int rows = min(kAnyTile, n - row);
        const bool whole = quads<DT>(x, D);
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
            const int i = threadIdx.x + k * kAnyThreads, r = i / (DP / 4), d = i % (DP / 4) * 4;
            v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (r >= rows || d >= D) continue;
            const char* p = base + ((int64_t)r * x.ld + d) * ES;
            if (whole) {
                if constexpr (DT == DPZ_BF16) {
                    const uint2 w = *reinterpret_cast<const uint2*>(p);
                    v[k] = make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
                } else {
                    v[k] = *reinterpret_cast<const float4*>(p);
                }
            } else {
                v[k].x = elem<DT>(p);
                if (d + 1 < D) v[k].y = elem<DT>(p + ES);
                if (d + 2 < D) v[k].z = elem<DT>(p + 2 * ES);
                if (d + 3 < D) v[k].w = elem<DT>(p + 3 * ES);
            }
        }
    }
    // rows DP + 4 floats apart
    __device__ __forceinline__ void store(float* s) const
    {
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
            const int i = threadIdx.x + k * kAnyThreads, r = i / (DP / 4), d = i % (DP / 4) * 4;
            *reinterpret_cast<float4*>(s + r * (DP + 4) + d) = v[k];
        }
    }
};

template <int DT, int DP>
__device__ __forceinline__ void load_tile(float* s, const Heads& x, int64_t first, int row, int n,
                                          int h, int D)
{
    TileLoad<DT, DP> t;
    t.load(x, first, row, n, h, D);
    t.store(s);
}

// Two tiles at once.
template <int DT, int DP>
__device__ __forceinline__ void load_tiles(float* s0, const Heads& x0, float* s1, const Heads& x1,
                                           int64_t first, int row, int n, int h, int D)
{
    TileLoad<DT, DP> t, u;
    t.load(x0, first, row, n, h, D);
    u.load(x1, first, row, n, h, D);
    t.store(s0);
    u.store(s1);
}

// acc[i][j] = a[row 4 ty + i] . b[row tx + 16 j]
template <int DP>
__device__ __forceinline__ void dot_tile(const float* a, const float* b, float acc[4][4])
{
    constexpr int DS = DP + 4;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(a + (4 * ty + i) * DS + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * DS + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = fmaf(x[i].w, y[j].w, fmaf(x[i].z, y[j].z,
                            fmaf(x[i].y, y[j].y, fmaf(x[i].x, y[j].x, acc[i][j]))));
    }
}

// acc[i][c][.] += sum over r of p[4 ty + i][r] * b[r][4 tx + 64 c + .]
template <int DP>
__device__ __forceinline__ void add_rows(const float* p, const float* b, float acc[4][DP / 64][4])
{
    constexpr int DS = DP + 4;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 2
    for (int r = 0; r < kAnyTile; r += 4) {
        float x[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(p + (4 * ty + i) * kAnyPs + r);
            x[i][0] = v.x; x[i][1] = v.y; x[i][2] = v.z; x[i][3] = v.w;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int c = 0; c < DP / 64; ++c) {
                const float4 y =
                    *reinterpret_cast<const float4*>(b + (r + k) * DS + 4 * tx + 64 * c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[i][c][0] = fmaf(x[i][k], y.x, acc[i][c][0]);
                    acc[i][c][1] = fmaf(x[i][k], y.y, acc[i][c][1]);
                    acc[i][c][2] = fmaf(x[i][k], y.z, acc[i][c][2]);
                    acc[i][c][3] = fmaf(x[i][k], y.w, acc[i][c][3]);
                }
            }
    }
}

// acc[j][c][.] += sum over r of p[r][4 ty + j] * b[r][4 tx + 64 c + .]
template <int DP>
__device__ __forceinline__ void add_rows_t(const float* p, const float* b, float acc[4][DP / 64][4])
{
    constexpr int DS = DP + 4;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 4
    for (int r = 0; r < kAnyTile; ++r) {
        const float4 x = *reinterpret_cast<const float4*>(p + r * kAnyPs + 4 * ty);
#pragma unroll
        for (int c = 0; c < DP / 64; ++c) {
            const float4 y = *reinterpret_cast<const float4*>(b + r * DS + 4 * tx + 64 * c);
            const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[j][c][0] = fmaf(xs[j], y.x, acc[j][c][0]);
                acc[j][c][1] = fmaf(xs[j], y.y, acc[j][c][1]);
                acc[j][c][2] = fmaf(xs[j], y.z, acc[j][c][2]);
                acc[j][c][3] = fmaf(xs[j], y.w, acc[j][c][3]);
            }
        }
    }
}

// Rows 4 ty + i of a tile of n rows of head h, times k[i], to x.
template <int DT, int DP>
__device__ __forceinline__ void store_rows(const Heads& x, int64_t first, int row, int n, int h,
                                           int D, const float acc[4][DP / 64][4], const float k[4])
{
    constexpr int ES = DT == DPZ_BF16 ? 2 : 4;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (row + 4 * ty + i >= n) continue;
        char* p = x.p + ((first + row + 4 * ty + i) * x.ld + (int64_t)h * x.hs) * ES;
#pragma unroll
        for (int c = 0; c < DP / 64; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = 4 * tx + 64 * c + e;
                if (d < D) put<DT>(p + (int64_t)d * ES, acc[i][c][e] * k[i]);
            }
    }
}

// Maximum and sum over the 16 threads that share a row.
__device__ __forceinline__ float row_max(float x)
{
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The keys [0, end) that a tile of queries sees: all of them, or those up to its
// last row's.
__device__ __forceinline__ int keys_end(const AttnArgs& a, const Tile& t, int rows)
{
    if (!a.causal) return t.nk;
    const int last = min(t.row0 + rows, t.nq) - 1;
    return max(0, min(t.nk, last + t.nk - t.nq + 1));
}

template <int DT, int DP>
__global__ void __launch_bounds__(kAnyThreads) k_attn_any(AttnArgs a)
{
    pdl_enter();
    extern __shared__ float4 smem4[];
    constexpr int kRows = kAnyTile * (DP + 4);
    float* q = reinterpret_cast<float*>(smem4);
    float *k = q + kRows, *v = k + kRows, *p = v + kRows;
    // the tiles at the end of a sequence see the most keys and go first
    const Tile t = find_tile(a, (int)(gridDim.x - 1 - blockIdx.x), kAnyTile, false);
    if (!t.any) return;
    const int h = blockIdx.y, hk = h / (a.Hq / a.Hk);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    load_tile<DT, DP>(q, a.q, t.q0, t.row0, t.nq, h, a.D);
    float acc[4][DP / 64][4] = {}, m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.0f;
    }
    const int end = keys_end(a, t, kAnyTile);
    for (int j0 = 0; j0 < end; j0 += kAnyTile) {
        __syncthreads();
        load_tiles<DT, DP>(k, a.k, v, a.v, t.k0, j0, t.nk, hk, a.D);
        __syncthreads();
        float s[4][4];
        dot_tile<DP>(q, k, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int seen = a.causal ? t.row0 + 4 * ty + i + t.nk - t.nq + 1 : t.nk;
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = j0 + tx + 16 * j;
                s[i][j] = key < t.nk && key < seen ? s[i][j] * a.scale : -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
            const float next = fmaxf(m[i], row_max(top));
            const float ref = next == -INFINITY ? 0.0f : next;
            const float fade = expf(m[i] - ref);
            m[i] = next;
            l[i] *= fade;
#pragma unroll
            for (int c = 0; c < DP / 64; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][c][e] *= fade;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w = expf(s[i][j] - ref);
                l[i] += w;
                p[(4 * ty + i) * kAnyPs + tx + 16 * j] = w;
            }
        }
        __syncthreads();
        add_rows<DP>(p, v, acc);
    }
    float inv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float sum = row_sum(l[i]);
        inv[i] = sum == 0.0f ? 0.0f : 1.0f / sum;
        if (a.lse != nullptr && tx == 0 && t.row0 + 4 * ty + i < t.nq)
            a.lse[(int64_t)h * a.Tq + t.q0 + t.row0 + 4 * ty + i] =
                sum == 0.0f ? -INFINITY : m[i] + logf(sum);
    }
    store_rows<DT, DP>(a.out, t.q0, t.row0, t.nq, h, a.D, acc, inv);
}

// The probabilities and the scores' gradient of a tile, from lse and delta.
template <int DP>
__device__ __forceinline__ void score_grad(const AttnArgs& a, const Tile& t, int i0, int j0,
                                           const float* q, const float* k, const float* dout,
                                           const float* v, const float lse[4],
                                           const float delta[4], float s[4][4], float ds[4][4])
{
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    dot_tile<DP>(q, k, s);
    dot_tile<DP>(dout, v, ds);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = i0 + 4 * ty + i;
        const int seen = row >= t.nq || lse[i] == -INFINITY ? 0
                         : a.causal ? row + t.nk - t.nq + 1 : t.nk;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int key = j0 + tx + 16 * j;
            const bool on = key < t.nk && key < seen;
            s[i][j] = on ? expf(fmaf(s[i][j], a.scale, -lse[i])) : 0.0f;
            ds[i][j] = on ? s[i][j] * (ds[i][j] - delta[i]) : 0.0f;
        }
    }
}

template <int DT, int DP>
__global__ void __launch_bounds__(kAnyThreads) k_attn_any_dq(AttnArgs a)
{
    pdl_enter();
    extern __shared__ float4 smem4[];
    constexpr int kRows = kAnyTile * (DP + 4), DS = DP + 4;
    float* q = reinterpret_cast<float*>(smem4);
    float *dout = q + kRows, *k = dout + kRows, *v = k + kRows, *p = v + kRows;
    const Tile t = find_tile(a, (int)(gridDim.x - 1 - blockIdx.x), kAnyTile, false);
    if (!t.any) return;
    const int h = blockIdx.y, hk = h / (a.Hq / a.Hk);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    load_tiles<DT, DP>(q, a.q, dout, a.dout, t.q0, t.row0, t.nq, h, a.D);
    load_tile<DT, DP>(k, a.out, t.q0, t.row0, t.nq, h, a.D);
    __syncthreads();
    float lse[4], delta[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float y = 0.0f;
        for (int d = tx; d < DP; d += 16) y = fmaf(dout[(4 * ty + i) * DS + d], k[(4 * ty + i) * DS + d], y);
        delta[i] = row_sum(y);
        const int row = t.row0 + 4 * ty + i;
        const int64_t at = (int64_t)h * a.Tq + t.q0 + row;
        lse[i] = row < t.nq ? a.lse[at] : -INFINITY;
        if (tx == 0 && row < t.nq) a.delta[at] = delta[i];
    }
    float acc[4][DP / 64][4] = {};
    const int end = keys_end(a, t, kAnyTile);
    for (int j0 = 0; j0 < end; j0 += kAnyTile) {
        __syncthreads();
        load_tiles<DT, DP>(k, a.k, v, a.v, t.k0, j0, t.nk, hk, a.D);
        __syncthreads();
        float s[4][4], ds[4][4];
        score_grad<DP>(a, t, t.row0, j0, q, k, dout, v, lse, delta, s, ds);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) p[(4 * ty + i) * kAnyPs + tx + 16 * j] = ds[i][j];
        __syncthreads();
        add_rows<DP>(p, k, acc);
    }
    const float scale[4] = {a.scale, a.scale, a.scale, a.scale};
    store_rows<DT, DP>(a.dq, t.q0, t.row0, t.nq, h, a.D, acc, scale);
}

template <int DT, int DP>
__global__ void __launch_bounds__(kAnyThreads) k_attn_any_dkv(AttnArgs a)
{
    pdl_enter();
    extern __shared__ float4 smem4[];
    constexpr int kRows = kAnyTile * (DP + 4);
    float* k = reinterpret_cast<float*>(smem4);
    float *v = k + kRows, *q = v + kRows, *dout = q + kRows, *p = dout + kRows,
          *ds = p + kAnyTile * kAnyPs;
    // the first keys of a sequence are seen by the most queries: tiles in order
    const Tile t = find_tile(a, (int)blockIdx.x, kAnyTile, true);
    if (!t.any) return;
    const int hk = blockIdx.y, G = a.Hq / a.Hk;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    load_tiles<DT, DP>(k, a.k, v, a.v, t.k0, t.row0, t.nk, hk, a.D);
    float dk[4][DP / 64][4] = {}, dv[4][DP / 64][4] = {};
    // the first query that sees this tile's first key
    const int first = a.causal ? max(0, t.row0 - (t.nk - t.nq)) / kAnyTile * kAnyTile : 0;
    for (int h = hk * G; h < (hk + 1) * G; ++h)
        for (int i0 = first; i0 < t.nq; i0 += kAnyTile) {
            __syncthreads();
            load_tiles<DT, DP>(q, a.q, dout, a.dout, t.q0, i0, t.nq, h, a.D);
            float lse[4], delta[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = i0 + 4 * ty + i;
                const int64_t at = (int64_t)h * a.Tq + t.q0 + row;
                lse[i] = row < t.nq ? a.lse[at] : -INFINITY;
                delta[i] = row < t.nq ? a.delta[at] : 0.0f;
            }
            __syncthreads();
            float s[4][4], g[4][4];
            score_grad<DP>(a, t, i0, t.row0, q, k, dout, v, lse, delta, s, g);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    p[(4 * ty + i) * kAnyPs + tx + 16 * j] = s[i][j];
                    ds[(4 * ty + i) * kAnyPs + tx + 16 * j] = g[i][j];
                }
            __syncthreads();
            add_rows_t<DP>(p, dout, dv);
            add_rows_t<DP>(ds, q, dk);
        }
    const float one[4] = {1.0f, 1.0f, 1.0f, 1.0f};
    const float scale[4] = {a.scale, a.scale, a.scale, a.scale};
    store_rows<DT, DP>(a.dv, t.k0, t.row0, t.nk, hk, a.D, dv, one);
    store_rows<DT, DP>(a.dk, t.k0, t.row0, t.nk, hk, a.D, dk, scale);
}

// Calls f with the type and the padded width as constants.
template <class F>
cudaError_t by_type(const AttnArgs& a, F&& f)
{
    using std::integral_constant;
    const bool wide = a.D > 64;
    if (a.dt == DPZ_BF16)
        return wide ? f(integral_constant<int, DPZ_BF16>{}, integral_constant<int, 128>{})
                    : f(integral_constant<int, DPZ_BF16>{}, integral_constant<int, 64>{});
    return wide ? f(integral_constant<int, DPZ_F32>{}, integral_constant<int, 128>{})
                : f(integral_constant<int, DPZ_F32>{}, integral_constant<int, 64>{});
}

// Launch with `tiles` tiles of operands and `squares` of probabilities.
template <int DP>
cudaError_t launch_tiles(void (*fn)(AttnArgs), SmemRaisedOn& raised, int tiles, int squares,
                         int64_t blocks, int heads, const AttnArgs& a, cudaStream_t s)
{
    const size_t smem = sizeof(float) * (size_t)(tiles * kAnyTile * (DP + 4) + squares * kAnyTile * kAnyPs);
    const cudaError_t e = raise_smem(raised, reinterpret_cast<const void*>(fn), smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(fn, dim3((unsigned)blocks, (unsigned)heads), dim3(kAnyThreads), smem, s,
                         true, 0u, a);
}

}  // namespace

cudaError_t launch_attn_any(const AttnArgs& a, cudaStream_t s)
{
    set_last_kernel_name("attn_forward");
    return by_type(a, [&](auto dt, auto dp) {
        static SmemRaisedOn raised;
        return launch_tiles<dp>(k_attn_any<dt, dp>, raised, 3, 1,
                                tiles_bound(a.cu_q, a.Tq, a.B, kAnyTile), a.Hq, a, s);
    });
}

cudaError_t launch_attn_any_dq(const AttnArgs& a, cudaStream_t s)
{
    set_last_kernel_name("attn_grad_dq");
    return by_type(a, [&](auto dt, auto dp) {
        static SmemRaisedOn raised;
        return launch_tiles<dp>(k_attn_any_dq<dt, dp>, raised, 4, 1,
                                tiles_bound(a.cu_q, a.Tq, a.B, kAnyTile), a.Hq, a, s);
    });
}

cudaError_t launch_attn_any_dkv(const AttnArgs& a, cudaStream_t s)
{
    set_last_kernel_name("attn_grad_dkv");
    return by_type(a, [&](auto dt, auto dp) {
        static SmemRaisedOn raised;
        return launch_tiles<dp>(k_attn_any_dkv<dt, dp>, raised, 4, 2,
                                tiles_bound(a.cu_k, a.Tk, a.B, kAnyTile), a.Hk, a, s);
    });
}

}  // namespace dpz
