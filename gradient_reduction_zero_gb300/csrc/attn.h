// Internal interface between the entry points of attn_api.cpp and the kernels
// of attn_rope.cu, attn_any.cu and attn_tc.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "dpz.h"
#include "internal.h"

namespace dpz {

// Element [t][h][d] at p + (t * ld + h * hs + d) elements.
struct Heads {
    char* p;
    int64_t ld, hs;
};

// ------------------------------------------------------------ norm and rotation

struct RopeArgs {
    Heads in[2], dout[2], out[2];   // queries, keys; dout: of the gradient only
    int64_t T;
    int H[2];                       // heads of queries and of keys
    int D, dt;
    const void* w[2];               // NULL: ones
    int wdt;
    float eps;
    const void* positions;          // NULL: no rotation
    int itype;
    const float* inv_freq;
    int R;                          // elements of a head that rotate, in pairs
    int interleaved;
    void* dw[2];                    // of wdt; NULL: not wanted
    float* partial;                 // [rope_parts(T)][2][D]
};

constexpr int kRopeMaxD = 256;
constexpr int kRopeParts = 304;     // most partial sums of the weights' gradients

// Tokens of one partial sum of the weights' gradients, and how many there are.
DPZ_HD inline int64_t rope_part_tokens(int64_t T)
{
    const int64_t n = (T + kRopeParts - 1) / kRopeParts;
    return n < 2 ? 2 : n;
}
DPZ_HD inline int64_t rope_parts(int64_t T)
{
    return (T + rope_part_tokens(T) - 1) / rope_part_tokens(T);
}

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s);
cudaError_t launch_rope_grad(const RopeArgs& a, cudaStream_t s);
cudaError_t launch_rope_dw(const RopeArgs& a, cudaStream_t s);

// ------------------------------------------------------------ attention

struct AttnArgs {
    Heads q, k, v, out;         // out: written by the forward pass, read by the gradient
    Heads dout, dq, dk, dv;     // of the gradient only
    float* lse;                 // [Hq][Tq]; NULL: not wanted (forward)
    float* delta;               // [Hq][Tq], workspace of the gradient
    int64_t Tq, Tk;
    int Hq, Hk, D, dt;
    int64_t B;
    const void *cu_q, *cu_k;    // NULL: B sequences of equal length,
    int len_q, len_k;           // these
    int itype;
    int causal;
    float scale;
};

constexpr int kAttnMaxD = 128;

cudaError_t launch_attn_any(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_attn_any_dq(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_attn_any_dkv(const AttnArgs& a, cudaStream_t s);

// The same on the tensor cores, for the calls that attn_tc_takes says.
bool attn_tc_takes(const AttnArgs& a, bool grad);
cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_attn_tc_dq(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_attn_tc_dkv(const AttnArgs& a, cudaStream_t s);

#if defined(__CUDACC__)
// Where a block's tile of rows lies: rows [row0, row0 + rows) of the sequence
// that has queries [q0, q0 + nq) and keys [k0, k0 + nk).
struct Tile {
    int64_t q0, k0;
    int nq, nk;
    int row0;        // first row of the tile within its sequence
    bool any;        // false: no such tile
};

__device__ __forceinline__ int64_t cu_at(const void* cu, int itype, int64_t i, int64_t T)
{
    const int64_t v = itype == DPZ_I64 ? static_cast<const int64_t*>(cu)[i]
                                       : (int64_t) static_cast<const int*>(cu)[i];
    return v < 0 ? 0 : v > T ? T : v;
}

// The bounds of sequence b: first row and length among T rows; `len` each without offsets.
__device__ __forceinline__ void seq_bounds(const void* cu, int itype, int64_t b, int len, int64_t T,
                                           int64_t* first, int* n)
{
    if (cu == nullptr) {
        *first = b * len;
        *n = len;
        return;
    }
    const int64_t a = cu_at(cu, itype, b, T), e = cu_at(cu, itype, b + 1, T);
    *first = a;
    *n = (int)(e > a ? e - a : 0);
}

constexpr int kSortedSeqs = 32;

// Tile number `tile` of all sequences' tiles of `per` rows, over the queries
// (of_keys false) or the keys: by position in sequences of equal length and in up to
// kSortedSeqs packed ones, else by sequence.  Called by whole warps with equal arguments: with offsets, 32
// sequences' numbers of tiles are summed at a time.  The number of tiles is at
// most tiles_bound(), below 2^31.
__device__ __forceinline__ Tile find_tile(const AttnArgs& a, int tile, int per, bool of_keys)
{
    const void* cu = of_keys ? a.cu_k : a.cu_q;
    const int64_t T = of_keys ? a.Tk : a.Tq;
    const int len = of_keys ? a.len_k : a.len_q;
    Tile t{};
    int b = -1;
    if (cu == nullptr) {
        // the same tile of every sequence, then the next: equal amounts of work side by side
        const unsigned n = (unsigned)a.B, at = (unsigned)tile / n;
        if ((int64_t)at * per < len) {
            b = (int)((unsigned)tile - at * n);
            t.row0 = (int)at * per;
        }
    } else if (a.B <= kSortedSeqs) {
        // a sequence to a lane; the tiles at one position of all that reach it, then the next
        // position's, in steps over which the same sequences reach it
        const int lane = threadIdx.x & 31;
        int64_t first;
        int n = 0, at = 0, left = tile;
        if (lane < a.B) seq_bounds(cu, a.itype, lane, 0, T, &first, &n);
        const int mine = (int)((unsigned)(n + per - 1) / (unsigned)per);
        while (true) {
            const unsigned reach = __ballot_sync(0xffffffffu, mine > at);
            if (reach == 0) break;
            const int many = __popc(reach);
            const int until = __reduce_min_sync(0xffffffffu, mine > at ? mine : 0x7fffffff);
            if (left < (until - at) * many) {
                b = (int)__fns(reach, 0, left % many + 1);
                t.row0 = (at + left / many) * per;
                break;
            }
            left -= (until - at) * many;
            at = until;
        }
    } else {
        const int lane = threadIdx.x & 31;
        int left = tile;
        for (int64_t base = 0; base < a.B; base += 32) {
            int64_t first;
            int n = 0;
            if (base + lane < a.B) seq_bounds(cu, a.itype, base + lane, 0, T, &first, &n);
            const int mine = (int)((unsigned)(n + per - 1) / (unsigned)per);
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            const unsigned past = __ballot_sync(0xffffffffu, upto > left);
            if (past != 0) {
                const int l = __ffs((int)past) - 1;
                b = (int)base + l;
                t.row0 = (left - __shfl_sync(0xffffffffu, upto - mine, l)) * per;
                break;
            }
            left -= __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    t.any = b >= 0;
    if (t.any) {
        seq_bounds(a.cu_q, a.itype, b, a.len_q, a.Tq, &t.q0, &t.nq);
        seq_bounds(a.cu_k, a.itype, b, a.len_k, a.Tk, &t.k0, &t.nk);
    }
    return t;
}
#endif

// Most tiles of `per` rows that B sequences of T rows in all have.
inline int64_t tiles_bound(const void* cu, int64_t T, int64_t B, int per)
{
    if (cu == nullptr) return B * ((T / B + per - 1) / per);
    const int64_t nonempty = B < T ? B : T;
    return T / per + nonempty;
}

}  // namespace dpz
