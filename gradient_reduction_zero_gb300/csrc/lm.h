// Internal interface between the entry points of lm_api.cpp and the kernels
// of lm_embed.cu, lm_logprobs.cu and lm_distill.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "dpz.h"
#include "internal.h"

namespace dpz {

// A row-major matrix of element type dt (DPZ_F32 or DPZ_BF16) whose rows are
// ld elements apart.
struct Mat {
    char* p;
    int64_t ld;
    int dt;
};

// Token ids of type it (DPZ_I32 or DPZ_I64).
struct Ids {
    const void* p;
    int it;
};

#if defined(__CUDACC__)
// An id as an int, -1 where it names none of V tokens (V < 2^30).
__device__ __forceinline__ int load_token(const Ids& ids, int64_t i, int64_t V)
{
    const int64_t v = ids.it == DPZ_I64 ? static_cast<const int64_t*>(ids.p)[i]
                                        : (int64_t) static_cast<const int*>(ids.p)[i];
    return v >= 0 && v < V ? (int)v : -1;
}
#endif

cudaError_t launch_embedding(const Mat& table, const Ids& ids, int64_t T, int64_t V, int64_t D,
                             float scale, const Mat& out, cudaStream_t s);

// ------------------------------------------------------------ embedding gradient
//
// Workspace: start and length of every token's run in the sorted order, the
// sorted order itself (token positions), the long runs (more than emb_piece(T)
// terms) by owner, and one fp32 partial row for each of their pieces.  Every
// word that a call reads it has written itself.
constexpr int kEmbMaxPiece = 64;
constexpr int kEmbLogBins = 10;   // a sorting block owns at most 2^10 ids

struct EmbWs {
    int4* owner;      // [owners] pieces, long runs and short runs of each owner
    int2* run;        // [V] first sorted position of token v, how often it occurs
    int* order;       // [T] token positions by (owner, id, position)
    int4* longs;      // [owners][2^kEmbLogBins] token, first position, length,
                      // pieces of the owner's long runs before it
    int4* shorts;     // [owners][2^kEmbLogBins] token, first position, length of the
                      // others, if the call adds in place
    float* partial;   // [pieces][Dpad] sums of pieces, by owner and run
    int64_t Dpad;     // row stride of partial
    int64_t pieces;   // most pieces there can be
    int piece;        // terms of a piece
};

// Owners of the ids: 128, one wave of sorting blocks, until a block would own
// more than 2^kEmbLogBins ids.
inline int emb_log_owners(int64_t V)
{
    int log_owners = 7;
    while ((V >> log_owners) >= (1 << kEmbLogBins)) ++log_owners;
    return log_owners;
}

// The longest run that one pass sums.  Short pieces are quick to sum and many
// to join, so few tokens take 32 and many 64: 8,192 tokens of D = 768 in bf16
// 25.4 us with 32 and 30.3 with 64, 32,768 tokens 39 and 45, 65,536 tokens of
// D = 1,600 110 and 104.
inline int emb_piece(int64_t T) { return T <= 49152 ? 32 : kEmbMaxPiece; }

// A run of n > piece terms has ceil(n / piece) < n / piece + 1 pieces.
inline int64_t emb_pieces(int64_t T)
{
    const int64_t runs = T / (emb_piece(T) + 1);
    return runs > 0 ? T / emb_piece(T) + runs : 0;
}

// Lays the workspace out from `p` (which may be NULL) and returns its bytes.
inline size_t emb_ws_layout(void* p, int64_t T, int64_t V, int64_t D, EmbWs* w)
{
    char* b = static_cast<char*>(p);
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    const size_t owners = size_t(1) << emb_log_owners(V);
    const int64_t Dpad = (D + 7) / 8 * 8, pieces = emb_pieces(T);
    const size_t o_owner = take(16 * owners), o_run = take(8 * size_t(V)), o_order = take(4 * size_t(T)),
                 o_longs = take(16 * (owners << kEmbLogBins)),
                 o_shorts = take(16 * (owners << kEmbLogBins)),
                 o_partial = take(4 * size_t(Dpad) * size_t(pieces));
    if (w && b)
        *w = EmbWs{reinterpret_cast<int4*>(b + o_owner), reinterpret_cast<int2*>(b + o_run),
                   reinterpret_cast<int*>(b + o_order),  reinterpret_cast<int4*>(b + o_longs),
                   reinterpret_cast<int4*>(b + o_shorts), reinterpret_cast<float*>(b + o_partial),
                   Dpad, pieces, emb_piece(T)};
    return at;
}

struct EmbGrad {
    Mat dout, base, dtable;   // base.p NULL: zeros
    Ids ids;
    int64_t T, V, D;
    float scale;
    EmbWs ws;
};
cudaError_t launch_emb_sort(const EmbGrad& g, cudaStream_t s);
cudaError_t launch_emb_rows(const EmbGrad& g, cudaStream_t s);
cudaError_t launch_emb_join(const EmbGrad& g, cudaStream_t s);

// ------------------------------------------------------------ rows of logits

struct LogprobArgs {
    Mat x;
    int64_t T;
    int V;
    float scale;
    Ids targets;       // p NULL: no logprob
    float *logprob, *lse, *entropy;
    int K;
    void* top_ids;     // of targets.it
    float* top_logprobs;
};
cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t s);

struct LogprobGradArgs {
    Mat x, dx;
    int64_t T;
    int V;
    float scale;
    Ids targets;
    const float *lse, *entropy, *dlogprob, *dentropy;
};
cudaError_t launch_logprobs_grad(const LogprobGradArgs& a, cudaStream_t s);

struct DistillArgs {
    Mat x, dx;          // dx.p NULL: no gradient
    int64_t T;
    int V;
    float inv_tau;
    Ids ids;
    Mat teacher;
    int K;
    const float* dloss;
    float* loss;        // NULL: gradient only, from lse_in
    float* lse;
    const float* lse_in;
};
cudaError_t launch_distill(const DistillArgs& a, cudaStream_t s);

}  // namespace dpz
