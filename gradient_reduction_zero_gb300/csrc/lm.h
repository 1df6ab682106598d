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

cudaError_t launch_embedding(const Mat& table, const Ids& ids, int64_t T, int64_t V, int64_t D,
                             float scale, const Mat& out, cudaStream_t s);

// ------------------------------------------------------------ embedding gradient
//
// Workspace: a header, start and count of every token's run in the sorted
// order, the sorted order itself (token positions), and two fp32 partial rows
// per piece of kEmbPiece sorted positions.
constexpr int kEmbPiece = 32;   // longest run that one pass sums

struct EmbWs {
    int* nvalid;      // sorted positions in all (tokens whose id names a token)
    int* start;       // [V] first sorted position of token v
    int* count;       // [V] how often it occurs
    int* order;       // [T] token positions by (owner, id, position)
    float* partial;   // [pieces][2][Dpad] sums of pieces of long runs
    int64_t Dpad;     // row stride of partial
    int64_t pieces;
};

inline int64_t emb_pieces(int64_t T) { return (T + kEmbPiece - 1) / kEmbPiece; }

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
    const size_t o_head = take(256), o_start = take(4 * size_t(V)), o_count = take(4 * size_t(V)),
                 o_order = take(4 * size_t(T));
    const int64_t Dpad = (D + 7) / 8 * 8, pieces = emb_pieces(T);
    const size_t o_partial = take(8 * size_t(Dpad) * size_t(pieces));
    if (w && b)
        *w = EmbWs{reinterpret_cast<int*>(b + o_head),    reinterpret_cast<int*>(b + o_start),
                   reinterpret_cast<int*>(b + o_count),   reinterpret_cast<int*>(b + o_order),
                   reinterpret_cast<float*>(b + o_partial), Dpad, pieces};
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
