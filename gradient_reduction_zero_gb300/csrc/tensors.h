// Internal interface between the entry points of tensors_api.cpp and the
// kernels of tensors.cu: lists of tensors.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "dpz.h"
#include "internal.h"

namespace dpz {

constexpr int kListChunk = 65536;   // bytes of a block's part of a tensor
constexpr int kListMost = 1024;     // tensors of one launch: their addresses are its parameters
constexpr int kListSmall = 64;      // smaller blocks of parameters for shorter lists
constexpr int kListMid = 256;

// Blocks of one tensor.
inline int64_t list_chunks(const dpz_tensor& t)
{
    const int64_t per = kListChunk / (t.dtype == DPZ_BF16 ? 2 : 4);
    return (t.n + per - 1) / per;
}

// n <= kListMost tensors, at least one of them not empty.
cudaError_t launch_tensors_sumsq(const dpz_tensor* in, int n, double* partial, cudaStream_t s);
cudaError_t launch_tensors_norm(const double* partial, int64_t n, float* norm_out, cudaStream_t s);
cudaError_t launch_tensors_clip(const dpz_tensor* in, const dpz_tensor* out, int n,
                                const float* norm, float clip, cudaStream_t s);

}  // namespace dpz
