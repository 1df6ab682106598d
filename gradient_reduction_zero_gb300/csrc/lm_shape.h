// Launch shapes of the kernels over rows of logits (lm_logprobs.cu and
// lm_distill.cu), on the host: threads per row, blocks per row, and figures of
// the current device that are asked for once.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "dpz.h"

namespace dpz {

// Positive figures of a device, by key, each asked for once (every time on
// devices beyond kDevices).
template <int KEYS>
struct PerDevice {
    static constexpr int kDevices = 64;
    std::atomic<int> got[kDevices][KEYS];

    // ask(device, &value) finds the current device's.
    template <class F>
    cudaError_t get(int key, int* value, F&& ask)
    {
        int d = 0;
        cudaError_t e = cudaGetDevice(&d);
        if (e != cudaSuccess) return e;
        const bool cached = d >= 0 && d < kDevices;
        *value = cached ? got[d][key].load(std::memory_order_relaxed) : 0;
        if (*value != 0) return cudaSuccess;
        e = ask(d, value);
        if (e == cudaSuccess && cached) got[d][key].store(*value, std::memory_order_relaxed);
        return e;
    }
};

// SMs of the current device.
inline cudaError_t sm_count(int* sms)
{
    static PerDevice<1> known;
    return known.get(0, sms, [](int d, int* n) {
        return cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, d);
    });
}

constexpr int kMaxCluster = 8;

// Threads per block for rows up to kShortRow bytes, up to kMidRow, and for
// longer ones or up to two rows per SM.  8,192 rows of bf16, in us:
//
//   logits                8,000 (16 KB)   16,000     24,000 (48 KB)
//   threads               64  128  256   128  256     128  256
//   log probabilities     27   30   40    47   55      66   70
//   eight alternatives    44   49   61    68   77      88   91
//   their gradient        39   37   42    71   71     107  104
//   distillation loss     28   30   43    48   57      66   72
//   its gradient          44   44   59    80   82     120  120
//
// Rows that all fit on the GPU at once want many threads each (152 SMs): 300 rows
// of 8,000 with eight alternatives take 7.4 us with 64 threads and 5.1 with 256, their
// gradient 4.2 and 2.5; at 450 rows of 2,000, 5.5 and 4.6, but 2.4 and 2.9.
constexpr int kRowThreads = 256, kMidThreads = 128, kShortThreads = 64;
constexpr int64_t kShortRow = 16384, kMidRow = 49152;

// Calls f with the threads for T rows of this length, as a constant.
template <class F>
cudaError_t by_row_threads(int64_t T, int64_t bytes, int sms, F&& f)
{
    if (T <= 2 * (int64_t)sms) return f(std::integral_constant<int, kRowThreads>{});
    if (bytes <= kShortRow) return f(std::integral_constant<int, kShortThreads>{});
    if (bytes <= kMidRow) return f(std::integral_constant<int, kMidThreads>{});
    return f(std::integral_constant<int, kRowThreads>{});
}

inline int64_t row_bytes(int64_t V, int dt) { return (int64_t)V * (dt == DPZ_F32 ? 4 : 2); }

// Blocks per row, a power of two up to 8.  With few rows, as many as keep the
// blocks at two per SM, each with at least one vector per thread; rows of
// half a megabyte and more are split for up to four, which hides a
// cluster's barriers (256 rows of 256,000 fp32: 76 us with one block, 55 with
// 2, 61 with 4; 300 rows of 50,257 bf16: 16.5 us with one, 20 with 2).
inline unsigned row_cluster(int64_t T, int64_t bytes, int threads, int sms)
{
    unsigned n = 1;
    while (n < kMaxCluster && bytes >= (int64_t)2 * n * threads * 16 &&
           (T * n <= sms || (T * n <= 2 * (int64_t)sms && bytes >= (int64_t)2 * n * (256 << 10))))
        n *= 2;
    return n;
}

}  // namespace dpz
