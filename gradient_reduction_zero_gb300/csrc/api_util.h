// What the entry points of api.cpp and lm_api.cpp share: status codes and the
// last-error message, checks of pointers and overlaps, and the launch with
// its accounting and optional per-launch event timing.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <initializer_list>
#include <mutex>
#include <string>
#include <vector>

#include "dpz.h"
#include "internal.h"

namespace dpz {

// Set the calling thread's error message and return `code`; clear it and
// return DPZ_OK.
__attribute__((format(printf, 2, 3))) int fail(int code, const char* fmt, ...);
int ok();

inline int elem_bytes(int dt) { return dt == DPZ_F32 ? 4 : 2; }

#define DPZ_TRY(x)                     \
    do {                               \
        int rc_ = (x);                 \
        if (rc_ != DPZ_OK) return rc_; \
    } while (0)

struct Range {
    const char* name;
    uintptr_t lo, hi;
};

inline Range range(const char* name, const void* p, int64_t bytes)
{
    uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {name, lo, lo + static_cast<uintptr_t>(bytes)};
}

// The byte ranges of one call's buffers, held on the stack (no allocation on
// the launch path).  A NULL buffer is not added.  No call has more than seven
// buffers; one past kMax would be dropped, never written out of bounds.
struct Ranges {
    static constexpr int kMax = 8;
    Range r[kMax];
    int n = 0;
    Ranges(std::initializer_list<Range> rs)
    {
        for (const Range& x : rs)
            if (n < kMax) r[n++] = x;
    }
    void add(const char* name, const void* p, int64_t bytes)
    {
        if (p != nullptr && n < kMax) r[n++] = range(name, p, bytes);
    }
};

inline int check_disjoint(const Ranges& rs)
{
    for (int i = 0; i < rs.n; ++i)
        for (int j = i + 1; j < rs.n; ++j)
            if (rs.r[i].lo < rs.r[j].hi && rs.r[j].lo < rs.r[i].hi)
                return fail(DPZ_ERR_INVALID_ARG, "buffers %s and %s overlap", rs.r[i].name,
                            rs.r[j].name);
    return DPZ_OK;
}

// ------------------------------------------------------------ profiling

struct Profiler {
    std::mutex mu;
    std::atomic<bool> on{false};     // read without the lock on every launch
    int cap = 0;
    int used = 0;
    std::vector<cudaEvent_t> ev;
    std::vector<std::string> names;
};
extern Profiler g_prof;
extern std::atomic<int64_t> g_launches;

template <class F>
int launch(cudaStream_t s, F&& f)
{
    int slot = -1;
    if (g_prof.on.load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lk(g_prof.mu);
        if (g_prof.on.load(std::memory_order_relaxed) && g_prof.used < g_prof.cap)
            slot = g_prof.used++;
    }
    if (slot >= 0) cudaEventRecord(g_prof.ev[2 * slot], s);
    cudaError_t e = f();
    const char* name = last_kernel_name();
    if (slot >= 0) {
        cudaEventRecord(g_prof.ev[2 * slot + 1], s);
        std::lock_guard<std::mutex> lk(g_prof.mu);
        g_prof.names[slot] = name;
    }
    if (e != cudaSuccess)
        return fail(DPZ_ERR_CUDA, "launch of %s failed: %s", name, cudaGetErrorString(e));
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return DPZ_OK;
}

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

}  // namespace dpz
