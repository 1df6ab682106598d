// The entry points of include/dpz.h over lists of tensors: their global norm
// and its clipping.  Every one validates all of its arguments before it
// launches anything.
#include <algorithm>
#include <cmath>

#include "api_check.h"
#include "api_util.h"
#include "tensors.h"

using namespace dpz;

namespace {

constexpr int kMaxTensors = DPZ_MAX_TENSORS;

int64_t bytes_of(const dpz_tensor& t) { return t.n * elem_bytes((int)t.dtype); }

int check_list(const dpz_tensor* l, int n, const char* what)
{
    if (n < 0 || n > kMaxTensors)
        return fail(DPZ_ERR_INVALID_ARG, "n = %d is outside [0, %d]", n, kMaxTensors);
    if (n > 0 && l == nullptr) return fail(DPZ_ERR_INVALID_ARG, "%s is NULL", what);
    int64_t chunks = 0;
    for (int i = 0; i < n; ++i) {
        if (l[i].dtype != DPZ_F32 && l[i].dtype != DPZ_BF16)
            return fail(DPZ_ERR_INVALID_ARG, "%s %d: dtype %lld is not supported", what, i,
                        (long long)l[i].dtype);
        if (l[i].n < 0 || l[i].n > int64_t(1) << 44)
            return fail(DPZ_ERR_INVALID_ARG, "%s %d: %lld elements are outside [0, 2^44]", what, i,
                        (long long)l[i].n);
        if (l[i].n == 0) continue;
        if (l[i].p == nullptr) return fail(DPZ_ERR_INVALID_ARG, "%s %d is NULL", what, i);
        if (reinterpret_cast<uintptr_t>(l[i].p) % elem_bytes((int)l[i].dtype) != 0)
            return fail(DPZ_ERR_ALIGN, "%s %d is not aligned to its elements", what, i);
        chunks += list_chunks(l[i]);
        if (chunks >= int64_t(1) << 31)
            return fail(DPZ_ERR_INVALID_ARG, "%s: the tensors exceed 2^47 bytes", what);
    }
    return DPZ_OK;
}

int64_t chunks_of(const dpz_tensor* l, int n)
{
    int64_t c = 0;
    for (int i = 0; i < n; ++i) c += list_chunks(l[i]);
    return c;
}

// A written range and the tensor that it is.
struct Span {
    uintptr_t lo, hi;
    int i;
};

// No output may share a byte with another, nor with an input other than its own,
// which it may be.  The outputs are sorted by address (they often are already).
int check_outputs(const dpz_tensor* in, const dpz_tensor* out, int n, const float* norm,
                  Span* spans)
{
    int m = 0;
    for (int i = 0; i < n; ++i)
        if (out[i].n > 0) {
            const uintptr_t lo = reinterpret_cast<uintptr_t>(out[i].p);
            spans[m++] = {lo, lo + (uintptr_t)bytes_of(out[i]), i};
        }
    const auto before = [](const Span& a, const Span& b) { return a.lo < b.lo; };
    if (!std::is_sorted(spans, spans + m, before)) std::sort(spans, spans + m, before);
    for (int j = 1; j < m; ++j)
        if (spans[j].lo < spans[j - 1].hi)
            return fail(DPZ_ERR_INVALID_ARG, "outputs %d and %d overlap", spans[j - 1].i, spans[j].i);
    // the first output that ends behind lo
    const auto first_past = [&](uintptr_t lo) {
        return std::upper_bound(spans, spans + m, lo,
                                [](uintptr_t x, const Span& s) { return x < s.hi; });
    };
    for (int i = 0; i < n; ++i) {
        if (in[i].n == 0) continue;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(in[i].p);
        const uintptr_t hi = lo + (uintptr_t)bytes_of(in[i]);
        const Span* s = first_past(lo);
        if (s == spans + m || s->lo >= hi) continue;
        const bool own = s->i == i && s->lo == lo && s->hi == hi && in[i].dtype == out[i].dtype;
        if (!own)
            return fail(DPZ_ERR_INVALID_ARG, "input %d and output %d overlap", i, s->i);
    }
    const uintptr_t at = reinterpret_cast<uintptr_t>(norm);
    const Span* s = first_past(at);
    if (s != spans + m && s->lo < at + 4)
        return fail(DPZ_ERR_INVALID_ARG, "norm and output %d overlap", s->i);
    return DPZ_OK;
}

}  // namespace

extern "C" {

DPZ_API size_t tensors_workspace_bytes(const dpz_tensor* tensors, int n)
{
    if (check_list(tensors, n, "tensor") != DPZ_OK) return 0;
    const int64_t c = chunks_of(tensors, n);
    return sizeof(double) * (size_t)(c > 0 ? c : 1);
}

DPZ_API int tensors_norm(const dpz_tensor* tensors, int n, float* norm_out, void* ws,
                            void* stream)
{
    DPZ_TRY(check_list(tensors, n, "tensor"));
    DPZ_TRY(check_addr(norm_out, "norm_out", 4));
    DPZ_TRY(check_addr(ws, "ws", 16));
    const int64_t chunks = chunks_of(tensors, n);
    const Range w = range("ws", ws, 8 * (chunks > 0 ? chunks : 1)), o = range("norm_out", norm_out, 4);
    if (w.lo < o.hi && o.lo < w.hi)
        return fail(DPZ_ERR_INVALID_ARG, "buffers ws and norm_out overlap");
    for (int i = 0; i < n; ++i) {
        const Range t = range("tensor", tensors[i].p, bytes_of(tensors[i]));
        if ((t.lo < w.hi && w.lo < t.hi) || (t.lo < o.hi && o.lo < t.hi))
            return fail(DPZ_ERR_INVALID_ARG, "tensor %d and ws or norm_out overlap", i);
    }
    cudaStream_t s = as_stream(stream);
    double* partial = static_cast<double*>(ws);
    for (int i = 0; i < n; i += kListMost) {
        const int m = std::min(kListMost, n - i);
        const int64_t c = chunks_of(tensors + i, m);
        if (c == 0) continue;
        DPZ_TRY(launch(s, [&] { return launch_tensors_sumsq(tensors + i, m, partial, s); }));
        partial += c;
    }
    DPZ_TRY(launch(s, [&] {
        return launch_tensors_norm(static_cast<double*>(ws), chunks, norm_out, s);
    }));
    return ok();
}

DPZ_API int tensors_clip(const dpz_tensor* tensors, const dpz_tensor* out, int n,
                            const float* norm, float clip_norm, void* stream)
{
    DPZ_TRY(check_list(tensors, n, "tensor"));
    DPZ_TRY(check_list(out, n, "output"));
    DPZ_TRY(check_addr(norm, "norm", 4));
    if (!(clip_norm > 0.0f) || !std::isfinite(clip_norm))
        return fail(DPZ_ERR_INVALID_ARG, "clip_norm = %g must be positive and finite", clip_norm);
    for (int i = 0; i < n; ++i)
        if (tensors[i].n != out[i].n)
            return fail(DPZ_ERR_INVALID_ARG, "output %d has %lld elements, its input %lld", i,
                        (long long)out[i].n, (long long)tensors[i].n);
    thread_local Span spans[kMaxTensors];
    DPZ_TRY(check_outputs(tensors, out, n, norm, spans));
    cudaStream_t s = as_stream(stream);
    for (int i = 0; i < n; i += kListMost) {
        const int m = std::min(kListMost, n - i);
        if (chunks_of(tensors + i, m) == 0) continue;
        DPZ_TRY(launch(s, [&] { return launch_tensors_clip(tensors + i, out + i, m, norm, clip_norm, s); }));
    }
    return ok();
}

}  // extern "C"
