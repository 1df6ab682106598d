// Rows of logits over a vocabulary: log probabilities of given tokens with
// entropy and top alternatives, distillation from a teacher's top logits, and
// the gradients of both.
#include <cfloat>
#include <cmath>

#include "bulk.cuh"
#include "device.cuh"
#include "internal.h"
#include "lm.h"

namespace dpz {

namespace {

constexpr int kRowThreads = 512;
constexpr int kRowWarps = kRowThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int load_token(const Ids& ids, int64_t i, int64_t V)
{
    const int64_t v = ids.it == DPZ_I64 ? static_cast<const int64_t*>(ids.p)[i]
                                        : (int64_t) static_cast<const int*>(ids.p)[i];
    return v >= 0 && v < V ? (int)v : -1;
}

// 2^u by the hardware's instruction: at most 2 units in the last place off,
// which is below the rounding of the exponent that it is given here.
__device__ __forceinline__ float ex2(float u)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(u));
    return e;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

// ------------------------------------------------------------ a row's elements
//
// A row may begin at any element (a vocabulary of 50,257 shifts each row), so
// it is a head of single elements up to the first 16-byte boundary, a body of
// 16-byte vectors, and a tail.

template <int DT>
struct El;

template <>
struct El<DPZ_F32> {
    static constexpr int kBytes = 4, kVec = 4;
    static __device__ __forceinline__ float load(const char* p)
    {
        return *reinterpret_cast<const float*>(p);
    }
    static __device__ __forceinline__ void store(char* p, float x)
    {
        *reinterpret_cast<float*>(p) = x;
    }
    static __device__ __forceinline__ void unpack(const uint4& w, float x[kVec])
    {
        x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float x[kVec])
    {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
    static __device__ __forceinline__ float vec_max(const uint4& w)
    {
        float x[kVec];
        unpack(w, x);
        return max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3]));
    }
};

template <>
struct El<DPZ_BF16> {
    static constexpr int kBytes = 2, kVec = 8;
    static __device__ __forceinline__ float load(const char* p)
    {
        return __uint_as_float((uint32_t)*reinterpret_cast<const unsigned short*>(p) << 16);
    }
    static __device__ __forceinline__ void store(char* p, float x)
    {
        *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(x);
    }
    static __device__ __forceinline__ void unpack(const uint4& w, float x[kVec])
    {
        Group<1>::unpack({w}, x);
    }
    static __device__ __forceinline__ uint4 pack(const float x[kVec])
    {
        return Group<1>::pack(x).w;
    }
    static __device__ __forceinline__ float vec_max(const uint4& w)
    {
        const auto b = [](const uint32_t& u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
        const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(b(w.x), b(w.y)), __hmax2_nan(b(w.z), b(w.w)));
        return max_nan(__low2float(m), __high2float(m));
    }
};

struct RowSpan {
    int head;      // elements before the first 16-byte boundary
    int nvec;      // 16-byte vectors
    int tail;      // elements after the last
};

template <int DT>
__device__ __forceinline__ RowSpan row_span(const char* p, int64_t V)
{
    constexpr int kB = El<DT>::kBytes, kV = El<DT>::kVec;
    const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15);
    RowSpan s;
    s.head = (int)min(V, (int64_t)((16 - off) & 15) / kB);
    s.nvec = (int)((V - s.head) / kV);
    s.tail = (int)(V - s.head - (int64_t)s.nvec * kV);
    return s;
}

// Calls f(x, j) for each element x of index j that belongs to this thread.
template <int DT, class F>
__device__ __forceinline__ void for_elements(const char* row, const RowSpan& s, F&& f)
{
    constexpr int kB = El<DT>::kBytes, kV = El<DT>::kVec;
    const int t = threadIdx.x;
    if (t < s.head) f(El<DT>::load(row + t * kB), t);
    const char* body = row + s.head * kB;
    for (int i = t; i < s.nvec; i += kRowThreads) {
        float x[kV];
        El<DT>::unpack(ld16(body + (int64_t)i * 16), x);
#pragma unroll
        for (int j = 0; j < kV; ++j) f(x[j], s.head + i * kV + j);
    }
    if (t < s.tail) {
        const int j = s.head + s.nvec * kV + t;
        f(El<DT>::load(row + (int64_t)j * kB), j);
    }
}

// ------------------------------------------------------------ softmax statistics
//
// Running maximum m, S = sum 2^u and U = sum u 2^u over a part of a row, with
// u = (x - m) c and c = scale * log2(e).  The difference is taken before the
// product, so a maximum of the type's lowest value does not overflow.  A
// masked element (-inf) has 2^u = 0; its u is held at a finite value so that
// 0 * u is 0.
struct Stat {
    float m, S, U;
};

constexpr float kMinExp = -16384.0f;

__device__ __forceinline__ void stat_rebase(Stat& s, float m, float c)
{
    // 2^((x - m) c) = 2^((x - s.m) c) * 2^d with d = (s.m - m) c
    const float d = fmaxf((s.m - m) * c, kMinExp);
    const float f = ex2(d);
    s.U = f * __fmaf_rn(d, s.S, s.U);
    s.S *= f;
    s.m = m;
}

__device__ __forceinline__ Stat stat_join(Stat a, Stat b, float c)
{
    const float m = max_nan(a.m, b.m);
    if (m == -INFINITY) return a;             // nothing in either
    stat_rebase(a, m, c);
    stat_rebase(b, m, c);
    return {m, a.S + b.S, a.U + b.U};
}

__device__ __forceinline__ Stat warp_stat(Stat s, float c)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Stat b{__shfl_xor_sync(0xffffffffu, s.m, o), __shfl_xor_sync(0xffffffffu, s.S, o),
                     __shfl_xor_sync(0xffffffffu, s.U, o)};
        s = stat_join(s, b, c);
    }
    return s;
}

// The statistics of a whole row, in every thread.
template <int DT>
__device__ __forceinline__ Stat row_stat(const char* row, const RowSpan& span, float c)
{
    __shared__ Stat warp_part[kRowWarps];
    Stat s{-INFINITY, 0.0f, 0.0f};
    for_elements<DT>(row, span, [&](float x, int) {
        const float m = max_nan(s.m, x);
        if (m != s.m) stat_rebase(s, m, c);
        const float u = x == -INFINITY ? kMinExp : fmaxf((x - m) * c, kMinExp);
        const float e = ex2(u);
        s.S += e;
        s.U = __fmaf_rn(e, u, s.U);
    });
    s = warp_stat(s, c);
    if ((threadIdx.x & 31) == 0) warp_part[threadIdx.x >> 5] = s;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    s = lane < kRowWarps ? warp_part[lane] : Stat{-INFINITY, 0.0f, 0.0f};
    return warp_stat(s, c);
}

// lse and entropy of a row's statistics; m NaN or +inf: NaN, m -inf: -inf and 0.
struct RowResult {
    float lse, log2S, entropy;
    bool empty, bad;
};

__device__ __forceinline__ RowResult row_result(const Stat& s, float scale)
{
    RowResult r;
    r.empty = s.m == -INFINITY;
    r.bad = !(s.m < INFINITY);
    r.log2S = log2f(s.S);
    r.lse = r.bad ? quiet_nan() : r.empty ? -INFINITY : __fmaf_rn(s.m, scale, r.log2S * kLn2);
    r.entropy = r.bad ? quiet_nan() : r.empty ? 0.0f : (r.log2S - s.U / s.S) * kLn2;
    return r;
}

__device__ __forceinline__ float logprob_of(float x, const Stat& s, const RowResult& r, float scale)
{
    if (r.bad) return quiet_nan();
    if (r.empty) return -INFINITY;
    return __fmaf_rn(x - s.m, scale, -r.log2S * kLn2);
}

// ------------------------------------------------------------ top alternatives
//
// An element's rank key: the value's order in the upper word (NaN highest),
// the complement of its index in the lower, so that the largest key is the
// largest value of the lowest index.  0 is below every key.

__device__ __forceinline__ uint64_t rank_key(float x, int j)
{
    const uint32_t b = __float_as_uint(x + 0.0f);   // -0 becomes +0
    uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
    if (x != x) o = 0xffffff00u;
    return (uint64_t)o << 32 | (0xffffffffu - (uint32_t)j);
}

__device__ __forceinline__ uint64_t warp_max64(uint64_t k)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t b = __shfl_xor_sync(0xffffffffu, k, o);
        k = b > k ? b : k;
    }
    return k;
}

// ------------------------------------------------------------ log probabilities

template <int DT>
__global__ void __launch_bounds__(kRowThreads) k_logprobs(LogprobArgs a)
{
    __shared__ uint64_t warp_best[kRowWarps];
    pdl_enter();
    const int64_t t = blockIdx.x;
    const char* row = a.x.p + t * a.x.ld * El<DT>::kBytes;
    const RowSpan span = row_span<DT>(row, a.V);
    const float c = a.scale * kLog2e;
    const Stat s = row_stat<DT>(row, span, c);
    const RowResult r = row_result(s, a.scale);
    if (threadIdx.x == 0) {
        if (a.logprob != nullptr) {
            const int y = load_token(a.targets, t, a.V);
            a.logprob[t] =
                y < 0 ? 0.0f : logprob_of(El<DT>::load(row + (int64_t)y * El<DT>::kBytes), s, r, a.scale);
        }
        if (a.lse != nullptr) a.lse[t] = r.lse;
        if (a.entropy != nullptr) a.entropy[t] = r.entropy;
    }
    // K rounds: the largest key below the last one.  Each thread keeps its own
    // best and looks for the next one only when its best was taken.
    uint64_t prev = ~uint64_t(0), best = 0;
    bool stale = true;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    for (int k = 0; k < a.K; ++k) {
        if (stale) {
            best = 0;
            for_elements<DT>(row, span, [&](float x, int j) {
                const uint64_t key = rank_key(x, j);
                if (key < prev && key > best) best = key;
            });
        }
        const uint64_t wb = warp_max64(best);
        if (lane == 0) warp_best[wid] = wb;
        __syncthreads();
        prev = warp_max64(lane < kRowWarps ? warp_best[lane] : 0);
        __syncthreads();
        stale = best == prev;
        if (threadIdx.x == 0) {
            const int j = (int)(0xffffffffu - (uint32_t)prev);
            const float x = El<DT>::load(row + (int64_t)j * El<DT>::kBytes);
            const int64_t at = t * a.K + k;
            if (a.targets.it == DPZ_I64) static_cast<int64_t*>(a.top_ids)[at] = j;
            else static_cast<int*>(a.top_ids)[at] = j;
            a.top_logprobs[at] = logprob_of(x, s, r, a.scale);
        }
    }
}

// ------------------------------------------------------------ gradients
//
// f(x, j) gives the gradient of element x of index j; a row is read and
// written by the same thread, so the output may be the input.
template <int DT, class F>
__device__ __forceinline__ void map_row(const char* row, char* out, const RowSpan& s, F&& f)
{
    constexpr int kB = El<DT>::kBytes, kV = El<DT>::kVec;
    const int t = threadIdx.x;
    if (t < s.head) El<DT>::store(out + t * kB, f(El<DT>::load(row + t * kB), t));
    // the output's rows may be aligned otherwise than the input's
    const bool same = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    const int64_t body = s.head * kB;
    for (int i = t; i < s.nvec; i += kRowThreads) {
        float x[kV];
        El<DT>::unpack(ld16(row + body + (int64_t)i * 16), x);
#pragma unroll
        for (int j = 0; j < kV; ++j) x[j] = f(x[j], s.head + i * kV + j);
        char* q = out + body + (int64_t)i * 16;
        if (same) st16(q, El<DT>::pack(x));
        else
#pragma unroll
            for (int j = 0; j < kV; ++j) El<DT>::store(q + j * kB, x[j]);
    }
    if (t < s.tail) {
        const int j = s.head + s.nvec * kV + t;
        El<DT>::store(out + (int64_t)j * kB, f(El<DT>::load(row + (int64_t)j * kB), j));
    }
}

template <int DT>
__device__ __forceinline__ void zero_row(char* out, int64_t V)
{
    const RowSpan s = row_span<DT>(out, V);
    constexpr int kB = El<DT>::kBytes, kV = El<DT>::kVec;
    const int t = threadIdx.x;
    if (t < s.head) El<DT>::store(out + t * kB, 0.0f);
    for (int i = t; i < s.nvec; i += kRowThreads)
        st16(out + s.head * kB + (int64_t)i * 16, make_uint4(0, 0, 0, 0));
    if (t < s.tail) El<DT>::store(out + (s.head + (int64_t)s.nvec * kV + t) * kB, 0.0f);
}

template <int DT>
__global__ void __launch_bounds__(kRowThreads) k_logprobs_grad(LogprobGradArgs a)
{
    pdl_enter();
    const int64_t t = blockIdx.x;
    const char* row = a.x.p + t * a.x.ld * El<DT>::kBytes;
    char* out = a.dx.p + t * a.dx.ld * El<DT>::kBytes;
    const int y = load_token(a.targets, t, a.V);
    const float g = y < 0 ? 0.0f : a.dlogprob[t];
    const float h = a.dentropy != nullptr ? a.dentropy[t] : 0.0f;
    const float lse = a.lse[t];
    if ((g == 0.0f && h == 0.0f) || lse == -INFINITY) {
        zero_row<DT>(out, a.V);
        return;
    }
    const float H = h != 0.0f ? a.entropy[t] : 0.0f;
    // -p (g + h (log p + H)) = p (A + B log2 p)
    const float A = -__fmaf_rn(h, H, g) * a.scale, B = -h * kLn2 * a.scale;
    const float gs = g * a.scale;
    map_row<DT>(row, out, row_span<DT>(row, a.V), [&](float x, int j) {
        const float u = max_nan(__fmaf_rn(x, a.scale, -lse) * kLog2e, kMinExp);
        const float d = ex2(u) * __fmaf_rn(B, u, A);
        return j == y ? d + gs : d;
    });
}

// ------------------------------------------------------------ distillation

// The teacher's entries of one row in shared memory: tokens (-1: absent), the
// student's logits there, probabilities and their logarithms.
struct Teacher {
    int id[DPZ_LM_MAX_TEACHER];
    float x[DPZ_LM_MAX_TEACHER], q[DPZ_LM_MAX_TEACHER], logq[DPZ_LM_MAX_TEACHER];
    int any;
};

__device__ __forceinline__ float warp_max_nan(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float warp_sum_all(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One warp loads a row's entries and their softmax.
template <int DT>
__device__ __forceinline__ void load_teacher(const DistillArgs& a, int64_t t, const char* row,
                                             Teacher& w)
{
    const int lane = threadIdx.x & 31;
    float m = -INFINITY;
    for (int k = lane; k < a.K; k += 32) {
        const int64_t at = t * a.K + k;
        int id = load_token(a.ids, at, a.V);
        float v = a.teacher.dt == DPZ_F32 ? El<DPZ_F32>::load(a.teacher.p + at * 4)
                                          : El<DPZ_BF16>::load(a.teacher.p + at * 2);
        if (v == -INFINITY) id = -1;
        if (id < 0) v = -INFINITY;
        w.id[k] = id;
        w.x[k] = id < 0 ? 0.0f : El<DT>::load(row + (int64_t)id * El<DT>::kBytes);
        w.logq[k] = v;
        m = max_nan(m, v);
    }
    m = warp_max_nan(m);
    float S = 0.0f;
    for (int k = lane; k < a.K; k += 32) {
        // the difference before the product, as for the student
        const float v = w.id[k] < 0 ? -INFINITY : (w.logq[k] - m) * a.inv_tau;
        w.logq[k] = v;
        S += w.id[k] < 0 ? 0.0f : expf(v);
    }
    S = warp_sum_all(S);
    const float logS = logf(S);
    for (int k = lane; k < a.K; k += 32) {
        const float v = w.logq[k] - logS;
        w.logq[k] = v;
        w.q[k] = w.id[k] < 0 ? 0.0f : expf(v);
    }
    if (lane == 0) w.any = m != -INFINITY;
}

template <int DT, bool LOSS, bool GRAD>
__global__ void __launch_bounds__(kRowThreads) k_distill(DistillArgs a)
{
    __shared__ Teacher w;
    pdl_enter();
    const int64_t t = blockIdx.x;
    const char* row = a.x.p + t * a.x.ld * El<DT>::kBytes;
    char* out = GRAD ? a.dx.p + t * a.dx.ld * El<DT>::kBytes : nullptr;
    const float wt = GRAD ? a.dloss[t] : 0.0f;
    if (!LOSS && wt == 0.0f) {
        zero_row<DT>(out, a.V);
        return;
    }
    const RowSpan span = row_span<DT>(row, a.V);
    const float c = a.inv_tau * kLog2e;
    if (threadIdx.x < 32) load_teacher<DT>(a, t, row, w);
    float lse;
    if (LOSS) {
        const Stat s = row_stat<DT>(row, span, c);
        const RowResult r = row_result(s, a.inv_tau);
        lse = r.lse;
        if (threadIdx.x < 32) {
            float sum = 0.0f;
            for (int k = threadIdx.x; k < a.K; k += 32)
                if (w.q[k] != 0.0f)
                    sum += w.q[k] * (w.logq[k] - logprob_of(w.x[k], s, r, a.inv_tau));
            sum = warp_sum_all(sum);
            if (threadIdx.x == 0) {
                a.loss[t] = w.any ? sum : 0.0f;
                if (a.lse != nullptr) a.lse[t] = lse;
            }
        }
    } else {
        lse = a.lse_in[t];
    }
    if (!GRAD) return;
    __syncthreads();
    if (wt == 0.0f || !w.any || lse == -INFINITY) {
        zero_row<DT>(out, a.V);
        return;
    }
    const float ws = wt * a.inv_tau;
    const auto p = [&](float x) {
        return ex2(max_nan(__fmaf_rn(x, a.inv_tau, -lse) * kLog2e, kMinExp));
    };
    map_row<DT>(row, out, span, [&](float x, int) { return ws * p(x); });
    __syncthreads();
    // the entries' tokens again, now with their q
    for (int k = threadIdx.x; k < a.K; k += kRowThreads) {
        const int id = w.id[k];
        if (id < 0) continue;
        float q = 0.0f;
        bool first = true;
        for (int i = 0; i < a.K; ++i)
            if (w.id[i] == id) {
                if (i < k) first = false;
                q += w.q[i];
            }
        if (first) El<DT>::store(out + (int64_t)id * El<DT>::kBytes, ws * (p(w.x[k]) - q));
    }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t s)
{
    set_last_kernel_name("lm_logprobs");
    auto fn = a.x.dt == DPZ_BF16 ? k_logprobs<DPZ_BF16> : k_logprobs<DPZ_F32>;
    return launch_kernel(fn, dim3((unsigned)a.T), dim3(kRowThreads), 0, s, true, 0u, a);
}

cudaError_t launch_logprobs_grad(const LogprobGradArgs& a, cudaStream_t s)
{
    set_last_kernel_name("lm_logprobs_grad");
    auto fn = a.x.dt == DPZ_BF16 ? k_logprobs_grad<DPZ_BF16> : k_logprobs_grad<DPZ_F32>;
    return launch_kernel(fn, dim3((unsigned)a.T), dim3(kRowThreads), 0, s, true, 0u, a);
}

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t s)
{
    const bool b = a.x.dt == DPZ_BF16;
    void (*fn)(DistillArgs);
    if (a.loss != nullptr && a.dx.p != nullptr) {
        set_last_kernel_name("lm_distill_step");
        fn = b ? k_distill<DPZ_BF16, true, true> : k_distill<DPZ_F32, true, true>;
    } else if (a.loss != nullptr) {
        set_last_kernel_name("lm_distill");
        fn = b ? k_distill<DPZ_BF16, true, false> : k_distill<DPZ_F32, true, false>;
    } else {
        set_last_kernel_name("lm_distill_grad");
        fn = b ? k_distill<DPZ_BF16, false, true> : k_distill<DPZ_F32, false, true>;
    }
    return launch_kernel(fn, dim3((unsigned)a.T), dim3(kRowThreads), 0, s, true, 0u, a);
}

}  // namespace dpz
