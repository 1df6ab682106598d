// The entry points of include/dpz.h for a replica's attention block: the norm
// of queries and keys with the position rotation, attention, and their
// gradients.  Every one validates all of its arguments before it launches
// anything.
#include "attn.h"

#include <cmath>

#include "api_check.h"
#include "api_util.h"

using namespace dpz;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxHeads = 65535;

int check_size(int64_t n, int64_t lo, int64_t hi, const char* what)
{
    if (n < lo || n > hi)
        return fail(DPZ_ERR_INVALID_ARG, "%s = %lld is outside [%lld, %lld]", what, (long long)n,
                    (long long)lo, (long long)hi);
    return DPZ_OK;
}

// One tensor of T tokens and H heads of D elements (bytes here), or a vector
// as one of each.
struct Buf {
    const char* name;
    uintptr_t lo;
    int64_t T, ld, H, hs, D;   // strides and D in bytes
    bool written;
    bool empty() const { return lo == 0 || T < 1 || H < 1 || D < 1; }
    uintptr_t hi() const { return lo + (T - 1) * ld + (H - 1) * hs + D; }
    // bytes of a token's heads, of a head's tokens
    int64_t token() const { return (H - 1) * hs + D; }
    int64_t head() const { return (T - 1) * ld + D; }
};

// Checks a tensor that has rows and takes its strides; those of a single token
// or head say nothing and become what a dense one's would be.
int take_heads(const dpz_heads* x, int64_t T, int64_t H, int64_t D, int dt, const char* what,
               bool written, Heads* out, Buf* buf)
{
    const int es = elem_bytes(dt);
    *out = {nullptr, D, D};
    *buf = {what, 0, 0, 0, 0, 0, 0, written};
    if (T == 0 || H == 0) return DPZ_OK;
    if (x == nullptr) return fail(DPZ_ERR_INVALID_ARG, "%s is NULL", what);
    DPZ_TRY(check_addr(x->p, what, es));
    int64_t ld = x->ld, hs = x->hs;
    if (H == 1) hs = D;
    if (T == 1) ld = hs > (int64_t(1) << 40) ? 0 : (H - 1) * hs + D;
    const int64_t most = int64_t(1) << 40;
    if (ld < D || hs < D || ld > most || hs > most || (T > 1 && ld > (int64_t(1) << 47) / T) ||
        (H > 1 && hs > (int64_t(1) << 47) / H))
        return fail(DPZ_ERR_INVALID_ARG, "%s: strides %lld (tokens) and %lld (heads) are below %lld "
                    "or too large", what, (long long)x->ld, (long long)x->hs, (long long)D);
    if (ld < (H - 1) * hs + D && hs < (T - 1) * ld + D)
        return fail(DPZ_ERR_INVALID_ARG, "%s: with strides %lld (tokens) and %lld (heads) its "
                    "elements share addresses", what, (long long)ld, (long long)hs);
    *out = {static_cast<char*>(x->p), ld, hs};
    *buf = {what, reinterpret_cast<uintptr_t>(x->p), T, ld * es, H, hs * es, D * es, written};
    return DPZ_OK;
}

Buf vec(const char* name, const void* p, int64_t bytes, bool written)
{
    return {name, reinterpret_cast<uintptr_t>(p), 1, bytes, 1, bytes, bytes, written};
}

// Whether bytes [0, wa) and [d, d + wb), both repeated every s bytes, are apart.
bool apart(uintptr_t a, int64_t wa, uintptr_t b, int64_t wb, int64_t s)
{
    const int64_t d = ((int64_t)(b - a) % s + s) % s;
    return wa <= d && d + wb <= s;
}

// Whether every step of x is a multiple of s.
bool steps_of(const Buf& x, int64_t s)
{
    return (x.T == 1 || x.ld % s == 0) && (x.H == 1 || x.hs % s == 0);
}

// Whether two buffers may share a byte: not if their ranges are apart, or if
// they interleave as ranges of columns of one larger tensor do.
bool overlap(const Buf& a, const Buf& b)
{
    if (a.empty() || b.empty() || a.lo >= b.hi() || b.lo >= a.hi()) return false;
    if (a.T > 1 && b.T > 1 && a.ld == b.ld && apart(a.lo, a.token(), b.lo, b.token(), a.ld))
        return false;
    if (a.H > 1 && b.H > 1 && a.hs == b.hs && apart(a.lo, a.head(), b.lo, b.head(), a.hs))
        return false;
    for (const int64_t s : {a.hs, a.ld})
        if (s > 0 && steps_of(a, s) && steps_of(b, s) && apart(a.lo, a.D, b.lo, b.D, s))
            return false;
    return true;
}

bool same(const Buf& a, const Buf& b)
{
    return a.lo == b.lo && a.ld == b.ld && a.hs == b.hs && a.T == b.T && a.H == b.H;
}

// No buffer that the call writes may share a byte with another one.
int check_bufs(std::initializer_list<Buf> bs)
{
    for (const Buf* a = bs.begin(); a != bs.end(); ++a)
        for (const Buf* b = a + 1; b != bs.end(); ++b)
            if ((a->written || b->written) && overlap(*a, *b))
                return fail(DPZ_ERR_INVALID_ARG, "buffers %s and %s overlap", a->name, b->name);
    return DPZ_OK;
}

Buf unless(bool skip, const Buf& b) { return skip ? Buf{b.name, 0, 0, 0, 0, 0, 0, false} : b; }

int check_rope_sizes(int64_t T, int64_t Hq, int64_t Hk, int64_t D)
{
    DPZ_TRY(check_size(T, 0, kMaxTokens, "T"));
    DPZ_TRY(check_size(Hq, 0, kMaxHeads, "Hq"));
    DPZ_TRY(check_size(Hk, 0, kMaxHeads, "Hk"));
    if (T * (Hq + Hk) > int64_t(1) << 33)
        return fail(DPZ_ERR_INVALID_ARG, "%lld tokens of %lld heads exceed 2^33 in all",
                    (long long)T, (long long)(Hq + Hk));
    return check_size(D, 1, kRopeMaxD, "D");
}

// What attn_qk_norm_rope and its gradient have in common: everything but the
// tensors.
int rope_common(RopeArgs* a, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int dtype,
                const void* wq, const void* wk, int wdtype, float eps, const void* positions,
                int itype, const float* inv_freq, int64_t R, int interleaved)
{
    DPZ_TRY(check_rope_sizes(T, Hq, Hk, D));
    DPZ_TRY(check_elem_type(dtype, "q"));
    DPZ_TRY(check_elem_type(wdtype, "weight"));
    if (!(eps >= 0.0f) || !std::isfinite(eps))
        return fail(DPZ_ERR_INVALID_ARG, "eps = %g must be finite and not negative", eps);
    if (R < 0 || R > D || R % 2 != 0)
        return fail(DPZ_ERR_INVALID_ARG, "R = %lld is not an even number in [0, D = %lld]",
                    (long long)R, (long long)D);
    if (wq != nullptr) DPZ_TRY(check_addr(wq, "wq", elem_bytes(wdtype)));
    if (wk != nullptr) DPZ_TRY(check_addr(wk, "wk", elem_bytes(wdtype)));
    DPZ_TRY(check_ids(positions, itype, R > 0 ? T : 0, "positions"));
    if (R > 0 && T > 0) DPZ_TRY(check_addr(inv_freq, "inv_freq", 4));
    a->T = T;
    a->H[0] = (int)Hq;
    a->H[1] = (int)Hk;
    a->D = (int)D;
    a->dt = dtype;
    a->w[0] = wq;
    a->w[1] = wk;
    a->wdt = wdtype;
    a->eps = eps;
    a->positions = R > 0 ? positions : nullptr;
    a->itype = itype;
    a->inv_freq = inv_freq;
    a->R = (int)R;
    a->interleaved = interleaved != 0;
    return DPZ_OK;
}

int check_attn_sizes(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hk, int64_t D)
{
    DPZ_TRY(check_size(Tq, 0, kMaxTokens, "Tq"));
    DPZ_TRY(check_size(Tk, 0, kMaxTokens, "Tk"));
    DPZ_TRY(check_size(B, 1, kMaxTokens, "B"));
    DPZ_TRY(check_size(Hq, 1, kMaxHeads, "Hq"));
    DPZ_TRY(check_size(Hk, 1, kMaxHeads, "Hk"));
    if (Hq % Hk != 0)
        return fail(DPZ_ERR_INVALID_ARG, "Hq = %lld is not a multiple of Hk = %lld", (long long)Hq,
                    (long long)Hk);
    return check_size(D, 1, kAttnMaxD, "D");
}

int attn_common(AttnArgs* a, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, int dtype,
                int64_t B, const void* cu_q, const void* cu_k, int itype, int causal, float scale)
{
    DPZ_TRY(check_attn_sizes(Tq, Tk, B, Hq, Hk, D));
    DPZ_TRY(check_elem_type(dtype, "q"));
    DPZ_TRY(check_factor(scale, "scale"));
    if ((cu_q == nullptr) != (cu_k == nullptr))
        return fail(DPZ_ERR_INVALID_ARG, "cu_q and cu_k come together");
    if (cu_q != nullptr) {
        DPZ_TRY(check_ids(cu_q, itype, 1, "cu_q"));
        DPZ_TRY(check_ids(cu_k, itype, 1, "cu_k"));
    } else if (Tq % B != 0 || Tk % B != 0) {
        return fail(DPZ_ERR_INVALID_ARG, "Tq = %lld and Tk = %lld are not multiples of B = %lld",
                    (long long)Tq, (long long)Tk, (long long)B);
    }
    a->Tq = Tq;
    a->Tk = Tk;
    a->Hq = (int)Hq;
    a->Hk = (int)Hk;
    a->D = (int)D;
    a->dt = dtype;
    a->B = B;
    a->cu_q = cu_q;
    a->cu_k = cu_k;
    a->len_q = (int)(Tq / B);
    a->len_k = (int)(Tk / B);
    a->itype = itype;
    a->causal = causal != 0;
    a->scale = scale;
    return DPZ_OK;
}

Buf cu_buf(const char* name, const void* cu, int64_t B, int itype)
{
    return vec(name, cu, cu ? (B + 1) * id_bytes(itype) : 0, false);
}

}  // namespace

extern "C" {

DPZ_API int attn_qk_norm_rope(const dpz_heads* q, const dpz_heads* k, int64_t T, int64_t Hq,
                              int64_t Hk, int64_t D, int dtype, const void* wq, const void* wk,
                              int wdtype, float eps, const void* positions, int itype,
                              const float* inv_freq, int64_t R, int interleaved,
                              const dpz_heads* q_out, const dpz_heads* k_out, void* stream)
{
    RopeArgs a{};
    DPZ_TRY(rope_common(&a, T, Hq, Hk, D, dtype, wq, wk, wdtype, eps, positions, itype, inv_freq, R,
                        interleaved));
    Buf bq, bk, oq, ok_;
    DPZ_TRY(take_heads(q, T, Hq, D, dtype, "q", false, &a.in[0], &bq));
    DPZ_TRY(take_heads(k, T, Hk, D, dtype, "k", false, &a.in[1], &bk));
    DPZ_TRY(take_heads(q_out, T, Hq, D, dtype, "q_out", true, &a.out[0], &oq));
    DPZ_TRY(take_heads(k_out, T, Hk, D, dtype, "k_out", true, &a.out[1], &ok_));
    DPZ_TRY(check_bufs({unless(same(bq, oq), bq), unless(same(bk, ok_), bk), oq, ok_,
                        vec("wq", wq, D * elem_bytes(wdtype), false),
                        vec("wk", wk, D * elem_bytes(wdtype), false),
                        vec("positions", a.positions, T * id_bytes(itype), false),
                        vec("inv_freq", R > 0 ? inv_freq : nullptr, R / 2 * 4, false)}));
    if (T == 0 || Hq + Hk == 0) return ok();
    cudaStream_t s = as_stream(stream);
    DPZ_TRY(launch(s, [&] { return launch_rope(a, s); }));
    return ok();
}

DPZ_API size_t attn_qk_norm_rope_workspace_bytes(int64_t T, int64_t Hq, int64_t Hk, int64_t D)
{
    if (check_rope_sizes(T, Hq, Hk, D) != DPZ_OK) return 0;
    const int64_t n = rope_parts(T);
    return sizeof(float) * 2 * (size_t)D * (size_t)(n > 0 ? n : 1);
}

DPZ_API int attn_qk_norm_rope_grad(const dpz_heads* q, const dpz_heads* k, const dpz_heads* dq_out,
                                   const dpz_heads* dk_out, int64_t T, int64_t Hq, int64_t Hk,
                                   int64_t D, int dtype, const void* wq, const void* wk, int wdtype,
                                   float eps, const void* positions, int itype,
                                   const float* inv_freq, int64_t R, int interleaved,
                                   const dpz_heads* dq, const dpz_heads* dk, void* dwq, void* dwk,
                                   void* ws, void* stream)
{
    RopeArgs a{};
    DPZ_TRY(rope_common(&a, T, Hq, Hk, D, dtype, wq, wk, wdtype, eps, positions, itype, inv_freq, R,
                        interleaved));
    Buf bq, bk, gq, gk, oq, ok_;
    DPZ_TRY(take_heads(q, T, Hq, D, dtype, "q", false, &a.in[0], &bq));
    DPZ_TRY(take_heads(k, T, Hk, D, dtype, "k", false, &a.in[1], &bk));
    DPZ_TRY(take_heads(dq_out, T, Hq, D, dtype, "dq_out", false, &a.dout[0], &gq));
    DPZ_TRY(take_heads(dk_out, T, Hk, D, dtype, "dk_out", false, &a.dout[1], &gk));
    DPZ_TRY(take_heads(dq, T, Hq, D, dtype, "dq", true, &a.out[0], &oq));
    DPZ_TRY(take_heads(dk, T, Hk, D, dtype, "dk", true, &a.out[1], &ok_));
    const int wb = elem_bytes(wdtype);
    if (dwq != nullptr) DPZ_TRY(check_addr(dwq, "dwq", wb));
    if (dwk != nullptr) DPZ_TRY(check_addr(dwk, "dwk", wb));
    const bool dw = dwq != nullptr || dwk != nullptr;
    const size_t wsb = dw ? attn_qk_norm_rope_workspace_bytes(T, Hq, Hk, D) : 0;
    if (dw) DPZ_TRY(check_addr(ws, "ws", 16));
    DPZ_TRY(check_bufs({bq, bk, unless(same(gq, oq), gq), unless(same(gk, ok_), gk), oq, ok_,
                        vec("wq", wq, D * wb, false), vec("wk", wk, D * wb, false),
                        vec("positions", a.positions, T * id_bytes(itype), false),
                        vec("inv_freq", R > 0 ? inv_freq : nullptr, R / 2 * 4, false),
                        vec("dwq", dwq, D * wb, true), vec("dwk", dwk, D * wb, true),
                        vec("ws", dw ? ws : nullptr, (int64_t)wsb, true)}));
    a.dw[0] = dwq;
    a.dw[1] = dwk;
    a.partial = static_cast<float*>(ws);
    cudaStream_t s = as_stream(stream);
    // without tokens or heads the weights' gradients are zeros
    if (Hq + Hk == 0) a.T = 0;
    if (a.T > 0) DPZ_TRY(launch(s, [&] { return launch_rope_grad(a, s); }));
    if (dw) DPZ_TRY(launch(s, [&] { return launch_rope_dw(a, s); }));
    return ok();
}

DPZ_API int attn_forward(const dpz_heads* q, const dpz_heads* k, const dpz_heads* v, int64_t Tq,
                         int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, int dtype, int64_t B,
                         const void* cu_q, const void* cu_k, int itype, int causal, float scale,
                         const dpz_heads* out, float* lse, void* stream)
{
    AttnArgs a{};
    DPZ_TRY(attn_common(&a, Tq, Tk, Hq, Hk, D, dtype, B, cu_q, cu_k, itype, causal, scale));
    Buf bq, bk, bv, bo;
    DPZ_TRY(take_heads(q, Tq, Hq, D, dtype, "q", false, &a.q, &bq));
    DPZ_TRY(take_heads(k, Tk, Hk, D, dtype, "k", false, &a.k, &bk));
    DPZ_TRY(take_heads(v, Tk, Hk, D, dtype, "v", false, &a.v, &bv));
    DPZ_TRY(take_heads(out, Tq, Hq, D, dtype, "out", true, &a.out, &bo));
    if (lse != nullptr) DPZ_TRY(check_addr(lse, "lse", 4));
    DPZ_TRY(check_bufs({bq, bk, bv, bo, vec("lse", lse, Hq * Tq * 4, true),
                        cu_buf("cu_q", cu_q, B, itype), cu_buf("cu_k", cu_k, B, itype)}));
    if (Tq == 0) return ok();
    a.lse = lse;
    cudaStream_t s = as_stream(stream);
    DPZ_TRY(launch(s, [&] {
        return attn_tc_takes(a, false) ? launch_attn_tc(a, s) : launch_attn_any(a, s);
    }));
    return ok();
}

DPZ_API size_t attn_grad_workspace_bytes(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hk,
                                         int64_t D)
{
    if (check_attn_sizes(Tq, Tk, B, Hq, Hk, D) != DPZ_OK) return 0;
    return sizeof(float) * (size_t)Hq * (size_t)(Tq > 0 ? Tq : 1);
}

DPZ_API int attn_grad(const dpz_heads* q, const dpz_heads* k, const dpz_heads* v,
                      const dpz_heads* out, const float* lse, const dpz_heads* dout, int64_t Tq,
                      int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, int dtype, int64_t B,
                      const void* cu_q, const void* cu_k, int itype, int causal, float scale,
                      const dpz_heads* dq, const dpz_heads* dk, const dpz_heads* dv, void* ws,
                      void* stream)
{
    AttnArgs a{};
    DPZ_TRY(attn_common(&a, Tq, Tk, Hq, Hk, D, dtype, B, cu_q, cu_k, itype, causal, scale));
    Buf bq, bk, bv, bo, bg, oq, ok_, ov;
    DPZ_TRY(take_heads(q, Tq, Hq, D, dtype, "q", false, &a.q, &bq));
    DPZ_TRY(take_heads(k, Tk, Hk, D, dtype, "k", false, &a.k, &bk));
    DPZ_TRY(take_heads(v, Tk, Hk, D, dtype, "v", false, &a.v, &bv));
    DPZ_TRY(take_heads(out, Tq, Hq, D, dtype, "out", false, &a.out, &bo));
    DPZ_TRY(take_heads(dout, Tq, Hq, D, dtype, "dout", false, &a.dout, &bg));
    DPZ_TRY(take_heads(dq, Tq, Hq, D, dtype, "dq", true, &a.dq, &oq));
    DPZ_TRY(take_heads(dk, Tk, Hk, D, dtype, "dk", true, &a.dk, &ok_));
    DPZ_TRY(take_heads(dv, Tk, Hk, D, dtype, "dv", true, &a.dv, &ov));
    if (Tq > 0) DPZ_TRY(check_addr(lse, "lse", 4));
    DPZ_TRY(check_addr(ws, "ws", 16));
    const size_t wsb = attn_grad_workspace_bytes(Tq, Tk, B, Hq, Hk, D);
    DPZ_TRY(check_bufs({bq, bk, bv, bo, vec("lse", Tq > 0 ? lse : nullptr, Hq * Tq * 4, false), bg,
                        oq, ok_, ov, vec("ws", ws, (int64_t)wsb, true),
                        cu_buf("cu_q", cu_q, B, itype), cu_buf("cu_k", cu_k, B, itype)}));
    a.lse = const_cast<float*>(lse);
    a.delta = static_cast<float*>(ws);
    cudaStream_t s = as_stream(stream);
    // the queries' gradient leaves delta in the workspace for the keys' and values'
    const bool tc = attn_tc_takes(a, true);
    if (Tq > 0)
        DPZ_TRY(launch(s, [&] { return tc ? launch_attn_tc_dq(a, s) : launch_attn_any_dq(a, s); }));
    if (Tk > 0)
        DPZ_TRY(launch(s, [&] { return tc ? launch_attn_tc_dkv(a, s) : launch_attn_any_dkv(a, s); }));
    return ok();
}

}  // extern "C"
