// The entry points of include/dpz.h that work on a replica's vocabulary-sized
// ends: embedding lookup and gradient, log probabilities, distillation.
// Every one validates all of its arguments before it launches anything.
#include "lm.h"

#include <cmath>

#include "api_check.h"
#include "api_util.h"

using namespace dpz;

namespace {

int check_rows(int64_t T, int64_t V)
{
    if (T < 0 || T >= (int64_t(1) << 31))
        return fail(DPZ_ERR_INVALID_ARG, "T = %lld is outside [0, 2^31)", (long long)T);
    if (V < 1 || V >= (int64_t(1) << 30))
        return fail(DPZ_ERR_INVALID_ARG, "V = %lld is outside [1, 2^30)", (long long)V);
    return DPZ_OK;
}

int check_width(int64_t D)
{
    if (D < 1 || D >= (int64_t(1) << 20))
        return fail(DPZ_ERR_INVALID_ARG, "D = %lld is outside [1, 2^20)", (long long)D);
    return DPZ_OK;
}

// A matrix of `rows` rows of `cols` elements; not looked at without rows.
int check_mat(const void* p, int64_t ld, int64_t rows, int64_t cols, int dt, const char* what)
{
    DPZ_TRY(check_elem_type(dt, what));
    if (ld < cols || ld >= (int64_t(1) << 40))
        return fail(DPZ_ERR_INVALID_ARG, "%s: row stride %lld is outside [%lld, 2^40)", what,
                    (long long)ld, (long long)cols);
    if (rows > 0 && ld > (int64_t(1) << 48) / rows)
        return fail(DPZ_ERR_INVALID_ARG, "%s: %lld rows of stride %lld exceed 2^48 elements", what,
                    (long long)rows, (long long)ld);
    return rows > 0 ? check_addr(p, what, elem_bytes(dt)) : DPZ_OK;
}

// Whether two matrices of one size and type are the same elements: a single
// row's stride says nothing.
bool same_mat(const void* p, int64_t ldp, const void* q, int64_t ldq, int64_t rows)
{
    return p == q && (ldp == ldq || rows < 2);
}

Mat mat(const void* p, int64_t ld, int dt)
{
    return {static_cast<char*>(const_cast<void*>(p)), ld, dt};
}

}  // namespace

extern "C" {

DPZ_API int lm_embedding(const void* table, int64_t ld_table, int64_t V, int64_t D, int wdtype,
                         const void* ids, int itype, int64_t T, float scale, void* out,
                         int64_t ld_out, int odtype, void* stream)
{
    DPZ_TRY(check_rows(T, V));
    DPZ_TRY(check_width(D));
    DPZ_TRY(check_mat(table, ld_table, V, D, wdtype, "table"));
    DPZ_TRY(check_ids(ids, itype, T, "ids"));
    DPZ_TRY(check_mat(out, ld_out, T, D, odtype, "out"));
    if (!std::isfinite(scale))
        return fail(DPZ_ERR_INVALID_ARG, "scale = %g must be finite", scale);
    DPZ_TRY(check_blocks({mat_block("table", table, ld_table, V, D, wdtype, false),
                          vec_block("ids", ids, T * id_bytes(itype), false),
                          mat_block("out", out, ld_out, T, D, odtype, true)}));
    if (T == 0) return ok();
    cudaStream_t s = as_stream(stream);
    DPZ_TRY(launch(s, [&] {
        return launch_embedding(mat(table, ld_table, wdtype), Ids{ids, itype}, T, V, D, scale,
                                mat(out, ld_out, odtype), s);
    }));
    return ok();
}

DPZ_API size_t lm_embedding_workspace_bytes(int64_t T, int64_t V, int64_t D)
{
    if (check_rows(T, V) != DPZ_OK || check_width(D) != DPZ_OK) return 0;
    return emb_ws_layout(nullptr, T, V, D, nullptr);
}

DPZ_API int lm_embedding_grad(const void* dout, int64_t ld_dout, int ddtype, const void* ids,
                              int itype, int64_t T, float scale, const void* base,
                              int64_t ld_base, void* dtable, int64_t ld_dtable, int gdtype,
                              int64_t V, int64_t D, void* ws, void* stream)
{
    DPZ_TRY(check_rows(T, V));
    DPZ_TRY(check_width(D));
    DPZ_TRY(check_mat(dout, ld_dout, T, D, ddtype, "dout"));
    DPZ_TRY(check_ids(ids, itype, T, "ids"));
    if (base != nullptr) DPZ_TRY(check_mat(base, ld_base, V, D, gdtype, "base"));
    DPZ_TRY(check_mat(dtable, ld_dtable, V, D, gdtype, "dtable"));
    DPZ_TRY(check_addr(ws, "ws", 16));
    if (!std::isfinite(scale))
        return fail(DPZ_ERR_INVALID_ARG, "scale = %g must be finite", scale);
    EmbGrad g{mat(dout, ld_dout, ddtype), mat(base, ld_base, gdtype),
              mat(dtable, ld_dtable, gdtype), Ids{ids, itype}, T, V, D, scale, {}};
    const size_t wsb = emb_ws_layout(ws, T, V, D, &g.ws);
    const bool in_place = same_mat(base, ld_base, dtable, ld_dtable, V);
    DPZ_TRY(check_blocks({mat_block("dout", dout, ld_dout, T, D, ddtype, false),
                          vec_block("ids", ids, T * id_bytes(itype), false),
                          mat_block("base", in_place ? nullptr : base, ld_base, V, D, gdtype,
                                    false),
                          mat_block("dtable", dtable, ld_dtable, V, D, gdtype, true),
                          vec_block("ws", ws, (int64_t)wsb, true)}));
    cudaStream_t s = as_stream(stream);
    DPZ_TRY(launch(s, [&] { return launch_emb_sort(g, s); }));
    DPZ_TRY(launch(s, [&] { return launch_emb_rows(g, s); }));
    // without enough tokens for a run longer than one piece there is none to join
    if (g.ws.pieces > 0) DPZ_TRY(launch(s, [&] { return launch_emb_join(g, s); }));
    return ok();
}

DPZ_API int lm_logprobs(const void* logits, int64_t ld, int64_t T, int64_t V, int dtype,
                        float scale, const void* targets, int itype, float* logprob, float* lse,
                        float* entropy, int K, void* top_ids, float* top_logprobs, void* stream)
{
    DPZ_TRY(check_rows(T, V));
    DPZ_TRY(check_mat(logits, ld, T, V, dtype, "logits"));
    DPZ_TRY(check_factor(scale, "scale"));
    DPZ_TRY(check_ids(targets, itype, logprob ? T : 0, "targets"));
    if (targets != nullptr && logprob == nullptr && T > 0)
        return fail(DPZ_ERR_INVALID_ARG, "logprob is NULL");
    if (K < 0 || K > DPZ_LM_MAX_TOP || K > V)
        return fail(DPZ_ERR_INVALID_ARG, "K = %d is outside 0..%d or above V = %lld", K,
                    DPZ_LM_MAX_TOP, (long long)V);
    if (logprob) DPZ_TRY(check_addr(logprob, "logprob", 4));
    if (lse) DPZ_TRY(check_addr(lse, "lse", 4));
    if (entropy) DPZ_TRY(check_addr(entropy, "entropy", 4));
    if (K > 0 && T > 0) {
        DPZ_TRY(check_addr(top_ids, "top_ids", id_bytes(itype)));
        DPZ_TRY(check_addr(top_logprobs, "top_logprobs", 4));
    }
    DPZ_TRY(check_blocks({mat_block("logits", logits, ld, T, V, dtype, false),
                          vec_block("targets", targets, T * id_bytes(itype), false),
                          vec_block("logprob", logprob, T * 4, true),
                          vec_block("lse", lse, T * 4, true),
                          vec_block("entropy", entropy, T * 4, true),
                          vec_block("top_ids", top_ids, T * K * id_bytes(itype), true),
                          vec_block("top_logprobs", top_logprobs, T * K * 4, true)}));
    if (T == 0) return ok();
    const LogprobArgs a{mat(logits, ld, dtype), T, (int)V, scale, Ids{logprob ? targets : nullptr, itype},
                        logprob, lse, entropy, K, top_ids, top_logprobs};
    cudaStream_t s = as_stream(stream);
    DPZ_TRY(launch(s, [&] { return launch_logprobs(a, s); }));
    return ok();
}

DPZ_API int lm_logprobs_grad(const void* logits, int64_t ld, int64_t T, int64_t V, int dtype,
                             float scale, const void* targets, int itype, const float* lse,
                             const float* entropy, const float* dlogprob, const float* dentropy,
                             void* dlogits, int64_t ld_dlogits, void* stream)
{
    DPZ_TRY(check_rows(T, V));
    DPZ_TRY(check_mat(logits, ld, T, V, dtype, "logits"));
    DPZ_TRY(check_mat(dlogits, ld_dlogits, T, V, dtype, "dlogits"));
    DPZ_TRY(check_factor(scale, "scale"));
    DPZ_TRY(check_ids(targets, itype, T, "targets"));
    if (T > 0) {
        DPZ_TRY(check_addr(lse, "lse", 4));
        DPZ_TRY(check_addr(dlogprob, "dlogprob", 4));
        if (dentropy != nullptr) {
            DPZ_TRY(check_addr(dentropy, "dentropy", 4));
            DPZ_TRY(check_addr(entropy, "entropy", 4));
        }
    }
    const bool in_place = same_mat(logits, ld, dlogits, ld_dlogits, T);
    DPZ_TRY(check_blocks({mat_block("logits", in_place ? nullptr : logits, ld, T, V, dtype, false),
                          vec_block("targets", targets, T * id_bytes(itype), false),
                          vec_block("lse", lse, T * 4, false),
                          vec_block("entropy", dentropy ? entropy : nullptr, T * 4, false),
                          vec_block("dlogprob", dlogprob, T * 4, false),
                          vec_block("dentropy", dentropy, T * 4, false),
                          mat_block("dlogits", dlogits, ld_dlogits, T, V, dtype, true)}));
    if (T == 0) return ok();
    const LogprobGradArgs a{mat(logits, ld, dtype), mat(dlogits, ld_dlogits, dtype), T, (int)V, scale,
                            Ids{targets, itype}, lse, entropy, dlogprob, dentropy};
    cudaStream_t s = as_stream(stream);
    DPZ_TRY(launch(s, [&] { return launch_logprobs_grad(a, s); }));
    return ok();
}

// The three distillation calls: loss NULL without the forward part, dlogits
// NULL without the gradient.
static int distill_common(const void* logits, int64_t ld, int64_t T, int64_t V, int dtype,
                          const void* teacher_ids, int itype, const void* teacher_logits,
                          int tdtype, int K, float temperature, bool with_loss, float* loss,
                          float* lse, const float* lse_in, bool with_grad, const float* dloss,
                          void* dlogits, int64_t ld_dlogits, void* stream)
{
    DPZ_TRY(check_rows(T, V));
    DPZ_TRY(check_mat(logits, ld, T, V, dtype, "logits"));
    if (K < 1 || K > DPZ_LM_MAX_TEACHER)
        return fail(DPZ_ERR_INVALID_ARG, "K = %d is outside 1..%d", K, DPZ_LM_MAX_TEACHER);
    DPZ_TRY(check_factor(temperature, "temperature"));
    const float inv_tau = 1.0f / temperature;
    DPZ_TRY(check_factor(inv_tau, "1 / temperature"));
    DPZ_TRY(check_ids(teacher_ids, itype, T, "teacher_ids"));
    DPZ_TRY(check_mat(teacher_logits, K, T, K, tdtype, "teacher_logits"));
    if (T > 0) {
        if (with_loss) DPZ_TRY(check_addr(loss, "loss", 4));
        else DPZ_TRY(check_addr(lse_in, "lse", 4));
        if (lse) DPZ_TRY(check_addr(lse, "lse", 4));
        if (with_grad) DPZ_TRY(check_addr(dloss, "dloss", 4));
    }
    if (with_grad) DPZ_TRY(check_mat(dlogits, ld_dlogits, T, V, dtype, "dlogits"));
    const bool in_place = with_grad && same_mat(logits, ld, dlogits, ld_dlogits, T);
    DPZ_TRY(check_blocks(
        {mat_block("logits", in_place ? nullptr : logits, ld, T, V, dtype, false),
         vec_block("teacher_ids", teacher_ids, T * K * id_bytes(itype), false),
         vec_block("teacher_logits", teacher_logits, T * K * elem_bytes(tdtype), false),
         vec_block("lse", lse_in, T * 4, false), vec_block("dloss", dloss, T * 4, false),
         vec_block("loss", loss, T * 4, true), vec_block("lse", lse, T * 4, true),
         mat_block("dlogits", dlogits, ld_dlogits, T, V, dtype, true)}));
    if (T == 0) return ok();
    const DistillArgs a{mat(logits, ld, dtype), mat(dlogits, ld_dlogits, dtype), T, (int)V, inv_tau,
                        Ids{teacher_ids, itype}, mat(teacher_logits, K, tdtype), K, dloss, loss,
                        lse, lse_in};
    cudaStream_t s = as_stream(stream);
    DPZ_TRY(launch(s, [&] { return launch_distill(a, s); }));
    return ok();
}

DPZ_API int lm_distill(const void* logits, int64_t ld, int64_t T, int64_t V, int dtype,
                       const void* teacher_ids, int itype, const void* teacher_logits, int tdtype,
                       int K, float temperature, float* loss, float* lse, void* stream)
{
    return distill_common(logits, ld, T, V, dtype, teacher_ids, itype, teacher_logits, tdtype, K,
                          temperature, true, loss, lse, nullptr, false, nullptr, nullptr, 0,
                          stream);
}

DPZ_API int lm_distill_grad(const void* logits, int64_t ld, int64_t T, int64_t V, int dtype,
                            const void* teacher_ids, int itype, const void* teacher_logits,
                            int tdtype, int K, float temperature, const float* lse,
                            const float* dloss, void* dlogits, int64_t ld_dlogits, void* stream)
{
    return distill_common(logits, ld, T, V, dtype, teacher_ids, itype, teacher_logits, tdtype, K,
                          temperature, false, nullptr, nullptr, lse, true, dloss, dlogits,
                          ld_dlogits, stream);
}

DPZ_API int lm_distill_step(const void* logits, int64_t ld, int64_t T, int64_t V, int dtype,
                            const void* teacher_ids, int itype, const void* teacher_logits,
                            int tdtype, int K, float temperature, const float* dloss, float* loss,
                            float* lse, void* dlogits, int64_t ld_dlogits, void* stream)
{
    return distill_common(logits, ld, T, V, dtype, teacher_ids, itype, teacher_logits, tdtype, K,
                          temperature, true, loss, lse, nullptr, true, dloss, dlogits, ld_dlogits,
                          stream);
}

}  // extern "C"
