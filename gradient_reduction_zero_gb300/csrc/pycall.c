/* CPython entry points for the compute calls of libdpz.so (include/dpz.h).
 *
 * Each function takes the C call's arguments as Python ints in the same order
 * (device addresses, sizes, dtype codes, the address of a dpz_adamw_cfg, the
 * stream handle; None for a NULL pointer), converts each once and makes the
 * call.  It returns the call's status code.  Nothing else happens here: the
 * checks, the error message and the launches are the library's.  The point is
 * the cost of a call from Python, which for the launch-bound workloads is most
 * of a step: a vectorcall with a fixed argument list instead of ctypes'
 * per-argument conversion objects.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits.h>
#include <stdint.h>
#include <string.h>

#include "dpz.h"

typedef union {
    void* p;
    int64_t l;
    int i;
    float f;
} Arg;

/* fmt: one character per argument, 'p' pointer (int or None), 'l' int64,
 * 'i' int, 'f' float.  Sets a Python exception and returns -1 on a bad argument. */
static int parse(PyObject* const* a, Py_ssize_t n, const char* fmt, Arg* out)
{
    const Py_ssize_t k = (Py_ssize_t)strlen(fmt);
    if (n != k) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", k, n);
        return -1;
    }
    for (Py_ssize_t j = 0; j < k; ++j) {
        PyObject* o = a[j];
        if (fmt[j] == 'p') {
            if (o == Py_None) {
                out[j].p = NULL;
                continue;
            }
            out[j].p = PyLong_AsVoidPtr(o);
            if (out[j].p == NULL && PyErr_Occurred()) return -1;
        } else if (fmt[j] == 'l') {
            const long long v = PyLong_AsLongLong(o);
            if (v == -1 && PyErr_Occurred()) return -1;
            out[j].l = (int64_t)v;
        } else if (fmt[j] == 'f') {
            const double v = PyFloat_AsDouble(o);
            if (v == -1.0 && PyErr_Occurred()) return -1;
            out[j].f = (float)v;
        } else {
            const long v = PyLong_AsLong(o);
            if (v == -1 && PyErr_Occurred()) return -1;
            if (v < INT_MIN || v > INT_MAX) {
                PyErr_SetString(PyExc_OverflowError, "argument does not fit a C int");
                return -1;
            }
            out[j].i = (int)v;
        }
    }
    return 0;
}

#define CALL(name, fmt, nargs, expr)                                             \
    static PyObject* py_##name(PyObject* self, PyObject* const* a, Py_ssize_t n) \
    {                                                                            \
        (void)self;                                                              \
        Arg s[nargs];                                                            \
        if (parse(a, n, fmt, s)) return NULL;                                    \
        return PyLong_FromLong((long)(expr));                                    \
    }

#define F(k) ((float*)s[k].p)
#define CFG(k) ((const dpz_adamw_cfg*)s[k].p)

CALL(dp_reduce_scatter_avg, "pliip", 5, dp_reduce_scatter_avg(s[0].p, s[1].l, s[2].i, s[3].i, s[4].p))
CALL(dp_allreduce_avg, "pliip", 5, dp_allreduce_avg(s[0].p, s[1].l, s[2].i, s[3].i, s[4].p))
CALL(dp_grad_global_norm, "pliippp", 7,
     dp_grad_global_norm(s[0].p, s[1].l, s[2].i, s[3].i, s[4].p, F(5), s[6].p))
CALL(dp_grad_global_norm_static, "pliipp", 6,
     dp_grad_global_norm_static(s[0].p, s[1].l, s[2].i, s[3].i, F(4), s[5].p))
CALL(zero1_adamw_step, "pppppliiippp", 12,
     zero1_adamw_step(s[0].p, F(1), F(2), F(3), s[4].p, s[5].l, s[6].i, s[7].i, s[8].i, CFG(9),
                      s[10].p, s[11].p))
CALL(dp_allgather, "pliip", 5, dp_allgather(s[0].p, s[1].l, s[2].i, s[3].i, s[4].p))
CALL(dp_zero1_step, "pppppliiipppp", 13,
     dp_zero1_step(s[0].p, F(1), F(2), F(3), s[4].p, s[5].l, s[6].i, s[7].i, s[8].i, CFG(9),
                   s[10].p, F(11), s[12].p))
CALL(dp_reduce_scatter_avg_range, "pliillpip", 9,
     dp_reduce_scatter_avg_range(s[0].p, s[1].l, s[2].i, s[3].i, s[4].l, s[5].l, s[6].p, s[7].i,
                                 s[8].p))
CALL(dp_reduce_scatter_avg_bucket, "pllpliipip", 10,
     dp_reduce_scatter_avg_bucket(s[0].p, s[1].l, s[2].l, s[3].p, s[4].l, s[5].i, s[6].i, s[7].p,
                                  s[8].i, s[9].p))
CALL(dp_grad_norm_finalize, "plipp", 5, dp_grad_norm_finalize(s[0].p, s[1].l, s[2].i, F(3), s[4].p))
CALL(dp_zero1_update, "pppppliiippp", 12,
     dp_zero1_update(s[0].p, F(1), F(2), F(3), s[4].p, s[5].l, s[6].i, s[7].i, s[8].i, CFG(9),
                     s[10].p, s[11].p))
CALL(dp_zero2_update, "pppppliiippp", 12,
     dp_zero2_update(s[0].p, F(1), F(2), F(3), s[4].p, s[5].l, s[6].i, s[7].i, s[8].i, CFG(9),
                     s[10].p, s[11].p))
CALL(lm_embedding, "plllipilfplip", 13,
     lm_embedding(s[0].p, s[1].l, s[2].l, s[3].l, s[4].i, s[5].p, s[6].i, s[7].l, s[8].f, s[9].p,
                  s[10].l, s[11].i, s[12].p))
CALL(lm_embedding_grad, "plipilfplplillpp", 16,
     lm_embedding_grad(s[0].p, s[1].l, s[2].i, s[3].p, s[4].i, s[5].l, s[6].f, s[7].p, s[8].l,
                       s[9].p, s[10].l, s[11].i, s[12].l, s[13].l, s[14].p, s[15].p))
CALL(lm_logprobs, "plllifpipppippp", 15,
     lm_logprobs(s[0].p, s[1].l, s[2].l, s[3].l, s[4].i, s[5].f, s[6].p, s[7].i, F(8), F(9), F(10),
                 s[11].i, s[12].p, F(13), s[14].p))
CALL(lm_logprobs_grad, "plllifpippppplp", 15,
     lm_logprobs_grad(s[0].p, s[1].l, s[2].l, s[3].l, s[4].i, s[5].f, s[6].p, s[7].i, F(8), F(9),
                      F(10), F(11), s[12].p, s[13].l, s[14].p))
CALL(lm_distill, "plllipipiifppp", 14,
     lm_distill(s[0].p, s[1].l, s[2].l, s[3].l, s[4].i, s[5].p, s[6].i, s[7].p, s[8].i, s[9].i,
                s[10].f, F(11), F(12), s[13].p))
CALL(lm_distill_grad, "plllipipiifppplp", 16,
     lm_distill_grad(s[0].p, s[1].l, s[2].l, s[3].l, s[4].i, s[5].p, s[6].i, s[7].p, s[8].i,
                     s[9].i, s[10].f, F(11), F(12), s[13].p, s[14].l, s[15].p))
CALL(lm_distill_step, "plllipipiifpppplp", 17,
     lm_distill_step(s[0].p, s[1].l, s[2].l, s[3].l, s[4].i, s[5].p, s[6].i, s[7].p, s[8].i,
                     s[9].i, s[10].f, F(11), F(12), F(13), s[14].p, s[15].l, s[16].p))

#define HEADS(k) ((const dpz_heads*)s[k].p)

CALL(attn_qk_norm_rope, "ppllllippifpiplippp", 19,
     attn_qk_norm_rope(HEADS(0), HEADS(1), s[2].l, s[3].l, s[4].l, s[5].l, s[6].i, s[7].p, s[8].p,
                       s[9].i, s[10].f, s[11].p, s[12].i, F(13), s[14].l, s[15].i, HEADS(16),
                       HEADS(17), s[18].p))
CALL(attn_qk_norm_rope_grad, "ppppllllippifpiplipppppp", 24,
     attn_qk_norm_rope_grad(HEADS(0), HEADS(1), HEADS(2), HEADS(3), s[4].l, s[5].l, s[6].l, s[7].l,
                            s[8].i, s[9].p, s[10].p, s[11].i, s[12].f, s[13].p, s[14].i, F(15),
                            s[16].l, s[17].i, HEADS(18), HEADS(19), s[20].p, s[21].p, s[22].p,
                            s[23].p))
CALL(attn_forward, "ppplllllilppiifppp", 18,
     attn_forward(HEADS(0), HEADS(1), HEADS(2), s[3].l, s[4].l, s[5].l, s[6].l, s[7].l, s[8].i,
                  s[9].l, s[10].p, s[11].p, s[12].i, s[13].i, s[14].f, HEADS(15), F(16), s[17].p))
CALL(attn_grad, "pppppplllllilppiifppppp", 23,
     attn_grad(HEADS(0), HEADS(1), HEADS(2), HEADS(3), F(4), HEADS(5), s[6].l, s[7].l, s[8].l,
               s[9].l, s[10].l, s[11].i, s[12].l, s[13].p, s[14].p, s[15].i, s[16].i, s[17].f,
               HEADS(18), HEADS(19), HEADS(20), s[21].p, s[22].p))
CALL(tensors_norm, "pippp", 5,
     tensors_norm((const dpz_tensor*)s[0].p, s[1].i, F(2), s[3].p, s[4].p))
CALL(tensors_clip, "ppipfp", 6,
     tensors_clip((const dpz_tensor*)s[0].p, (const dpz_tensor*)s[1].p, s[2].i, F(3), s[4].f,
                     s[5].p))

#define ENTRY(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, NULL}

static PyMethodDef methods[] = {
    ENTRY(dp_reduce_scatter_avg),
    ENTRY(dp_allreduce_avg),
    ENTRY(dp_grad_global_norm),
    ENTRY(dp_grad_global_norm_static),
    ENTRY(zero1_adamw_step),
    ENTRY(dp_allgather),
    ENTRY(dp_zero1_step),
    ENTRY(dp_reduce_scatter_avg_range),
    ENTRY(dp_reduce_scatter_avg_bucket),
    ENTRY(dp_grad_norm_finalize),
    ENTRY(dp_zero1_update),
    ENTRY(dp_zero2_update),
    ENTRY(lm_embedding),
    ENTRY(lm_embedding_grad),
    ENTRY(lm_logprobs),
    ENTRY(lm_logprobs_grad),
    ENTRY(lm_distill),
    ENTRY(lm_distill_grad),
    ENTRY(lm_distill_step),
    ENTRY(attn_qk_norm_rope),
    ENTRY(attn_qk_norm_rope_grad),
    ENTRY(attn_forward),
    ENTRY(attn_grad),
    ENTRY(tensors_norm),
    ENTRY(tensors_clip),
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {
    PyModuleDef_HEAD_INIT, "_dpzcall",
    "The compute calls of libdpz.so, with Python ints for arguments.", -1, methods,
    NULL, NULL, NULL, NULL,
};

PyMODINIT_FUNC PyInit__dpzcall(void) { return PyModule_Create(&module); }
