"""Thin ctypes binding of libdpz.so (include/dpz.h): argument marshalling only.

Every function of the C-ABI is exposed under its own name.  Tensor arguments
are torch CUDA tensors (device memory and streams come from PyTorch); the
computation is entirely the library's own CUDA kernels.  If libdpz.so is
missing, importing this module raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import re

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdpz.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "dpz.h")

F32, BF16, BF16_ACC32 = 0, 1, 2
I32, I64 = 16, 17
LM_MAX_TOP, LM_MAX_TEACHER = 32, 256
OK, ERR_INVALID_ARG, ERR_ALIGN, ERR_CUDA = 0, 1, 2, 3
MAX_RANKS = 64
# the per-call status word of a workspace (include/dpz.h)
WS_STATUS_OFFSET = 20
STATUS_NORM_SKIPPED, STATUS_UPDATE_SKIPPED = 1, 2


class DpzError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"dpz error {code}: {msg}")
        self.code = code


class AdamWCfg(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("step", ctypes.c_int64), ("clip_norm", ctypes.c_float),
                ("store_avg", ctypes.c_int)]


class KernelStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int64),
                ("total_ms", ctypes.c_double)]


_VP = ctypes.c_void_p
_FP = ctypes.c_void_p     # float* (device)
_L, _I, _F = ctypes.c_int64, ctypes.c_int, ctypes.c_float

_SIGS = {
    "dpz_workspace_bytes": ([ctypes.c_int64, ctypes.c_int], ctypes.c_size_t),
    "dp_reduce_scatter_avg": ([_VP, ctypes.c_int64, ctypes.c_int, ctypes.c_int, _VP], ctypes.c_int),
    "dp_allreduce_avg": ([_VP, ctypes.c_int64, ctypes.c_int, ctypes.c_int, _VP], ctypes.c_int),
    "dp_grad_global_norm": ([_VP, ctypes.c_int64, ctypes.c_int, ctypes.c_int, _VP, _FP, _VP],
                            ctypes.c_int),
    "zero1_adamw_step": ([_VP, _FP, _FP, _FP, _VP, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                          ctypes.c_int, _VP, _VP, _VP], ctypes.c_int),
    "dp_allgather": ([_VP, ctypes.c_int64, ctypes.c_int, ctypes.c_int, _VP], ctypes.c_int),
    "dp_zero1_step": ([_VP, _FP, _FP, _FP, _VP, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                       ctypes.c_int, _VP, _VP, _FP, _VP], ctypes.c_int),
    "dp_grad_global_norm_static": ([_VP, ctypes.c_int64, ctypes.c_int, ctypes.c_int, _FP, _VP],
                                   ctypes.c_int),
    "dp_reduce_scatter_avg_range": ([_VP, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                     ctypes.c_int64, ctypes.c_int64, _VP, ctypes.c_int, _VP],
                                    ctypes.c_int),
    "dp_reduce_scatter_avg_bucket": ([_VP, ctypes.c_int64, ctypes.c_int64, _VP, ctypes.c_int64,
                                      ctypes.c_int, ctypes.c_int, _VP, ctypes.c_int, _VP],
                                     ctypes.c_int),
    "dp_grad_norm_finalize": ([_VP, ctypes.c_int64, ctypes.c_int, _FP, _VP], ctypes.c_int),
    "dp_zero1_update": ([_VP, _FP, _FP, _FP, _VP, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                         ctypes.c_int, _VP, _VP, _VP], ctypes.c_int),
    "dp_zero2_update": ([_VP, _FP, _FP, _FP, _VP, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                         ctypes.c_int, _VP, _VP, _VP], ctypes.c_int),
    "lm_embedding": ([_VP, _L, _L, _L, _I, _VP, _I, _L, _F, _VP, _L, _I, _VP], _I),
    "lm_embedding_workspace_bytes": ([_L, _L, _L], ctypes.c_size_t),
    "lm_embedding_grad": ([_VP, _L, _I, _VP, _I, _L, _F, _VP, _L, _VP, _L, _I, _L, _L, _VP, _VP],
                          _I),
    "lm_logprobs": ([_VP, _L, _L, _L, _I, _F, _VP, _I, _FP, _FP, _FP, _I, _VP, _FP, _VP], _I),
    "lm_logprobs_grad": ([_VP, _L, _L, _L, _I, _F, _VP, _I, _FP, _FP, _FP, _FP, _VP, _L, _VP],
                         _I),
    "lm_distill": ([_VP, _L, _L, _L, _I, _VP, _I, _VP, _I, _I, _F, _FP, _FP, _VP], _I),
    "lm_distill_grad": ([_VP, _L, _L, _L, _I, _VP, _I, _VP, _I, _I, _F, _FP, _FP, _VP, _L, _VP],
                        _I),
    "lm_distill_step": ([_VP, _L, _L, _L, _I, _VP, _I, _VP, _I, _I, _F, _FP, _FP, _FP, _VP, _L,
                         _VP], _I),
    "dpz_last_error": ([], ctypes.c_char_p),
    "dpz_version": ([], ctypes.c_char_p),
    "dpz_launch_count": ([], ctypes.c_int64),
    "dpz_device_status": ([ctypes.POINTER(ctypes.c_int)], ctypes.c_int),
    "dpz_selftest_staged_timeout": ([ctypes.c_int, _VP, _VP], ctypes.c_int),
    "dpz_selftest_average_division": ([ctypes.c_int, _VP, _VP], ctypes.c_int),
    "dpz_profile_start": ([ctypes.c_int], ctypes.c_int),
    "dpz_profile_stop": ([ctypes.POINTER(KernelStat), ctypes.c_int,
                          ctypes.POINTER(ctypes.c_int)], ctypes.c_int),
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run gradient_reduction_zero_gb300.build.build() "
            "(there is no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    for name, (args, res) in _SIGS.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    return L


lib = _load()


def _load_call():
    """The CPython module that makes the compute calls (loaded after lib, so
    that both use the one loaded libdpz.so); lib itself where it was not
    built.  Both take the same arguments: Python ints, None for NULL."""
    try:
        from . import _dpzcall
    except ImportError:
        return lib
    return _dpzcall


_C = _load_call()


def header_symbols(path: str = HEADER) -> list[str]:
    """Names of the functions include/dpz.h declares."""
    text = open(path).read()
    return re.findall(r"DPZ_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)


def _check(rc: int) -> None:
    if rc != OK:
        raise DpzError(rc, lib.dpz_last_error().decode())


# ------------------------------------------------------------ tensor helpers

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_CODES: dict = {}


def dtype_code(t, acc32: bool = False) -> int:
    """DPZ dtype code of a tensor; acc32 selects the fp32-accumulating ring for
    a bf16 gradient arena."""
    if not _CODES:
        torch = _torch()
        _CODES.update({torch.bfloat16: BF16, torch.float32: F32})
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    if acc32:
        if code != BF16:
            raise TypeError("fp32 accumulation applies to bf16 gradient arenas")
        return BF16_ACC32
    return code


def _stream_handle(stream) -> int:
    if stream is None:
        stream = _torch().cuda.current_stream()
    return stream.cuda_stream


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def make_cfg(lr, beta1, beta2, eps, weight_decay, step, clip_norm=0.0, store_avg=False) -> AdamWCfg:
    return AdamWCfg(lr, beta1, beta2, eps, weight_decay, int(step), clip_norm, int(bool(store_avg)))


def workspace(P: int, N: int, device=None):
    """A device tensor of dpz_workspace_bytes(P, N) bytes."""
    torch = _torch()
    nb = lib.dpz_workspace_bytes(P, N)
    if nb == 0:
        raise DpzError(ERR_INVALID_ARG, f"no workspace size for P={P}, N={N}")
    return torch.empty(nb, dtype=torch.uint8, device=device or "cuda")


def _np(arena, N: int) -> int:
    n = arena.numel()
    if n % N:
        raise ValueError("arena size is not a multiple of N")
    return n // N


# ------------------------------------------------------------ the calls

def dp_reduce_scatter_avg(grads, N: int, stream=None, acc32: bool = False) -> None:
    _check(_C.dp_reduce_scatter_avg(_ptr(grads), _np(grads, N), N, dtype_code(grads, acc32),
                                     _stream_handle(stream)))


def dp_allreduce_avg(grads, N: int, stream=None, acc32: bool = False) -> None:
    _check(_C.dp_allreduce_avg(_ptr(grads), _np(grads, N), N, dtype_code(grads, acc32),
                                _stream_handle(stream)))


def dp_grad_global_norm(grads, N: int, ws, norm_out=None, stream=None) -> None:
    _check(_C.dp_grad_global_norm(_ptr(grads), _np(grads, N), N, dtype_code(grads), _ptr(ws),
                                   _ptr(norm_out), _stream_handle(stream)))


def dp_grad_global_norm_static(grads, N: int, norm_out, stream=None) -> None:
    """The global norm without a caller workspace (fixed device scratch)."""
    _check(_C.dp_grad_global_norm_static(_ptr(grads), _np(grads, N), N, dtype_code(grads),
                                          _ptr(norm_out), _stream_handle(stream)))


def zero1_adamw_step(grads, master, m, v, weights, N: int, cfg: AdamWCfg, ws=None,
                     stream=None) -> None:
    _check(_C.zero1_adamw_step(_ptr(grads), _ptr(master), _ptr(m), _ptr(v), _ptr(weights),
                                _np(grads, N), N, dtype_code(grads), dtype_code(weights),
                                ctypes.addressof(cfg), _ptr(ws), _stream_handle(stream)))


def dp_allgather(weights, N: int, stream=None) -> None:
    _check(_C.dp_allgather(_ptr(weights), _np(weights, N), N, dtype_code(weights),
                            _stream_handle(stream)))


def dp_zero1_step(grads, master, m, v, weights, N: int, cfg: AdamWCfg, ws=None, norm_out=None,
                  stream=None, acc32: bool = False) -> None:
    _check(_C.dp_zero1_step(_ptr(grads), _ptr(master), _ptr(m), _ptr(v), _ptr(weights),
                             _np(grads, N), N, dtype_code(grads, acc32), dtype_code(weights),
                             ctypes.addressof(cfg), _ptr(ws), _ptr(norm_out),
                             _stream_handle(stream)))


def dp_reduce_scatter_avg_range(grads, N: int, lo: int, n: int, ws=None, stream=None,
                                acc32: bool = False, max_ctas: int = 0) -> None:
    """max_ctas: 0 = one pass over the range; > 0 caps the kernel's blocks
    (for example one per SM) to leave the GPU to kernels on other streams."""
    _check(_C.dp_reduce_scatter_avg_range(_ptr(grads), _np(grads, N), N, dtype_code(grads, acc32),
                                           lo, n, _ptr(ws), max_ctas, _stream_handle(stream)))


def dp_reduce_scatter_avg_bucket(staging, lo: int, shards, N: int, ws=None, stream=None,
                                 acc32: bool = False, max_ctas: int = 0) -> None:
    """staging: [N*n] (rank r's values of arena elements [lo, lo+n) at r*n);
    shards: [P].  max_ctas as in dp_reduce_scatter_avg_range."""
    n = _np(staging, N)
    _check(_C.dp_reduce_scatter_avg_bucket(_ptr(staging), lo, n, _ptr(shards), shards.numel(),
                                            N, dtype_code(staging, acc32), _ptr(ws), max_ctas,
                                            _stream_handle(stream)))


def dp_grad_norm_finalize(ws, P: int, N: int, norm_out=None, stream=None) -> None:
    _check(_C.dp_grad_norm_finalize(_ptr(ws), P, N, _ptr(norm_out), _stream_handle(stream)))


def dp_zero1_update(grads, master, m, v, weights, N: int, cfg: AdamWCfg, ws=None,
                    stream=None) -> None:
    _check(_C.dp_zero1_update(_ptr(grads), _ptr(master), _ptr(m), _ptr(v), _ptr(weights),
                               _np(grads, N), N, dtype_code(grads), dtype_code(weights),
                               ctypes.addressof(cfg), _ptr(ws), _stream_handle(stream)))


def dp_zero2_update(shards, master, m, v, weights, N: int, cfg: AdamWCfg, ws=None,
                    stream=None) -> None:
    _check(_C.dp_zero2_update(_ptr(shards), _ptr(master), _ptr(m), _ptr(v), _ptr(weights),
                               shards.numel(), N, dtype_code(shards), dtype_code(weights),
                               ctypes.addressof(cfg), _ptr(ws), _stream_handle(stream)))


# ------------------------------------------------------------ vocabulary-sized ends
#
# Shapes, strides, types and devices are checked here (the C call sees
# addresses only, and launches on the current device); sizes, alignment and
# overlaps by the library.  The checks ask a tensor for few things, because on
# a small call they are most of it.

_ID_CODES: dict = {}
_float32 = None


def _dtypes() -> dict:
    """Element and id type codes by torch dtype."""
    global _float32
    if not _ID_CODES:
        torch = _torch()
        _ID_CODES.update({torch.int32: I32, torch.int64: I64})
        _CODES.update({torch.bfloat16: BF16, torch.float32: F32})
        _float32 = torch.float32
    return _CODES


# The first call of each puts torch's own function in its place.

def _current_device() -> int:
    global _current_device
    _current_device = _torch()._C._cuda_getDevice
    return _current_device()


def _raw_stream(dev: int) -> int:
    """The handle of the GPU's current stream."""
    global _raw_stream
    _raw_stream = _torch()._C._cuda_getCurrentRawStream
    return _raw_stream(dev)


def _bad_device(t, what: str) -> None:
    d = t.get_device()
    raise ValueError(f"{what} must be a CUDA tensor, not on {t.device}" if d < 0 else
                     f"{what} is on cuda:{d}, which is not the current device")


def _current_stream(dev: int, stream) -> int:
    """The handle of `stream`, or of the current stream of the GPU."""
    if stream is None:
        return _raw_stream(dev)
    if getattr(stream, "device_index", dev) != dev:
        raise ValueError(f"stream is of cuda:{stream.device_index}, the tensors are on cuda:{dev}")
    return stream.cuda_stream


def _bad_mat(t, what, dev, rows, cols):
    if t.dtype not in _dtypes():
        raise TypeError(f"{what}: unsupported dtype {t.dtype}")
    want = f" [{rows}, {cols}]" if rows >= 0 and cols >= 0 else ""
    raise ValueError(f"{what} must be a matrix{want} of unit column stride on cuda:{dev}, not "
                     f"{list(t.shape)} with strides {list(t.stride())} on {t.device}")


def _mat(t, what: str, dev: int, rows: int = -1, cols: int = -1) -> tuple:
    """(address, row stride, dtype code, rows, columns) of a 2-D matrix of unit
    column stride on GPU `dev`."""
    if not _ID_CODES:
        _dtypes()
    shape, strides = t.shape, t.stride()
    code = _CODES.get(t.dtype)
    if code is None or len(shape) != 2 or t.get_device() != dev:
        _bad_mat(t, what, dev, rows, cols)
    r, c = shape
    ld, step = strides
    if (rows >= 0 and (r != rows or c != cols)) or (step != 1 and c > 1):
        _bad_mat(t, what, dev, rows, cols)
    if r < 2 and ld < c:
        ld = c
    return t.data_ptr(), ld, code, r, c


def _dense(t, what: str, dev: int, n: int, k: int = 0, dtype=None):
    """The address of a dense tensor [n] ([n, k] with k) of fp32 (or dtype) on
    GPU `dev`; None for None."""
    if t is None:
        return None
    shape = t.shape
    want = dtype or _float32
    if t.dtype != want:
        raise TypeError(f"{what} must be {want}, not {t.dtype}")
    ok = len(shape) == 1 and shape[0] == n if not k else \
        len(shape) == 2 and shape[0] == n and shape[1] == k
    if not ok or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{what} must be a dense tensor of shape {[n, k] if k else [n]} on "
                         f"cuda:{dev}, not {list(shape)} on {t.device}")
    return t.data_ptr()


def _tokens(t, what: str, dev: int, n: int, k: int = 0) -> tuple:
    """(address, id type code) of token ids [n] or [n, k]."""
    code = _ID_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be int32 or int64, not {t.dtype}")
    return _dense(t, what, dev, n, k, t.dtype), code


def lm_embedding(table, ids, out, scale: float = 1.0, stream=None) -> None:
    """out[t] = scale * table[ids[t]] (a row of zeros where ids[t] is outside
    the table).  table [V, D] and out [T, D], bf16 or fp32 with any row
    stride; ids [T], int32 or int64."""
    dev = table.get_device()
    if dev != _current_device():     # the other tensors are compared with it
        _bad_device(table, "table")
    pt, ldt, tc, V, D = _mat(table, "table", dev)
    T = ids.numel()
    po, ldo, oc, _, _ = _mat(out, "out", dev, T, D)
    p, it = _tokens(ids, "ids", dev, T)
    _check(_C.lm_embedding(pt, ldt, V, D, tc, p, it, T, scale, po, ldo, oc,
                           _current_stream(dev, stream)))


def lm_embedding_workspace(T: int, V: int, D: int, device=None):
    """A device tensor of lm_embedding_workspace_bytes(T, V, D) bytes."""
    nb = lib.lm_embedding_workspace_bytes(T, V, D)
    if nb == 0:
        raise DpzError(ERR_INVALID_ARG, lib.dpz_last_error().decode())
    return _torch().empty(nb, dtype=_torch().uint8, device=device or "cuda")


def lm_embedding_grad(dout, ids, dtable, ws, base=None, scale: float = 1.0, stream=None) -> None:
    """dtable[v] = base[v] + scale * (sum of the rows dout[t] with ids[t] = v),
    base None: zeros; base may be dtable itself (rows of absent tokens are
    then left as they are).  dout [T, D], dtable and base [V, D]; ws:
    lm_embedding_workspace(T, V, D) or larger."""
    dev = dtable.get_device()
    if dev != _current_device():     # the other tensors are compared with it
        _bad_device(dtable, "dtable")
    pg, ldg, gc, V, D = _mat(dtable, "dtable", dev)
    T = ids.numel()
    pd, ldd, dc, _, _ = _mat(dout, "dout", dev, T, D)
    p, it = _tokens(ids, "ids", dev, T)
    pb, ldb = None, 0
    if base is not None:
        pb, ldb, bc, _, _ = _mat(base, "base", dev, V, D)
        if bc != gc:
            raise TypeError("base and dtable must have one dtype")
    need = lib.lm_embedding_workspace_bytes(T, V, D)
    if ws.get_device() != dev or not ws.is_contiguous() or ws.nbytes < need:
        raise ValueError(f"ws must be a dense tensor of at least {need} bytes on cuda:{dev}")
    _check(_C.lm_embedding_grad(pd, ldd, dc, p, it, T, scale, pb, ldb, pg, ldg, gc, V, D,
                                ws.data_ptr(), _current_stream(dev, stream)))


def lm_logprobs(logits, targets=None, logprob=None, lse=None, entropy=None, top_ids=None,
                top_logprobs=None, scale: float = 1.0, stream=None) -> None:
    """Log probabilities of `targets` [T] under softmax(scale * logits), into
    logprob [T] (both or neither); lse [T], entropy [T], and the K largest
    logits' ids (of targets' dtype, if given) and log probabilities, top_ids and
    top_logprobs [T, K], where given.  logits [T, V], bf16 or fp32 with any row
    stride."""
    dev = logits.get_device()
    if dev != _current_device():     # the other tensors are compared with it
        _bad_device(logits, "logits")
    px, ld, xc, T, V = _mat(logits, "logits", dev)
    if (targets is None) != (logprob is None):
        raise ValueError("targets and logprob come together")
    K, p, pt, pl, it = 0, None, None, None, I64
    if targets is not None:
        p, it = _tokens(targets, "targets", dev, T)
    if top_ids is not None:
        if top_ids.dim() != 2 or top_logprobs is None:
            raise ValueError("top_ids must be [T, K] and come with top_logprobs")
        K = top_ids.shape[1]
        if K > 0:
            pt, kt = _tokens(top_ids, "top_ids", dev, T, K)
            if targets is not None and kt != it:
                raise TypeError("targets and top_ids must have one dtype")
            it = kt
            pl = _dense(top_logprobs, "top_logprobs", dev, T, K)
        elif tuple(top_ids.shape) != (T, 0) or tuple(top_logprobs.shape) != (T, 0):
            raise ValueError(f"top_ids and top_logprobs must be [{T}, K]")
    elif top_logprobs is not None:
        raise ValueError("top_logprobs comes with top_ids")
    _check(_C.lm_logprobs(px, ld, T, V, xc, scale, p, it, _dense(logprob, "logprob", dev, T),
                          _dense(lse, "lse", dev, T), _dense(entropy, "entropy", dev, T), K, pt, pl,
                          _current_stream(dev, stream)))


def lm_logprobs_grad(logits, targets, lse, dlogprob, dlogits, entropy=None, dentropy=None,
                     scale: float = 1.0, stream=None) -> None:
    """The gradient of lm_logprobs' logprob (weighted by dlogprob [T]) and
    entropy (by dentropy [T], with the entropy it gave) with respect to the
    logits, into dlogits, which may be logits itself."""
    dev = logits.get_device()
    if dev != _current_device():     # the other tensors are compared with it
        _bad_device(logits, "logits")
    px, ld, xc, T, V = _mat(logits, "logits", dev)
    pd, ldd, dc, _, _ = _mat(dlogits, "dlogits", dev, T, V)
    if dc != xc:
        raise TypeError("logits and dlogits must have one dtype")
    p, it = _tokens(targets, "targets", dev, T)
    _check(_C.lm_logprobs_grad(px, ld, T, V, xc, scale, p, it, _dense(lse, "lse", dev, T),
                               _dense(entropy, "entropy", dev, T),
                               _dense(dlogprob, "dlogprob", dev, T),
                               _dense(dentropy, "dentropy", dev, T), pd, ldd,
                               _current_stream(dev, stream)))


def _distill_args(logits, teacher_ids, teacher_logits, temperature) -> tuple:
    """The GPU and the arguments that the three calls have in common."""
    dev = logits.get_device()
    if dev != _current_device():     # the other tensors are compared with it
        _bad_device(logits, "logits")
    px, ld, xc, T, V = _mat(logits, "logits", dev)
    if teacher_ids.dim() != 2:
        raise ValueError(f"teacher_ids must be [T, K], not {list(teacher_ids.shape)}")
    K = teacher_ids.shape[1]
    if K == 0:
        raise ValueError("teacher_ids must have at least one column")
    p, it = _tokens(teacher_ids, "teacher_ids", dev, T, K)
    tc = _CODES.get(teacher_logits.dtype)
    if tc is None:
        raise TypeError(f"teacher_logits: unsupported dtype {teacher_logits.dtype}")
    return dev, (px, ld, T, V, xc, p, it,
                 _dense(teacher_logits, "teacher_logits", dev, T, K, teacher_logits.dtype), tc,
                 K, temperature)


def lm_distill(logits, teacher_ids, teacher_logits, loss, lse=None, temperature: float = 1.0,
               stream=None) -> None:
    """Per-row distillation loss from a teacher's top logits: teacher_ids
    [T, K] (int32 or int64) and teacher_logits [T, K] (bf16 or fp32), softmax
    over the K entries at the given temperature, against softmax(logits /
    temperature) over the whole vocabulary.  loss and lse: [T]."""
    dev, args = _distill_args(logits, teacher_ids, teacher_logits, temperature)
    T = args[2]
    _check(_C.lm_distill(*args, _dense(loss, "loss", dev, T), _dense(lse, "lse", dev, T),
                         _current_stream(dev, stream)))


def lm_distill_grad(logits, teacher_ids, teacher_logits, lse, dloss, dlogits,
                    temperature: float = 1.0, stream=None) -> None:
    """The gradient of sum(dloss * loss) of lm_distill with respect to the
    logits, from its lse, into dlogits, which may be logits itself."""
    dev, args = _distill_args(logits, teacher_ids, teacher_logits, temperature)
    T, V = args[2], args[3]
    pd, ldd, dc, _, _ = _mat(dlogits, "dlogits", dev, T, V)
    if dc != args[4]:
        raise TypeError("logits and dlogits must have one dtype")
    _check(_C.lm_distill_grad(*args, _dense(lse, "lse", dev, T),
                              _dense(dloss, "dloss", dev, T), pd, ldd,
                              _current_stream(dev, stream)))


def lm_distill_step(logits, teacher_ids, teacher_logits, dloss, loss, dlogits, lse=None,
                    temperature: float = 1.0, stream=None) -> None:
    """lm_distill and lm_distill_grad in one pass over the logits, for weights
    dloss [T] known beforehand; dlogits may be logits itself."""
    dev, args = _distill_args(logits, teacher_ids, teacher_logits, temperature)
    T, V = args[2], args[3]
    pd, ldd, dc, _, _ = _mat(dlogits, "dlogits", dev, T, V)
    if dc != args[4]:
        raise TypeError("logits and dlogits must have one dtype")
    _check(_C.lm_distill_step(*args, _dense(dloss, "dloss", dev, T), _dense(loss, "loss", dev, T),
                              _dense(lse, "lse", dev, T), pd, ldd, _current_stream(dev, stream)))


class PreparedCall:
    """One C-ABI call whose arguments were marshalled once: calling it makes
    the same call again (the library validates the arguments and launches its
    kernels every time).  For a training loop that runs the same step on the
    same buffers, this leaves out the per-call Python work of turning tensors
    into pointers and dtype codes.  It keeps the tensors and the AdamW
    settings alive; changing a cfg field after preparing changes the calls."""
    __slots__ = ("_fn", "_args", "_keep")

    def __init__(self, fn, args, keep):
        self._fn = fn
        self._args = tuple(args)
        self._keep = keep

    def __call__(self) -> None:
        rc = self._fn(*self._args)
        if rc != OK:
            _check(rc)


def _prepare(name: str, args: tuple, keep) -> PreparedCall:
    """A PreparedCall of the compute call `name` with `args` (Python ints,
    None for NULL).  Through ctypes they are converted here, once."""
    fn = getattr(_C, name)
    if _C is lib:
        args = tuple(t(v) for t, v in zip(fn.argtypes, args))
    return PreparedCall(fn, args, keep)


def prepare_zero1_step(grads, master, m, v, weights, N: int, cfg: AdamWCfg, ws=None,
                       norm_out=None, stream=None, acc32: bool = False) -> PreparedCall:
    """dp_zero1_step with its arguments marshalled once (PreparedCall)."""
    args = (_ptr(grads), _ptr(master), _ptr(m), _ptr(v), _ptr(weights), _np(grads, N), N,
            dtype_code(grads, acc32), dtype_code(weights), ctypes.addressof(cfg), _ptr(ws),
            _ptr(norm_out), _stream_handle(stream))
    return _prepare("dp_zero1_step", args, (grads, master, m, v, weights, cfg, ws, norm_out))


def prepare_allreduce_avg(grads, N: int, stream=None, acc32: bool = False) -> PreparedCall:
    """dp_allreduce_avg with its arguments marshalled once (PreparedCall)."""
    args = (_ptr(grads), _np(grads, N), N, dtype_code(grads, acc32), _stream_handle(stream))
    return _prepare("dp_allreduce_avg", args, (grads,))


def launch_count() -> int:
    return int(lib.dpz_launch_count())


def device_status() -> int:
    """The device error flag (1 if a kernel's bounded wait on its own copies
    ran out since the last call), read and cleared."""
    f = ctypes.c_int()
    _check(lib.dpz_device_status(ctypes.byref(f)))
    return f.value


def ws_status(ws) -> int:
    """The DPZ_STATUS_* bits of a workspace tensor's status word (a read of
    device memory; it synchronises with the current stream)."""
    return int(ws[WS_STATUS_OFFSET:WS_STATUS_OFFSET + 4].view(_torch().int32).item())


SELFTEST_BUF_BYTES = 4096
SELFTEST_UPDATE, SELFTEST_NORM, SELFTEST_STEP = 0, 1, 2
# offsets in the self-test buffer (include/dpz.h)
SELFTEST_NORM_OUT, SELFTEST_GRADS = 2560, 2816


def selftest_staged_timeout(kernel: int, buf, stream=None) -> None:
    """Launch one staged kernel (SELFTEST_*) on the one-tile arena laid out in
    `buf` (a 256-byte aligned device tensor of at least SELFTEST_BUF_BYTES
    bytes) with a barrier that never completes and a short wait bound, so
    that the kernel gives up on its tile and reports it."""
    if buf.numel() * buf.element_size() < SELFTEST_BUF_BYTES:
        raise ValueError(f"buf must hold at least {SELFTEST_BUF_BYTES} bytes")
    _check(lib.dpz_selftest_staged_timeout(int(kernel), _ptr(buf), _stream_handle(stream)))


def selftest_average_division(N: int, counter, stream=None) -> None:
    """Count, into `counter` (a device int64 tensor of one element), the
    float inputs whose average division by N differs bit for bit from an
    IEEE division, over all 2^32 bit patterns; 0 means correctly rounded."""
    if counter.numel() != 1 or counter.element_size() != 8:
        raise ValueError("counter must be a one-element 8-byte tensor")
    _check(lib.dpz_selftest_average_division(int(N), _ptr(counter), _stream_handle(stream)))


def version() -> str:
    return lib.dpz_version().decode()


def profile_start(max_launches: int = 4096) -> None:
    _check(lib.dpz_profile_start(max_launches))


def profile_stop() -> dict:
    """{kernel name: (launches, total_ms)} for the launches since profile_start."""
    stats = (KernelStat * 64)()
    n = ctypes.c_int()
    _check(lib.dpz_profile_stop(stats, 64, ctypes.byref(n)))
    return {stats[i].name.decode(): (int(stats[i].launches), float(stats[i].total_ms))
            for i in range(min(n.value, 64))}
