"""Binding of libobadam.so: the C-ABI entry points under the same names, by ctypes, and the calls over lists of
tensors by the compiled module _obtorch (csrc/ob_torch.cpp).

Argument marshalling only: torch tensors are turned into device pointers (``data_ptr()``) and torch's
current HIP stream; every step of the optimizer runs in the library's HIP kernels.  There is no
fallback: if the library is not built, or a tensor is not on the GPU, a call raises.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libobadam.so")

OB_OK, OB_ERR_ARG, OB_ERR_ALIGN, OB_ERR_DTYPE, OB_ERR_HIP, OB_ERR_OOM, OB_ERR_SIZE = range(7)
OB_NOALLOC_SCRATCH_BYTES = 64 << 20
OB_F32, OB_BF16, OB_F16 = 0, 1, 2
OB_EF_PLAIN, OB_EF_EMA = 0, 1
OB_ROUND_NEAREST, OB_ROUND_STOCHASTIC = 0, 1
OB_NORM_2, OB_NORM_MAX = 0, 1
OB_MUON_PLAIN, OB_MUON_SHAPE, OB_MUON_MATCH_RMS = 0, 1, 2
OB_STATE_BLOCK = 256
OB_CONTROL_PARTIALS = 2048
OB_CONTROL_BYTES = 64 + 8 * OB_CONTROL_PARTIALS
(OB_KERNEL_CHUNK_SUMSQ, OB_KERNEL_COMPRESS, OB_KERNEL_DENSE, OB_KERNEL_SERVER_SUMSQ,
 OB_KERNEL_SERVER_APPLY, OB_KERNEL_UNPACK, OB_KERNEL_TRUST_RATIO, OB_KERNEL_LAMB_APPLY,
 OB_KERNEL_DIAG, OB_KERNEL_SCALE, OB_KERNEL_WORKER_COMPRESS, OB_KERNEL_WORKER_UPDATE) = range(12)
KERNEL_NAMES = {
    OB_KERNEL_CHUNK_SUMSQ: "chunk_sumsq", OB_KERNEL_COMPRESS: "compress", OB_KERNEL_DENSE: "dense",
    OB_KERNEL_SERVER_SUMSQ: "server_sumsq", OB_KERNEL_SERVER_APPLY: "server_apply",
    OB_KERNEL_UNPACK: "unpack", OB_KERNEL_TRUST_RATIO: "trust_ratio", OB_KERNEL_LAMB_APPLY: "lamb_apply",
    OB_KERNEL_DIAG: "diag", OB_KERNEL_SCALE: "scale", OB_KERNEL_WORKER_COMPRESS: "worker_compress",
    OB_KERNEL_WORKER_UPDATE: "worker_update",
}


class ObError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {ob_status_str(status)} (status {status})")


class ob_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("clip", ctypes.c_float), ("ef_mode", ctypes.c_int32),
                ("ef_beta", ctypes.c_float), ("bias_correction", ctypes.c_int32),
                ("step", ctypes.c_int64), ("err_rounding", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("sr_seed", ctypes.c_uint64)]


def hparams(lr=1e-4, beta1=0.9, beta2=0.999, eps=1e-8, clip=0.0, ef_mode=OB_EF_PLAIN, ef_beta=0.9,
            bias_correction=False, step=0, err_rounding=OB_ROUND_NEAREST, sr_seed=0) -> ob_hparams:
    return ob_hparams(lr, beta1, beta2, eps, clip, ef_mode, ef_beta, 1 if bias_correction else 0, step,
                      err_rounding, 0, sr_seed)


class ob_adamw_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float), ("bias_correction", ctypes.c_int32),
                ("step", ctypes.c_int64), ("rounding", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("sr_seed", ctypes.c_uint64)]


def adamw_hparams(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, bias_correction=True, step=1,
                  rounding=OB_ROUND_NEAREST, sr_seed=0) -> ob_adamw_hparams:
    return ob_adamw_hparams(lr, beta1, beta2, eps, weight_decay, 1 if bias_correction else 0, step, rounding, 0,
                            sr_seed)


class ob_muon_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float), ("weight_decay", ctypes.c_float), ("eps", ctypes.c_float),
                ("nesterov", ctypes.c_int32), ("iterations", ctypes.c_int32), ("scale", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


def muon_hparams(lr=1e-3, momentum=0.95, weight_decay=0.1, eps=1e-7, nesterov=True, iterations=5,
                 scale=OB_MUON_MATCH_RMS) -> ob_muon_hparams:
    return ob_muon_hparams(lr, momentum, weight_decay, eps, 1 if nesterov else 0, iterations, scale, 0)


class ob_product(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("m", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("a", ctypes.c_void_p), ("a_row", ctypes.c_int64), ("a_col", ctypes.c_int64), ("a_batch", ctypes.c_int64),
                ("b", ctypes.c_void_p), ("b_row", ctypes.c_int64), ("b_col", ctypes.c_int64), ("b_batch", ctypes.c_int64),
                ("c", ctypes.c_void_p), ("c_row", ctypes.c_int64), ("c_batch", ctypes.c_int64),
                ("d", ctypes.c_void_p), ("d_row", ctypes.c_int64), ("d_batch", ctypes.c_int64),
                ("in_type", ctypes.c_int32), ("out_type", ctypes.c_int32), ("alpha", ctypes.c_float),
                ("beta", ctypes.c_float), ("symmetric", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("workspace", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libobadam.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                           "(there is no non-HIP fallback)")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    HP = ctypes.POINTER(ob_hparams)
    sig = {
        "ob_plan_create": (I32, [I64, I64, P, I64, ctypes.POINTER(P)]),
        "ob_plan_destroy": (I32, [P]),
        "ob_plan_num_elements": (I64, [P]),
        "ob_plan_num_chunks": (I64, [P]),
        "ob_plan_num_blocks": (I64, [P]),
        "ob_plan_block_elems": (I64, [P]),
        "ob_plan_num_groups": (I64, [P, I32, I32, I32]),
        "ob_adam_warmup_step": (I32, [P, P, I32, P, P, P, HP, P]),
        "ob_adam_compress_step": (I32, [P, P, I32, P, I32, P, P, P, P, P, P, P, HP, P]),
        "ob_adam_compress_step_noalloc": (I32, [I64, I64, P, I32, P, I32, P, P, P, P, P, P, P, HP, P]),
        "ob_lamb_compress_step": (I32, [P, P, I32, P, I32, P, P, P, P, P, P, P, P, HP, P]),
        "ob_lamb_warmup_step": (I32, [P, P, I32, P, P, P, P, HP, P]),
        "ob_adam_worker_compress": (I32, [P, P, I32, P, I32, P, P, P, P, HP, P]),
        "ob_adam_worker_update": (I32, [P, P, P, P, P, P, HP, P]),
        "ob_lamb_worker_update": (I32, [P, P, P, P, P, P, P, HP, P]),
        "ob_server_reduce": (I32, [P, I32, P, P, P, P, P, P]),
        "ob_pack": (I32, [P, I32, I64, P, P]),
        "ob_unpack": (I32, [P, P, I64, P, P, P]),
        "ob_status_str": (ctypes.c_char_p, [I32]),
        "ob_plan_set_timing": (I32, [P, I32]),
        "ob_plan_set_diagnostics": (I32, [P, P, P]),
        "ob_plan_set_guard": (I32, [P, P]),
        "ob_plan_read_timing": (I32, [P, I32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(I64)]),
        "ob_tensors_create": (I32, [I64, P, P, P, P, P, ctypes.POINTER(P)]),
        "ob_tensors_destroy": (I32, [P]),
        "ob_tensors_count": (I64, [P]),
        "ob_tensors_num_elements": (I64, [P]),
        "ob_tensors_state_elems": (I64, [P]),
        "ob_tensors_state_offset": (I64, [P, I64]),
        "ob_grad_norm": (I32, [P, P, ctypes.c_float, ctypes.c_float, ctypes.POINTER(ob_adamw_hparams), P, P]),
        "ob_adamw_step": (I32, [P, P, P, P, P, P, ctypes.POINTER(ob_adamw_hparams), P, P]),
        "ob_adamw8_step": (I32, [P, P, P, P, P, P, P, P, ctypes.POINTER(ob_adamw_hparams), P, P]),
        "ob_adamw_check": (I32, [P, P, P, P, P, P, ctypes.POINTER(ob_adamw_hparams), P]),
        "ob_adamw8_check": (I32, [P, P, P, P, P, P, P, P, ctypes.POINTER(ob_adamw_hparams), P]),
        "ob_state8_encode": (I32, [I64, P, P, P, P, P, P, P]),
        "ob_state8_decode": (I32, [I64, P, P, P, P, P, P, P]),
        "ob_tensor_norms_workspace": (I64, [P]),
        "ob_tensor_norms": (I32, [P, P, ctypes.c_float, I32, P, P, P]),
        "ob_clip_grads": (I32, [P, P, P, P, ctypes.c_float, ctypes.c_float, I32, P]),
        "ob_muon_create": (I32, [P, P, P, ctypes.POINTER(P)]),
        "ob_muon_destroy": (I32, [P]),
        "ob_muon_workspace": (I64, [P]),
        "ob_muon_step": (I32, [P, P, P, P, P, P, ctypes.POINTER(ob_muon_hparams), P, P]),
        "ob_muon_check": (I32, [P, P, P, P, P, P, ctypes.POINTER(ob_muon_hparams), P]),
        "ob_matmul": (I32, [ctypes.POINTER(ob_product), P]),
        "ob_matmul_workspace": (I64, [ctypes.POINTER(ob_product)]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


_torch_module = None


def _obtorch():
    """Load the _obtorch module (raises if it has not been built)."""
    global _torch_module
    if _torch_module is None:
        lib()   # the library that the module links to
        if not os.path.exists(os.path.join(_PKG, "_obtorch.so")):
            raise RuntimeError(f"{_PKG}/_obtorch.so is missing: build it with __graft_entry__.build()")
        from . import _obtorch as module
        _torch_module = module
    return _torch_module


def ob_status_str(status: int) -> str:
    return lib().ob_status_str(status).decode()


def _check(status: int, what: str):
    if status != OB_OK:
        raise ObError(status, what)


def _dev(t: torch.Tensor | None, name: str):
    """Device pointer of a contiguous GPU tensor (None -> NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on the GPU (got {t.device}); there is no CPU path")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _want(t, name, dtype, numel=None):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")


def _gdtype(g: torch.Tensor) -> int:
    if g.dtype == torch.float32:
        return OB_F32
    if g.dtype == torch.bfloat16:
        return OB_BF16
    raise TypeError(f"gradient dtype must be float32 or bfloat16, got {g.dtype}")


_ERR_DTYPES = {torch.float32: OB_F32, torch.bfloat16: OB_BF16, torch.float16: OB_F16}


def _errdtype(err: torch.Tensor) -> int:
    if err.dtype not in _ERR_DTYPES:
        raise TypeError(f"error buffer dtype must be float32, bfloat16 or float16, got {err.dtype}")
    return _ERR_DTYPES[err.dtype]


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


class Plan:
    """Owner of an ob_plan handle (destroyed with the object)."""

    def __init__(self, handle: ctypes.c_void_p, n: int):
        self.handle = handle
        self.n = n

    @property
    def num_chunks(self) -> int:
        return int(lib().ob_plan_num_chunks(self.handle))

    @property
    def num_blocks(self) -> int:
        return int(lib().ob_plan_num_blocks(self.handle))

    @property
    def block_elems(self) -> int:
        return int(lib().ob_plan_block_elems(self.handle))

    def num_groups(self, g_dtype: int, err_dtype: int = OB_F32, lamb: bool = False) -> int:
        """Launches of each of the compressed step's two kernels per step (its chunk groups)."""
        return int(lib().ob_plan_num_groups(self.handle, g_dtype, err_dtype, 1 if lamb else 0))

    def destroy(self):
        if self.handle:
            _check(lib().ob_plan_destroy(self.handle), "ob_plan_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def ob_plan_create(n: int, chunk_size: int = 0, chunk_offsets=None) -> Plan:
    """Plan over n elements: uniform chunks of chunk_size, or per-tensor chunk_offsets (K+1 ints)."""
    h = ctypes.c_void_p()
    if chunk_offsets is not None:
        offs = (ctypes.c_int64 * len(chunk_offsets))(*[int(o) for o in chunk_offsets])
        st = lib().ob_plan_create(n, 0, offs, len(chunk_offsets) - 1, ctypes.byref(h))
    else:
        st = lib().ob_plan_create(n, chunk_size, None, 0, ctypes.byref(h))
    _check(st, "ob_plan_create")
    return Plan(h, n)


def ob_adam_warmup_step(plan: Plan, g, m, v, p, hp: ob_hparams, stream=None):
    n = plan.n
    _want(g, "g", g.dtype, n)
    for name, t in (("m", m), ("v", v), ("p", p)):
        _want(t, name, torch.float32, n)
    _check(lib().ob_adam_warmup_step(plan.handle, _dev(g, "g"), _gdtype(g), _dev(m, "m"), _dev(v, "v"),
                                     _dev(p, "p"), ctypes.byref(hp), _stream(stream)),
           "ob_adam_warmup_step")


def ob_adam_compress_step(plan: Plan, g, err, m, v, p, words_out, scales_out, hp: ob_hparams,
                          signs_out=None, nonfinite_out=None, stream=None):
    n = plan.n
    _want(g, "g", g.dtype, n)
    _want(err, "err", err.dtype, n)
    for name, t in (("m", m), ("v", v), ("p", p)):
        _want(t, name, torch.float32, n)
    _want(words_out, "words_out", torch.int32, (n + 31) // 32)
    _want(scales_out, "scales_out", torch.float32, plan.num_chunks)
    _want(signs_out, "signs_out", torch.int8, n)
    _want(nonfinite_out, "nonfinite_out", torch.int64, 1)
    _check(lib().ob_adam_compress_step(
        plan.handle, _dev(g, "g"), _gdtype(g), _dev(err, "err"), _errdtype(err), _dev(m, "m"), _dev(v, "v"),
        _dev(p, "p"),
        _dev(words_out, "words_out"), _dev(scales_out, "scales_out"), _dev(signs_out, "signs_out"),
        _dev(nonfinite_out, "nonfinite_out"), ctypes.byref(hp), _stream(stream)), "ob_adam_compress_step")


def ob_adam_compress_step_noalloc(n: int, chunk_size: int, g, err, m, v, p, words_out, scales_out,
                                  hp: ob_hparams, signs_out=None, nonfinite_out=None, stream=None):
    """ob_adam_compress_step for uniform chunks of chunk_size, without a plan and without any device
    allocation (the library's static buffer holds the tables and partial sums)."""
    K = (n + chunk_size - 1) // chunk_size if n > 0 and chunk_size > 0 else 0
    _want(g, "g", g.dtype, n)
    _want(err, "err", err.dtype, n)
    for name, t in (("m", m), ("v", v), ("p", p)):
        _want(t, name, torch.float32, n)
    _want(words_out, "words_out", torch.int32, (n + 31) // 32)
    _want(scales_out, "scales_out", torch.float32, K)
    _want(signs_out, "signs_out", torch.int8, n)
    _want(nonfinite_out, "nonfinite_out", torch.int64, 1)
    _check(lib().ob_adam_compress_step_noalloc(
        n, chunk_size, _dev(g, "g"), _gdtype(g), _dev(err, "err"), _errdtype(err), _dev(m, "m"), _dev(v, "v"),
        _dev(p, "p"), _dev(words_out, "words_out"), _dev(scales_out, "scales_out"), _dev(signs_out, "signs_out"),
        _dev(nonfinite_out, "nonfinite_out"), ctypes.byref(hp), _stream(stream)), "ob_adam_compress_step_noalloc")


def ob_adam_worker_compress(plan: Plan, g, err, words_out, scales_out, hp: ob_hparams, signs_out=None,
                            nonfinite_out=None, stream=None):
    """The worker's half before the exchange: signs, scales and the error from its own g_hat."""
    n = plan.n
    _want(g, "g", g.dtype, n)
    _want(err, "err", err.dtype, n)
    _want(words_out, "words_out", torch.int32, (n + 31) // 32)
    _want(scales_out, "scales_out", torch.float32, plan.num_chunks)
    _want(signs_out, "signs_out", torch.int8, n)
    _want(nonfinite_out, "nonfinite_out", torch.int64, 1)
    _check(lib().ob_adam_worker_compress(
        plan.handle, _dev(g, "g"), _gdtype(g), _dev(err, "err"), _errdtype(err), _dev(words_out, "words_out"),
        _dev(scales_out, "scales_out"), _dev(signs_out, "signs_out"), _dev(nonfinite_out, "nonfinite_out"),
        ctypes.byref(hp), _stream(stream)), "ob_adam_worker_compress")


def ob_adam_worker_update(plan: Plan, words, scales, m, v, p, hp: ob_hparams, stream=None):
    """The worker's half after the exchange: g_hat from the exchanged words and scales, then m and p."""
    n = plan.n
    _want(words, "words", torch.int32, (n + 31) // 32)
    _want(scales, "scales", torch.float32, plan.num_chunks)
    for name, t in (("m", m), ("v", v), ("p", p)):
        _want(t, name, torch.float32, n)
    _check(lib().ob_adam_worker_update(
        plan.handle, _dev(words, "words"), _dev(scales, "scales"), _dev(m, "m"), _dev(v, "v"), _dev(p, "p"),
        ctypes.byref(hp), _stream(stream)), "ob_adam_worker_update")


def ob_lamb_worker_update(plan: Plan, words, scales, m, v, p, ratios_out, hp: ob_hparams, stream=None):
    """1-bit LAMB's half after the exchange: m on the exchanged g_hat, then trust ratios and the update."""
    n = plan.n
    _want(words, "words", torch.int32, (n + 31) // 32)
    _want(scales, "scales", torch.float32, plan.num_chunks)
    _want(ratios_out, "ratios_out", torch.float32, plan.num_chunks)
    for name, t in (("m", m), ("v", v), ("p", p)):
        _want(t, name, torch.float32, n)
    _check(lib().ob_lamb_worker_update(
        plan.handle, _dev(words, "words"), _dev(scales, "scales"), _dev(m, "m"), _dev(v, "v"), _dev(p, "p"),
        _dev(ratios_out, "ratios_out"), ctypes.byref(hp), _stream(stream)), "ob_lamb_worker_update")


def ob_lamb_compress_step(plan: Plan, g, err, m, v, p, words_out, scales_out, ratios_out, hp: ob_hparams,
                          signs_out=None, nonfinite_out=None, stream=None):
    n = plan.n
    _want(g, "g", g.dtype, n)
    _want(err, "err", err.dtype, n)
    for name, t in (("m", m), ("v", v), ("p", p)):
        _want(t, name, torch.float32, n)
    _want(words_out, "words_out", torch.int32, (n + 31) // 32)
    _want(scales_out, "scales_out", torch.float32, plan.num_chunks)
    _want(ratios_out, "ratios_out", torch.float32, plan.num_chunks)
    _want(signs_out, "signs_out", torch.int8, n)
    _want(nonfinite_out, "nonfinite_out", torch.int64, 1)
    _check(lib().ob_lamb_compress_step(
        plan.handle, _dev(g, "g"), _gdtype(g), _dev(err, "err"), _errdtype(err), _dev(m, "m"), _dev(v, "v"),
        _dev(p, "p"), _dev(words_out, "words_out"), _dev(scales_out, "scales_out"),
        _dev(ratios_out, "ratios_out"), _dev(signs_out, "signs_out"), _dev(nonfinite_out, "nonfinite_out"),
        ctypes.byref(hp), _stream(stream)), "ob_lamb_compress_step")


def ob_lamb_warmup_step(plan: Plan, g, m, v, p, ratios_out, hp: ob_hparams, stream=None):
    n = plan.n
    _want(g, "g", g.dtype, n)
    for name, t in (("m", m), ("v", v), ("p", p)):
        _want(t, name, torch.float32, n)
    _want(ratios_out, "ratios_out", torch.float32, plan.num_chunks)
    _check(lib().ob_lamb_warmup_step(plan.handle, _dev(g, "g"), _gdtype(g), _dev(m, "m"), _dev(v, "v"),
                                     _dev(p, "p"), _dev(ratios_out, "ratios_out"), ctypes.byref(hp),
                                     _stream(stream)), "ob_lamb_warmup_step")


def ob_server_reduce(plan: Plan, worker_words, worker_scales, server_err, words_out, scales_out,
                     stream=None):
    n = plan.n
    W = worker_words.shape[0]
    _want(worker_words, "worker_words", torch.int32, W * ((n + 31) // 32))
    _want(worker_scales, "worker_scales", torch.float32, W * plan.num_chunks)
    _want(server_err, "server_err", torch.float32, n)
    _want(words_out, "words_out", torch.int32, (n + 31) // 32)
    _want(scales_out, "scales_out", torch.float32, plan.num_chunks)
    _check(lib().ob_server_reduce(plan.handle, W, _dev(worker_words, "worker_words"),
                                  _dev(worker_scales, "worker_scales"), _dev(server_err, "server_err"),
                                  _dev(words_out, "words_out"), _dev(scales_out, "scales_out"),
                                  _stream(stream)), "ob_server_reduce")


def ob_pack(x, words_out, stream=None):
    n = x.numel()
    _want(words_out, "words_out", torch.int32, (n + 31) // 32)
    _check(lib().ob_pack(_dev(x, "x"), _gdtype(x), n, _dev(words_out, "words_out"), _stream(stream)),
           "ob_pack")


def ob_unpack(plan: Plan | None, words, n: int, out, scales=None, stream=None):
    _want(words, "words", torch.int32, (n + 31) // 32)
    _want(out, "out", torch.float32, n)
    if scales is not None:
        if plan is None:
            raise ValueError("ob_unpack with scales needs the plan that defines the chunks")
        _want(scales, "scales", torch.float32, plan.num_chunks)
    _check(lib().ob_unpack(plan.handle if plan is not None else None, _dev(words, "words"), n,
                           _dev(scales, "scales"), _dev(out, "out"), _stream(stream)), "ob_unpack")


def ob_plan_set_diagnostics(plan: Plan, err_sumsq=None, plus_count=None):
    """Per-chunk diagnostics of later compressed steps into err_sumsq (float64[K]) and plus_count
    (int64[K]); both None switches them off."""
    _want(err_sumsq, "err_sumsq", torch.float64, plan.num_chunks)
    _want(plus_count, "plus_count", torch.int64, plan.num_chunks)
    _check(lib().ob_plan_set_diagnostics(plan.handle, _dev(err_sumsq, "err_sumsq"),
                                         _dev(plus_count, "plus_count")), "ob_plan_set_diagnostics")


def ob_plan_set_guard(plan: Plan, norm=None):
    """Leave out later steps that find norm (one fp32 element) not finite when they run on the GPU; None: leave out none."""
    _want(norm, "norm", torch.float32, 1)
    _check(lib().ob_plan_set_guard(plan.handle, _dev(norm, "norm")), "ob_plan_set_guard")


def ob_plan_set_timing(plan: Plan, enable: bool):
    _check(lib().ob_plan_set_timing(plan.handle, 1 if enable else 0), "ob_plan_set_timing")


def ob_plan_read_timing(plan: Plan, kernel: int) -> tuple[float, int]:
    ms = ctypes.c_double()
    cnt = ctypes.c_int64()
    _check(lib().ob_plan_read_timing(plan.handle, kernel, ctypes.byref(ms), ctypes.byref(cnt)),
           "ob_plan_read_timing")
    return ms.value, cnt.value


# ---- AdamW over lists of tensors ----

class Tensors:
    """Owner of an ob_tensors handle (destroyed with the object): a list of tensors by size and type."""

    def __init__(self, handle: ctypes.c_void_p, sizes, g_dtypes, p_dtypes, device: torch.device):
        self.handle = handle
        self.sizes = tuple(sizes)
        self.g_dtypes = tuple(g_dtypes)
        self.p_dtypes = tuple(p_dtypes)
        self.device = device
        self.state_elems = int(lib().ob_tensors_state_elems(handle))
        self.norm_bytes = int(lib().ob_tensor_norms_workspace(handle))
        module = _obtorch()
        self.native = module.list(handle.value, self.sizes, bytes(module.scalar_type(d) for d in self.g_dtypes),
                                  bytes(module.scalar_type(d) for d in self.p_dtypes), device.index, self.state_elems)

    def __len__(self) -> int:
        return len(self.sizes)

    @property
    def num_elements(self) -> int:
        return int(lib().ob_tensors_num_elements(self.handle))

    def state_offset(self, t: int) -> int:
        return int(lib().ob_tensors_state_offset(self.handle, t))

    def destroy(self):
        if self.handle:
            self.native = None
            _check(lib().ob_tensors_destroy(self.handle), "ob_tensors_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    def _fail(self, code, what, lists, flats, names=("grads", "params")):
        """Raise what a call's code says: a status of the library, or the place of the first argument that is
        not as it should be (lists: gradients, parameters; flats: (name, tensor, type, elements))."""
        if code > 0:
            raise ObError(code, what)
        where, j = divmod(-code - 1, 1 << 32)
        if where >= 2:
            name, t, dtype, numel = flats[where - 2]
        else:
            name, ts = names[where], lists[where]
            if len(ts) != len(self.sizes):
                raise ValueError(f"{name} must have {len(self.sizes)} tensors, got {len(ts)}")
            if ts[j] is None:
                raise TypeError(f"{name}[{j}] must be a torch.Tensor")
            name, t, dtype, numel = f"{name}[{j}]", ts[j], (self.g_dtypes, self.p_dtypes)[where][j], self.sizes[j]
        self._refuse(t, name, dtype, numel)

    def _refuse(self, t, name, dtype, numel):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.layout is not torch.strided:
            raise ValueError(f"{name} must be a dense tensor, got {t.layout}")
        _want(t, name, dtype, numel)
        _dev(t, name)
        _want_memory(t, name)
        raise ValueError(f"{name} must be on {self.device}, the list's device (got {t.device})")


def _want_memory(t, name):
    if t is None:
        return
    if t.is_neg():
        raise ValueError(f"{name} must not be a negated view")
    if t.untyped_storage().nbytes() < (t.storage_offset() + t.numel()) * t.element_size():
        raise ValueError(f"{name} must have its memory (its storage was released or shrunk)")


def _dtype_list(d, count, name):
    ds = [d] * count if isinstance(d, torch.dtype) else list(d)
    if len(ds) != count:
        raise ValueError(f"{name} must have {count} entries, got {len(ds)}")
    for x in ds:
        if x not in _ERR_DTYPES:
            raise TypeError(f"{name} must be float32, bfloat16 or float16, got {x}")
    return ds


def _mult_array(x, count, name):
    if x is None:
        return None
    x = [float(y) for y in x]
    if len(x) != count:
        raise ValueError(f"{name} must have {count} entries, got {len(x)}")
    return (ctypes.c_float * count)(*x)


def ob_tensors_create(sizes, g_dtype, p_dtype, lr_mults=None, wd_mults=None, device=None) -> Tensors:
    """List of tensors of the given element counts; g_dtype and p_dtype: one torch dtype, or one per
    tensor.  device: the list's GPU (the current one by default)."""
    sizes = [int(s) for s in sizes]
    T = len(sizes)
    gd, pd = _dtype_list(g_dtype, T, "g_dtype"), _dtype_list(p_dtype, T, "p_dtype")
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError(f"the list must be on the GPU (got {device}); there is no CPU path")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    codes = [(ctypes.c_int32 * T)(*[_ERR_DTYPES[x] for x in ds]) for ds in (gd, pd)]
    h = ctypes.c_void_p()
    with torch.cuda.device(device):
        _check(lib().ob_tensors_create(T, (ctypes.c_int64 * T)(*sizes), *codes, _mult_array(lr_mults, T, "lr_mults"),
                                       _mult_array(wd_mults, T, "wd_mults"), ctypes.byref(h)), "ob_tensors_create")
    return Tensors(h, sizes, gd, pd, device)


def control_create(device=None) -> torch.Tensor:
    """A control block (ob_control and the norm's partial sums) for ob_grad_norm and the steps."""
    c = torch.zeros(OB_CONTROL_BYTES // 4, dtype=torch.int32, device="cuda" if device is None else device)
    c[10:11].view(torch.float32).fill_(1.0)
    return c


def control_fields(control: torch.Tensor) -> dict:
    """The control block's fields as views of it (one element each): norm, grad_scale, step, skipped, bc1, bc2,
    lr_scale, skip.  Reading a value waits for the GPU; lr_scale may be written."""
    f, q, d = control.view(torch.float32), control.view(torch.int64), control.view(torch.float64)
    return {"norm": f[0:1], "grad_scale": f[1:2], "step": q[1:2], "skipped": q[2:3], "bc1": d[3:4], "bc2": d[4:5],
            "lr_scale": f[10:11], "skip": control[11:12]}


def _list_stream(tensors: Tensors, stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(tensors.device.index)  # what current_stream() wraps, at 1/25 of its time
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _list(x):
    return x if isinstance(x, (list, tuple)) else list(x)


def _hparams(hp):
    if type(hp) is not ob_adamw_hparams:
        raise TypeError(f"hp must be made by adamw_hparams, got {type(hp)}")
    return ctypes.addressof(hp)


_CONTROL = (torch.int32, OB_CONTROL_BYTES // 4)


def ob_grad_norm(tensors: Tensors, grads, control, g_mult=1.0, max_norm=0.0, hp: ob_adamw_hparams | None = None,
                 stream=None):
    """Global norm of the gradients (a list; None: no gradient) and the factor that clips it to max_norm
    (<= 0 or infinite: no clipping), into the control block; with hp also the step count and the bias
    corrections of the step that follows."""
    if control is None:
        raise TypeError("control must be a torch.Tensor")
    grads = _list(grads)
    code = _obtorch().grad_norm(tensors.native, grads, g_mult, max_norm, None if hp is None else _hparams(hp), control,
                                _list_stream(tensors, stream))
    if code:
        tensors._fail(code, "ob_grad_norm", (grads,), (("control", control, *_CONTROL),))


def ob_adamw_step(tensors: Tensors, grads, params, m, v, hp: ob_adamw_hparams, master=None, control=None, stream=None,
                  norm=None):
    """AdamW step with fp32 states: m, v and the optional master copy flat, of tensors.state_elems.  norm=(g_mult,
    max_norm): ob_grad_norm with these and hp first, once the arguments of both are checked."""
    if norm is not None and control is None:
        raise TypeError("control must be a torch.Tensor")
    grads, params = _list(grads), _list(params)
    code = _obtorch().adamw_step(tensors.native, grads, params, _hparams(hp), _list_stream(tensors, stream), master, m, v,
                                 control, norm)
    if code:
        f32 = (torch.float32, tensors.state_elems)
        tensors._fail(code, "ob_adamw_step", (grads, params),
                      (("master", master, *f32), ("m", m, *f32), ("v", v, *f32), ("control", control, *_CONTROL)))


def ob_adamw8_step(tensors: Tensors, grads, params, m_codes, m_scales, v_codes, v_scales, hp: ob_adamw_hparams,
                   master=None, control=None, stream=None, norm=None):
    """AdamW step with 8-bit states: int8 / uint8 codes of tensors.state_elems, one fp32 scale per 256.  norm as
    ob_adamw_step."""
    if norm is not None and control is None:
        raise TypeError("control must be a torch.Tensor")
    grads, params = _list(grads), _list(params)
    code = _obtorch().adamw8_step(tensors.native, grads, params, _hparams(hp), _list_stream(tensors, stream), master,
                                  m_codes, m_scales, v_codes, v_scales, control, norm)
    if code:
        N = tensors.state_elems
        scales = (torch.float32, N // OB_STATE_BLOCK)
        tensors._fail(code, "ob_adamw8_step", (grads, params),
                      (("master", master, torch.float32, N), ("m_codes", m_codes, torch.int8, N),
                       ("m_scales", m_scales, *scales), ("v_codes", v_codes, torch.uint8, N),
                       ("v_scales", v_scales, *scales), ("control", control, *_CONTROL)))


def _state8(what, encode, stream, *tensors):
    """A conversion of (m, v, m_codes, m_scales, v_codes, v_scales); either moment may be None throughout."""
    m, v = tensors[:2]
    lead = m if m is not None else v
    if lead is None:
        raise ValueError("neither moment is given")
    for name, x, codes, scales in (("m", m, *tensors[2:4]), ("v", v, *tensors[4:])):
        if (x is None) != (codes is None) or (x is None) != (scales is None):
            raise ValueError(f"{name}, {name}_codes and {name}_scales come together")
    n, index = lead.numel(), lead.get_device()
    if index < 0:
        code = -1   # not on a GPU
    elif index == torch.cuda.current_device():
        s = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream).value or 0
        code = _obtorch().state8(encode, n, index, s, *tensors)
    else:
        with torch.cuda.device(index):
            code = _obtorch().state8(encode, n, index, _stream(stream).value or 0, *tensors)
    if code > 0:
        raise ObError(code, what)
    if code < 0:
        blocks = -(-n // OB_STATE_BLOCK)
        names = ("m", "v", "m_codes", "m_scales", "v_codes", "v_scales")
        dtypes = (torch.float32, torch.float32, torch.int8, torch.float32, torch.uint8, torch.float32)
        for t, name, dtype, numel in zip(tensors, names, dtypes, (n, n, n, blocks, n, blocks)):
            _want(t, name, dtype, numel)
        for t, name in zip(tensors, names):
            _dev(t, name)
            _want_memory(t, name)
        j = (-code - 1 >> 32) - 2
        raise ValueError(f"{names[j]} must be on {lead.device} (got {tensors[j].device})")


def ob_state8_encode(m, v, m_codes, m_scales, v_codes, v_scales, stream=None):
    """fp32 moments into the 8-bit format, rounded to nearest (m or v with its codes and scales: None)."""
    _state8("ob_state8_encode", True, stream, m, v, m_codes, m_scales, v_codes, v_scales)


def ob_state8_decode(m_codes, m_scales, v_codes, v_scales, m, v, stream=None):
    """The fp32 moments that 8-bit codes and scales stand for (m or v with its codes and scales: None)."""
    _state8("ob_state8_decode", False, stream, m, v, m_codes, m_scales, v_codes, v_scales)


# ---- norms of many tensors, and clipped gradients ----

def _workspace(workspace, nbytes, device, stream):
    """The caller's workspace, or a new one: of the stream that the call is enqueued on, behind what its memory was used for."""
    if workspace is not None:
        return workspace
    if stream is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device)
    with torch.cuda.stream(stream):
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def _fail_workspace(tensors, workspace, nbytes, code, place):
    """Raise where a call's code names its workspace."""
    if code < 0 and (-code - 1) >> 32 == place:
        if isinstance(workspace, torch.Tensor) and workspace.dtype == torch.uint8 and workspace.numel() < nbytes:
            raise ValueError(f"workspace must have at least {nbytes} bytes, got {workspace.numel()}")
        tensors._refuse(workspace, "workspace", torch.uint8, workspace.numel() if isinstance(workspace, torch.Tensor) else 0)


def ob_tensor_norms_workspace(tensors: Tensors) -> int:
    """Bytes of the workspace of ob_tensor_norms."""
    return int(lib().ob_tensor_norms_workspace(tensors.handle))


def ob_tensor_norms(tensors: Tensors, grads, norms, g_mult=1.0, kind=OB_NORM_2, workspace=None, stream=None):
    """Norm of every gradient (a list; None: 0) times |g_mult|, and behind them the norm of all, into norms (fp32, one more than
    tensors).  kind: OB_NORM_2 or OB_NORM_MAX.  workspace: a byte tensor of ob_tensor_norms_workspace, or None for a new one."""
    grads = _list(grads)
    need = tensors.norm_bytes
    workspace = _workspace(workspace, need, tensors.device, stream)
    code = _obtorch().tensor_norms(tensors.native, grads, norms, workspace, need, g_mult, kind, _list_stream(tensors, stream))
    if code:
        _fail_workspace(tensors, workspace, need, code, 3)
        tensors._fail(code, "ob_tensor_norms", (grads,), (("norms", norms, torch.float32, len(tensors) + 1),))


def ob_clip_grads(tensors: Tensors, grads, norms, max_norm, g_mult=1.0, out=None, per_tensor=False, stream=None):
    """The gradients times g_mult min(1, max_norm / (norm + 1e-6)) (max_norm <= 0 or infinite: times g_mult), by the norm of
    all or, per_tensor, each by its own; a norm that is not finite makes them NaN.  out: tensors of the list's parameter
    types; None: in place."""
    grads, out = _list(grads), None if out is None else _list(out)
    code = _obtorch().clip_grads(tensors.native, grads, out, norms, max_norm, g_mult, per_tensor, _list_stream(tensors, stream))
    if code:
        tensors._fail(code, "ob_clip_grads", (grads, out), (("norms", norms, torch.float32, len(tensors) + 1),), ("grads", "out"))


# ---- Muon over lists of matrices ----

class MuonPlan:
    """Owner of an ob_muon handle (destroyed with the object): the matrices of a list's tensors."""

    def __init__(self, handle: ctypes.c_void_p, tensors: Tensors):
        self.handle, self.tensors = handle, tensors
        self.workspace_bytes = int(lib().ob_muon_workspace(handle))

    def destroy(self):
        if self.handle:
            _check(lib().ob_muon_destroy(self.handle), "ob_muon_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def ob_muon_create(tensors: Tensors, shapes) -> MuonPlan:
    """Plan for a list whose tensors have these shapes: (rows, columns), or more dimensions in front for matrices behind each
    other."""
    shapes = [tuple(int(n) for n in s) for s in shapes]
    if len(shapes) != len(tensors):
        raise ValueError(f"shapes must have {len(tensors)} entries, got {len(shapes)}")
    for j, (s, n) in enumerate(zip(shapes, tensors.sizes)):
        if len(s) < 2:
            raise ValueError(f"tensor {j} is no matrix: shape {s}")
        if math.prod(s) != n:
            raise ValueError(f"tensor {j} has {n} elements, its shape {s} has {math.prod(s)}")
    rows, cols = ((ctypes.c_int64 * len(shapes))(*[max(s[d], 1) if math.prod(s) == 0 else s[d] for s in shapes]) for d in (-2, -1))
    h = ctypes.c_void_p()
    _check(lib().ob_muon_create(tensors.handle, rows, cols, ctypes.byref(h)), "ob_muon_create")
    return MuonPlan(h, tensors)


def ob_muon_step(plan: MuonPlan, grads, params, m, hp: ob_muon_hparams, workspace, master=None, control=None, stream=None,
                 norm=None):
    """Muon step: m and the optional master copy flat, of the list's state_elems; workspace: a byte tensor of
    plan.workspace_bytes (None where that is 0).  norm=(g_mult, max_norm): ob_grad_norm with these first, once the arguments of both are checked; it
    counts the step in control."""
    if norm is not None and control is None:
        raise TypeError("control must be a torch.Tensor")
    if type(hp) is not ob_muon_hparams:
        raise TypeError(f"hp must be made by muon_hparams, got {type(hp)}")
    if not plan.handle:
        raise ValueError("the plan is destroyed")
    grads, params, tensors = _list(grads), _list(params), plan.tensors
    code = _obtorch().muon_step(tensors.native, plan.handle.value, grads, params, ctypes.addressof(hp), _list_stream(tensors, stream),
                                master, m, workspace, plan.workspace_bytes, control, norm)
    if code:
        _fail_workspace(tensors, workspace, plan.workspace_bytes, code, 4)
        f32 = (torch.float32, tensors.state_elems)
        tensors._fail(code, "ob_muon_step", (grads, params),
                      (("master", master, *f32), ("m", m, *f32), None, ("control", control, *_CONTROL)))


# ---- matrix products ----

def _refuse_product(a, b, out, c):
    """Raise what the binding saw in a product's tensors."""
    ts = [("a", a), ("b", b), ("out", out)] + ([] if c is None else [("c", c)])
    for name, t in ts:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    for name, t in ts:
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be on the GPU (got {t.device}); there is no CPU path")
        if t.layout is not torch.strided:
            raise ValueError(f"{name} must be a dense tensor, got {t.layout}")
        if t.is_neg() or t.is_conj():
            raise ValueError(f"{name} must not be a negated or conjugated view")
        if t.dim() != out.dim() or t.dim() not in (2, 3):
            raise ValueError(f"{name} must have two dimensions, or all three of them three (got {tuple(t.shape)})")
        if t.device != out.device:
            raise ValueError(f"{name} must be on {out.device} (got {t.device})")
    for name, t in ts[:2]:
        if t.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    if b.dtype != a.dtype:
        raise TypeError(f"b must be {a.dtype}, got {b.dtype}")
    if out.dtype not in _ERR_DTYPES:
        raise TypeError(f"out must be float32, bfloat16 or float16, got {out.dtype}")
    want = (*out.shape[:-2], a.shape[-2], b.shape[-1])
    if tuple(out.shape) != want or b.shape[-2] != a.shape[-1] or a.shape[:-2] != out.shape[:-2] or b.shape[:-2] != out.shape[:-2]:
        raise ValueError(f"shapes {tuple(a.shape)}, {tuple(b.shape)} and {tuple(out.shape)} are no product")
    if c is not None:
        if c.shape != out.shape:
            raise ValueError(f"c must have out's shape {tuple(out.shape)}, got {tuple(c.shape)}")
        if c.dtype != out.dtype:
            raise TypeError(f"c must be {out.dtype}, got {c.dtype}")
    for name, t in ts[2:]:
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must lie by rows (strides {t.stride()})")
    for name, t in ts:
        if t.untyped_storage().nbytes() < (t.storage_offset() + 1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride()))) * t.element_size():
            raise ValueError(f"{name} must have its memory (its storage was released or shrunk)")
    raise ValueError("the tensors are refused")


def ob_matmul(a, b, out, alpha=1.0, beta=0.0, c=None, symmetric=False, stream=None, workspace=None):
    """out = alpha * a @ b + beta * c for matrices or batches of them: a, b bfloat16 or float16, either by rows or transposed
    views; out and c (which may be out) float32, bfloat16 or float16, by rows.  symmetric: the caller knows that a @ b and
    c are; what is below the diagonal is computed and written above it too.  workspace: a byte tensor, or None to take what
    a product with few tiles and a long sum has use for (at most some 100 MB) from torch's allocator."""
    if stream is None:
        index = out.get_device() if isinstance(out, torch.Tensor) else -1
        code = _obtorch().matmul(a, b, out, c, alpha, beta, symmetric, torch._C._cuda_getCurrentRawStream(index) if index >= 0 else 0,
                                 workspace)
    else:
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), out.device if isinstance(out, torch.Tensor) else None)
        with torch.cuda.stream(stream):   # so that the workspace is the stream's
            code = _obtorch().matmul(a, b, out, c, alpha, beta, symmetric, stream.cuda_stream, workspace)
    if code > 0:
        raise ObError(code, "ob_matmul")
    if code < 0:
        if (-code - 1) >> 32 == 4:
            raise ValueError("workspace must be a contiguous byte tensor on the tensors' device, as large as the product has use for")
        _refuse_product(a, b, out, c)
