"""Python binding of libmoonep.so, the MoonEP balanced expert-parallel hot path on MI355X.

Thin ctypes marshalling only: every function here checks tensor shapes, dtypes,
devices and contiguity, then passes raw device pointers and the current HIP
stream to the C entry point of the same name (declared in include/moonep.h).
Tensors must live on the current device, and an explicit stream must belong to it.
All computation happens in the library's HIP kernels; there is no Python or
CPU fallback, and importing this package fails loudly if the library was not
built (``python -m balanced_token_dispatch_moonep_amd.build``).

PyTorch is used only to own device memory and streams.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

__all__ = [
    "MoonEPError", "Dims", "LIB_PATH", "lib", "NSTATS", "STAT_NAMES", "TRAINING", "F32_ROWS", "GRAD_ACCUM",
    "PLAN_LOWMIG",
    "PHASE_GATE_UP", "PHASE_DOWN", "PHASE_DACT", "PHASE_DX", "PHASE_DW2", "PHASE_DW13",
    "ST_BAD_ID", "ST_DUP_ID", "ST_CAPACITY", "ST_OVERFLOW", "ST_TRAIN_FALLBACK",
    "moonep_plan_workspace_bytes", "moonep_plan", "moonep_plan_noalloc", "NOALLOC_WS_BYTES",
    "moonep_prefetch", "moonep_dispatch",
    "moonep_combine", "moonep_dispatch_staged", "moonep_combine_staged", "moonep_grouped_ffn",
    "moonep_grouped_ffn_backward", "moonep_reduce_grad", "moonep_strerror", "moonep_version", "EXPORTED",
    "moonep_layer_norm", "moonep_layer_norm_workspace_bytes", "moonep_layer_norm_backward",
    "GradList", "moonep_grad_norm_workspace_bytes", "moonep_grad_norm", "moonep_grad_clip",
    "W4_MAX_PAIRS", "moonep_w4_code_bytes", "moonep_w4_scale_bytes", "moonep_quantize_w4",
    "moonep_w4_ffn_workspace_bytes", "moonep_w4_ffn",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoonep.so")

TRAINING = 1
F32_ROWS = 2
GRAD_ACCUM = 4
PLAN_LOWMIG = 512      # the planner's low-migration rule
# phase selection of the expert FFN calls (one GEMM kernel each; none set = all of the call's)
PHASE_GATE_UP, PHASE_DOWN = 8, 16
PHASE_DACT, PHASE_DX, PHASE_DW2, PHASE_DW13 = 32, 64, 128, 256
NSTATS = 16
ST_BAD_ID, ST_DUP_ID, ST_CAPACITY, ST_OVERFLOW, ST_TRAIN_FALLBACK = 1, 2, 4, 8, 16
STAT_NAMES = (
    "status", "replicas", "slot_replicas", "fallback_replicas", "fallback_rows",
    "migrated_rows", "migration_bound", "max_expert_load", "max_rank_load",
    "min_rank_load", "donors", "receivers", "max_replicas_per_rank", "total_rows",
    "reserved14", "reserved15",
)
NOALLOC_WS_BYTES = 8 << 20     # static plan workspace of moonep_plan_noalloc, per GPU
W4_MAX_PAIRS = 8192            # (token, k) pairs of one moonep_w4_ffn call, at most
EXPORTED = (
    "moonep_plan_workspace_bytes", "moonep_plan", "moonep_plan_noalloc", "moonep_prefetch", "moonep_dispatch",
    "moonep_combine", "moonep_dispatch_staged", "moonep_combine_staged", "moonep_grouped_ffn",
    "moonep_grouped_ffn_backward", "moonep_reduce_grad", "moonep_strerror", "moonep_version",
    "moonep_layer_norm", "moonep_layer_norm_workspace_bytes", "moonep_layer_norm_backward",
    "moonep_grad_norm_workspace_bytes", "moonep_grad_norm", "moonep_grad_clip",
    "moonep_w4_code_bytes", "moonep_w4_scale_bytes", "moonep_quantize_w4",
    "moonep_w4_ffn_workspace_bytes", "moonep_w4_ffn",
)


class MoonEPError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {moonep_strerror(code)} ({code})")
        self.code = code


class Dims(ctypes.Structure):
    """moonep_dims_t."""
    _fields_ = [("R", ctypes.c_int32), ("E", ctypes.c_int32), ("B", ctypes.c_int32),
                ("S", ctypes.c_int32), ("K", ctypes.c_int32), ("H", ctypes.c_int32),
                ("I", ctypes.c_int32), ("flags", ctypes.c_uint32)]

    @classmethod
    def make(cls, R, E, B, S, K, H, I=0, training=False, f32_rows=False, grad_accum=False, phases=0,
             plan_rule="chain") -> "Dims":
        if plan_rule not in ("chain", "lowmig"):
            raise ValueError(f"unknown plan rule {plan_rule!r}")
        flags = (TRAINING if training else 0) | (F32_ROWS if f32_rows else 0) | (GRAD_ACCUM if grad_accum else 0)
        flags |= int(phases) | (PLAN_LOWMIG if plan_rule == "lowmig" else 0)
        return cls(R, E, B, S, K, H, I, flags)

    def with_flags(self, flags: int) -> "Dims":
        return Dims(self.R, self.E, self.B, self.S, self.K, self.H, self.I, int(flags))

    @property
    def C(self) -> int:
        return self.S * self.K


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m balanced_token_dispatch_moonep_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, SZ, VP = ctypes.POINTER(Dims), ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
    L.moonep_plan_workspace_bytes.argtypes = [P]
    L.moonep_plan_workspace_bytes.restype = SZ
    L.moonep_plan.argtypes = [P, VP, VP, VP, VP, VP, VP]
    L.moonep_plan_noalloc.argtypes = [P, VP, VP, VP, VP, VP]
    L.moonep_prefetch.argtypes = [P, VP, VP, VP, VP, VP, VP]
    L.moonep_dispatch.argtypes = [P, VP, VP, VP, VP, VP]
    L.moonep_combine.argtypes = [P, VP, VP, VP, VP, VP]
    L.moonep_dispatch_staged.argtypes = [P, VP, VP, VP, VP, VP, VP]
    L.moonep_combine_staged.argtypes = [P, VP, VP, VP, VP, VP, VP]
    L.moonep_grouped_ffn.argtypes = [P, VP, VP, VP, VP, VP, VP, VP, VP, VP, VP, VP]
    L.moonep_grouped_ffn_backward.argtypes = [P] + [VP] * 16
    L.moonep_reduce_grad.argtypes = [P, VP, VP, VP, VP, VP, VP]
    for n in ("moonep_plan", "moonep_plan_noalloc", "moonep_prefetch", "moonep_dispatch", "moonep_combine",
              "moonep_dispatch_staged", "moonep_combine_staged", "moonep_grouped_ffn",
              "moonep_grouped_ffn_backward", "moonep_reduce_grad"):
        getattr(L, n).restype = I32
    F32, N32 = ctypes.c_float, ctypes.c_int32
    L.moonep_layer_norm.argtypes = [P, VP, VP, VP, F32, VP, VP, VP, VP]
    L.moonep_layer_norm_workspace_bytes.argtypes = [P]
    L.moonep_layer_norm_backward.argtypes = [P] + [VP] * 10
    L.moonep_grad_norm_workspace_bytes.argtypes = [N32]
    L.moonep_grad_norm.argtypes = [N32] + [VP] * 6
    L.moonep_grad_clip.argtypes = [N32] + [VP] * 4 + [F32, VP]
    L.moonep_w4_code_bytes.argtypes = L.moonep_w4_scale_bytes.argtypes = [N32, N32]
    L.moonep_quantize_w4.argtypes = [N32, N32, N32] + [VP] * 4
    L.moonep_w4_ffn_workspace_bytes.argtypes = [P]
    L.moonep_w4_ffn.argtypes = [P] + [VP] * 10
    for n in ("moonep_layer_norm_workspace_bytes", "moonep_grad_norm_workspace_bytes", "moonep_w4_code_bytes",
              "moonep_w4_scale_bytes", "moonep_w4_ffn_workspace_bytes"):
        getattr(L, n).restype = SZ
    for n in ("moonep_layer_norm", "moonep_layer_norm_backward", "moonep_grad_norm", "moonep_grad_clip",
              "moonep_quantize_w4", "moonep_w4_ffn"):
        getattr(L, n).restype = I32
    L.moonep_strerror.argtypes = [I32]
    L.moonep_strerror.restype = ctypes.c_char_p
    L.moonep_version.argtypes = []
    L.moonep_version.restype = ctypes.c_char_p
    return L


_LIB = None


def _lib():
    """The loaded library (loaded on first use; raises ImportError if it was never built)."""
    global _LIB
    if _LIB is None:
        _LIB = _load()
    return _LIB


def __getattr__(name):
    if name == "lib":
        return _lib()
    raise AttributeError(name)


def moonep_strerror(code: int) -> str:
    return _lib().moonep_strerror(int(code)).decode()


def moonep_version() -> str:
    return _lib().moonep_version().decode()


# ----------------------------------------------------------------------------
# marshalling helpers
# ----------------------------------------------------------------------------

_TORCH = None


def _torch():
    """torch, imported with the first call that needs it."""
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return int(stream) if isinstance(stream, int) else int(stream.cuda_stream)
    torch = _torch()
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _ptr(t, name, dtype=None, shape=None, numel=None, optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (the library has no CPU path)")
    if t.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}; the library runs on the current device "
                         f"cuda:{torch.cuda.current_device()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")
    return t.data_ptr()


def _ws(d: Dims, plan_ws):
    """The plan workspace: uint8, exactly moonep_plan_workspace_bytes(d) bytes."""
    return _ptr(plan_ws, "plan_ws", _torch().uint8, numel=moonep_plan_workspace_bytes(d))


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise MoonEPError(rc, where)


def _rows_dtype(d: Dims):
    torch = _torch()
    return torch.float32 if d.flags & F32_ROWS else torch.bfloat16


# ----------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ----------------------------------------------------------------------------

def moonep_plan_workspace_bytes(d: Dims) -> int:
    n = _lib().moonep_plan_workspace_bytes(ctypes.byref(d))
    if n == 0:
        raise MoonEPError(-1, "moonep_plan_workspace_bytes")
    return int(n)


def moonep_plan(d: Dims, topk, plan_ws, cu_seqlens, dest, stats, stream=None) -> None:
    torch = _torch()
    args = (
        _ptr(topk, "topk", torch.int32, (d.R, d.S, d.K)),
        _ws(d, plan_ws),
        _ptr(cu_seqlens, "cu_seqlens", torch.int32, (d.R, d.E + d.B + 1)),
        _ptr(dest, "dest", torch.int32, (d.R, d.S, d.K)),
        _ptr(stats, "stats", torch.int32, (NSTATS,)),
    )
    _check(_lib().moonep_plan(ctypes.byref(d), *args, _stream(stream)), "moonep_plan")


def moonep_plan_noalloc(d: Dims, topk, cu_seqlens, dest, stats, stream=None) -> None:
    """moonep_plan with the library's static plan workspace (no device allocation); for the
    plan + dispatch + combine path.  Calls overlapping on one GPU race."""
    torch = _torch()
    args = (
        _ptr(topk, "topk", torch.int32, (d.R, d.S, d.K)),
        _ptr(cu_seqlens, "cu_seqlens", torch.int32, (d.R, d.E + d.B + 1)),
        _ptr(dest, "dest", torch.int32, (d.R, d.S, d.K)),
        _ptr(stats, "stats", torch.int32, (NSTATS,)),
    )
    _check(_lib().moonep_plan_noalloc(ctypes.byref(d), *args, _stream(stream)), "moonep_plan_noalloc")


def moonep_prefetch(d: Dims, plan_ws, w13_home, w2_home, w13_slot, w2_slot, stream=None) -> None:
    torch = _torch()
    bf = torch.bfloat16
    args = (
        _ws(d, plan_ws),
        _ptr(w13_home, "w13_home", bf, (d.E, d.H, 2 * d.I)),
        _ptr(w2_home, "w2_home", bf, (d.E, d.I, d.H)),
        _ptr(w13_slot, "w13_slot", bf, (d.R, d.B, d.H, 2 * d.I), optional=d.B == 0),
        _ptr(w2_slot, "w2_slot", bf, (d.R, d.B, d.I, d.H), optional=d.B == 0),
    )
    _check(_lib().moonep_prefetch(ctypes.byref(d), *args, _stream(stream)), "moonep_prefetch")


def moonep_dispatch(d: Dims, dest, src, row_scale, recv, stream=None) -> None:
    torch = _torch()
    rt = _rows_dtype(d)
    args = (
        _ptr(dest, "dest", torch.int32, (d.R, d.S, d.K)),
        _ptr(src, "src", rt, (d.R, d.S, d.H)),
        _ptr(row_scale, "row_scale", torch.float32, (d.R, d.S, d.K), optional=True),
        _ptr(recv, "recv", rt, (d.R * d.S * d.K, d.H)),
    )
    _check(_lib().moonep_dispatch(ctypes.byref(d), *args, _stream(stream)), "moonep_dispatch")


def moonep_combine(d: Dims, dest, y, gates, out, stream=None) -> None:
    torch = _torch()
    rt = _rows_dtype(d)
    args = (
        _ptr(dest, "dest", torch.int32, (d.R, d.S, d.K)),
        _ptr(y, "y", rt, (d.R * d.S * d.K, d.H)),
        _ptr(gates, "gates", torch.float32, (d.R, d.S, d.K), optional=True),
        _ptr(out, "out", rt, (d.R, d.S, d.H)),
    )
    _check(_lib().moonep_combine(ctypes.byref(d), *args, _stream(stream)), "moonep_combine")


def moonep_dispatch_staged(d: Dims, dest, src, row_scale, stage, recv, stream=None) -> None:
    """Non-zero-copy baseline of moonep_dispatch (arrival-order copy, then a sort-copy)."""
    torch = _torch()
    rt = _rows_dtype(d)
    M = d.R * d.S * d.K
    args = (
        _ptr(dest, "dest", torch.int32, (d.R, d.S, d.K)),
        _ptr(src, "src", rt, (d.R, d.S, d.H)),
        _ptr(row_scale, "row_scale", torch.float32, (d.R, d.S, d.K), optional=True),
        _ptr(stage, "stage", rt, (M, d.H)),
        _ptr(recv, "recv", rt, (M, d.H)),
    )
    _check(_lib().moonep_dispatch_staged(ctypes.byref(d), *args, _stream(stream)), "moonep_dispatch_staged")


def moonep_combine_staged(d: Dims, dest, y, gates, stage, out, stream=None) -> None:
    """Non-zero-copy baseline of moonep_combine (gather to arrival order, then reduce)."""
    torch = _torch()
    rt = _rows_dtype(d)
    M = d.R * d.S * d.K
    args = (
        _ptr(dest, "dest", torch.int32, (d.R, d.S, d.K)),
        _ptr(y, "y", rt, (M, d.H)),
        _ptr(gates, "gates", torch.float32, (d.R, d.S, d.K), optional=True),
        _ptr(stage, "stage", rt, (M, d.H)),
        _ptr(out, "out", rt, (d.R, d.S, d.H)),
    )
    _check(_lib().moonep_combine_staged(ctypes.byref(d), *args, _stream(stream)), "moonep_combine_staged")


def moonep_grouped_ffn(d: Dims, plan_ws, cu_seqlens, recv, w13_home, w2_home, w13_slot, w2_slot,
                       gu_save, act, y, stream=None) -> None:
    torch = _torch()
    bf = torch.bfloat16
    M = d.R * d.S * d.K
    args = (
        _ws(d, plan_ws),
        _ptr(cu_seqlens, "cu_seqlens", torch.int32, (d.R, d.E + d.B + 1)),
        _ptr(recv, "recv", bf, (M, d.H)),
        _ptr(w13_home, "w13_home", bf, (d.E, d.H, 2 * d.I)),
        _ptr(w2_home, "w2_home", bf, (d.E, d.I, d.H)),
        _ptr(w13_slot, "w13_slot", bf, (d.R, d.B, d.H, 2 * d.I), optional=d.B == 0),
        _ptr(w2_slot, "w2_slot", bf, (d.R, d.B, d.I, d.H), optional=d.B == 0),
        _ptr(gu_save, "gu_save", bf, (M, 2 * d.I), optional=True),
        _ptr(act, "act", bf, (M, d.I)),
        _ptr(y, "y", bf, (M, d.H)),
    )
    _check(_lib().moonep_grouped_ffn(ctypes.byref(d), *args, _stream(stream)), "moonep_grouped_ffn")


def moonep_grouped_ffn_backward(d: Dims, plan_ws, cu_seqlens, recv, gu_save, act, dy, w13_home,
                                w2_home, w13_slot, w2_slot, drecv, dw13_home, dw2_home, dw13_red,
                                dw2_red, stream=None) -> None:
    """gu_save holds Gt|U from the forward on entry and dGt|dU on return."""
    torch = _torch()
    bf, f32 = torch.bfloat16, torch.float32
    M = d.R * d.S * d.K
    nb = d.B == 0
    args = (
        _ws(d, plan_ws),
        _ptr(cu_seqlens, "cu_seqlens", torch.int32, (d.R, d.E + d.B + 1)),
        _ptr(recv, "recv", bf, (M, d.H)),
        _ptr(gu_save, "gu_save", bf, (M, 2 * d.I)),
        _ptr(act, "act", bf, (M, d.I)),
        _ptr(dy, "dy", bf, (M, d.H)),
        _ptr(w13_home, "w13_home", bf, (d.E, d.H, 2 * d.I)),
        _ptr(w2_home, "w2_home", bf, (d.E, d.I, d.H)),
        _ptr(w13_slot, "w13_slot", bf, (d.R, d.B, d.H, 2 * d.I), optional=nb),
        _ptr(w2_slot, "w2_slot", bf, (d.R, d.B, d.I, d.H), optional=nb),
        _ptr(drecv, "drecv", bf, (M, d.H)),
        _ptr(dw13_home, "dw13_home", f32, (d.E, d.H, 2 * d.I)),
        _ptr(dw2_home, "dw2_home", f32, (d.E, d.I, d.H)),
        _ptr(dw13_red, "dw13_red", f32, (d.R, d.B, d.H, 2 * d.I), optional=nb),
        _ptr(dw2_red, "dw2_red", f32, (d.R, d.B, d.I, d.H), optional=nb),
    )
    _check(_lib().moonep_grouped_ffn_backward(ctypes.byref(d), *args, _stream(stream)),
           "moonep_grouped_ffn_backward")


def moonep_reduce_grad(d: Dims, plan_ws, dw13_home, dw2_home, dw13_red, dw2_red, stream=None) -> None:
    torch = _torch()
    f32 = torch.float32
    nb = d.B == 0
    args = (
        _ws(d, plan_ws),
        _ptr(dw13_home, "dw13_home", f32, (d.E, d.H, 2 * d.I)),
        _ptr(dw2_home, "dw2_home", f32, (d.E, d.I, d.H)),
        _ptr(dw13_red, "dw13_red", f32, (d.R, d.B, d.H, 2 * d.I), optional=nb),
        _ptr(dw2_red, "dw2_red", f32, (d.R, d.B, d.I, d.H), optional=nb),
    )
    _check(_lib().moonep_reduce_grad(ctypes.byref(d), *args, _stream(stream)), "moonep_reduce_grad")


# ----------------------------------------------------------------------------
# round the layer: norm, gradient clipping, decoding with 4-bit experts
# ----------------------------------------------------------------------------

def _bytes(n: int, where: str, code=lambda: -1) -> int:
    """What a size function said; its 0 is raised as the code that the sizes' own call returns for them."""
    if n == 0:
        raise MoonEPError(code(), where)
    return int(n)


@functools.lru_cache(maxsize=1024)
def _dims_bytes(name: str, dims: bytes) -> int:
    """What the size function `name` says for these dims (a pure function of them)."""
    d = ctypes.byref(Dims.from_buffer_copy(dims))
    # sizes are looked at before the pointers, and a NULL one ends the call: nothing is enqueued
    call = dict(moonep_w4_ffn_workspace_bytes=lambda: _lib().moonep_w4_ffn(d, *[None] * 10),
                moonep_layer_norm_workspace_bytes=lambda: _lib().moonep_layer_norm(d, *[None] * 3, 0.0, *[None] * 4))
    return _bytes(getattr(_lib(), name)(d), name, call[name])


def moonep_layer_norm(d: Dims, x, weight, bias, eps, y, mean=None, rstd=None, stream=None) -> None:
    """y = layer norm of the [R, S, H] rows x.  weight, bias [H] float32 or None; mean, rstd [R*S]
    float32, for the backward, or both None."""
    f32, rt = _torch().float32, _rows_dtype(d)
    args = (
        _ptr(x, "x", rt, (d.R, d.S, d.H)),
        _ptr(weight, "weight", f32, (d.H,), optional=True),
        _ptr(bias, "bias", f32, (d.H,), optional=True),
        float(eps),
        _ptr(y, "y", rt, (d.R, d.S, d.H)),
        _ptr(mean, "mean", f32, (d.R * d.S,), optional=True),
        _ptr(rstd, "rstd", f32, (d.R * d.S,), optional=True),
    )
    _check(_lib().moonep_layer_norm(ctypes.byref(d), *args, _stream(stream)), "moonep_layer_norm")


def moonep_layer_norm_workspace_bytes(d: Dims) -> int:
    return _dims_bytes("moonep_layer_norm_workspace_bytes", bytes(d))


def moonep_layer_norm_backward(d: Dims, dy, x, weight, mean, rstd, dx, dweight, dbias, ws=None, stream=None) -> None:
    """dx, and the sums dweight and dbias [H] float32 over all rows (either may be None; ws too if both
    are).  With GRAD_ACCUM the sums are added to what dweight and dbias hold."""
    torch = _torch()
    f32, rt = torch.float32, _rows_dtype(d)
    sums = dweight is not None or dbias is not None
    args = (
        _ptr(dy, "dy", rt, (d.R, d.S, d.H)),
        _ptr(x, "x", rt, (d.R, d.S, d.H)),
        _ptr(weight, "weight", f32, (d.H,), optional=True),
        _ptr(mean, "mean", f32, (d.R * d.S,)),
        _ptr(rstd, "rstd", f32, (d.R * d.S,)),
        _ptr(dx, "dx", rt, (d.R, d.S, d.H)),
        _ptr(dweight, "dweight", f32, (d.H,), optional=True),
        _ptr(dbias, "dbias", f32, (d.H,), optional=True),
        _ptr(ws, "ws", torch.uint8, numel=moonep_layer_norm_workspace_bytes(d), optional=not sums),
    )
    _check(_lib().moonep_layer_norm_backward(ctypes.byref(d), *args, _stream(stream)), "moonep_layer_norm_backward")


class GradList:
    """The gradients that moonep_grad_norm and moonep_grad_clip work on: contiguous float32 or bf16
    GPU tensors of any shape, made once and used step after step.

    Every call takes the tensors as they are at that moment: one given other memory is followed, and one
    whose length, type or device changed, or that is no longer contiguous, is refused."""

    def __init__(self, tensors):
        torch = _torch()
        types = {torch.float32: 0, torch.bfloat16: 1}
        self.tensors = tuple(tensors)
        for i, t in enumerate(self.tensors):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"gradient {i} must be a torch.Tensor")
            if t.dtype not in types:
                raise ValueError(f"gradient {i} must be float32 or bfloat16, got {t.dtype}")
            _ptr(t, f"gradient {i}")
        n = len(self.tensors)
        self.n = n
        self.device = self.tensors[0].device if n else None
        self._form = self._form_now()
        self._c_numel = (ctypes.c_int64 * n)(*(t.numel() for t in self.tensors))
        self._c_dtype = (ctypes.c_int32 * n)(*(types[t.dtype] for t in self.tensors))
        self._at = (None, None)          # the last addresses, and the same for C

    def _form_now(self):
        """What the kernels take for granted of the tensors besides their addresses (9.5 us for 60)."""
        T = _torch().Tensor
        return [list(map(f, self.tensors)) for f in (T.numel, T.is_contiguous, T.dtype.__get__, T.get_device)]

    def _arrays(self):
        torch = _torch()
        if self.n and self.device.index != torch.cuda.current_device():
            raise ValueError(f"the gradients are on {self.device}; the library runs on the current device "
                             f"cuda:{torch.cuda.current_device()}")
        # at an old address too: a tensor may have been cut short or read as another type in its place
        if self._form_now() != self._form:
            raise ValueError("a gradient changed its length, layout, type or device since the list was made")
        at = list(map(torch.Tensor.data_ptr, self.tensors))
        old, c_at = self._at
        if at != old:
            c_at = (ctypes.c_void_p * self.n)(*at)
            self._at = (at, c_at)
        return self.n, c_at, self._c_numel, self._c_dtype


def moonep_grad_norm_workspace_bytes(grads: GradList) -> int:
    return _bytes(_lib().moonep_grad_norm_workspace_bytes(grads.n), "moonep_grad_norm_workspace_bytes")


def moonep_grad_norm(grads: GradList, ws, norm, stream=None) -> None:
    """norm[0] (float32) = the 2-norm of all gradients together."""
    torch = _torch()
    ws = _ptr(ws, "ws", torch.uint8, numel=moonep_grad_norm_workspace_bytes(grads))
    norm = _ptr(norm, "norm", torch.float32, (1,))
    _check(_lib().moonep_grad_norm(*grads._arrays(), ws, norm, _stream(stream)), "moonep_grad_norm")


def moonep_grad_clip(grads: GradList, norm, max_norm, stream=None) -> None:
    """Scales the gradients in place by max_norm / norm[0] where norm[0] is larger than max_norm."""
    norm = _ptr(norm, "norm", _torch().float32, (1,))
    _check(_lib().moonep_grad_clip(*grads._arrays(), norm, float(max_norm), _stream(stream)), "moonep_grad_clip")


def _matrix_code(Kin: int, N: int) -> int:
    return _lib().moonep_quantize_w4(1, Kin, N, None, None, None, None)


@functools.lru_cache(maxsize=1024)
def moonep_w4_code_bytes(Kin: int, N: int) -> int:
    return _bytes(_lib().moonep_w4_code_bytes(Kin, N), "moonep_w4_code_bytes", lambda: _matrix_code(Kin, N))


@functools.lru_cache(maxsize=1024)
def moonep_w4_scale_bytes(Kin: int, N: int) -> int:
    return _bytes(_lib().moonep_w4_scale_bytes(Kin, N), "moonep_w4_scale_bytes", lambda: _matrix_code(Kin, N))


def moonep_quantize_w4(w, codes, scales, stream=None) -> None:
    """Quantises w [E, Kin, N] bf16 to 4 bits: codes [E, moonep_w4_code_bytes(Kin, N)] and scales
    [E, moonep_w4_scale_bytes(Kin, N)], both uint8."""
    torch = _torch()
    pw = _ptr(w, "w", torch.bfloat16)
    if w.dim() != 3:
        raise ValueError(f"w must have shape (E, Kin, N), got {tuple(w.shape)}")
    E, Kin, N = w.shape
    args = (pw, _ptr(codes, "codes", torch.uint8, (E, moonep_w4_code_bytes(Kin, N))),
            _ptr(scales, "scales", torch.uint8, (E, moonep_w4_scale_bytes(Kin, N))))
    _check(_lib().moonep_quantize_w4(E, Kin, N, *args, _stream(stream)), "moonep_quantize_w4")


def moonep_w4_ffn_workspace_bytes(d: Dims) -> int:
    return _dims_bytes("moonep_w4_ffn_workspace_bytes", bytes(d))


def moonep_w4_ffn(d: Dims, topk, gates, x, w13_codes, w13_scales, w2_codes, w2_scales, ws, out, stream=None) -> None:
    """out [R, S, H] = the gated sum of each token's experts' FFN, weights in 4 bits (moonep_quantize_w4
    of w13 [E, H, 2I] and w2 [E, I, H]).  Ids outside [0, E) add nothing."""
    torch = _torch()
    u8, bf = torch.uint8, torch.bfloat16
    wsb = moonep_w4_ffn_workspace_bytes(d)
    args = (
        _ptr(topk, "topk", torch.int32, (d.R, d.S, d.K)),
        _ptr(gates, "gates", torch.float32, (d.R, d.S, d.K)),
        _ptr(x, "x", bf, (d.R, d.S, d.H)),
        _ptr(w13_codes, "w13_codes", u8, (d.E, moonep_w4_code_bytes(d.H, 2 * d.I))),
        _ptr(w13_scales, "w13_scales", u8, (d.E, moonep_w4_scale_bytes(d.H, 2 * d.I))),
        _ptr(w2_codes, "w2_codes", u8, (d.E, moonep_w4_code_bytes(d.I, d.H))),
        _ptr(w2_scales, "w2_scales", u8, (d.E, moonep_w4_scale_bytes(d.I, d.H))),
        _ptr(ws, "ws", u8, numel=wsb),
        _ptr(out, "out", bf, (d.R, d.S, d.H)),
    )
    _check(_lib().moonep_w4_ffn(ctypes.byref(d), *args, _stream(stream)), "moonep_w4_ffn")
