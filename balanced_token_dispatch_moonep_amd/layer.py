"""Static-shape buffers and call order for one balanced expert-parallel MoE layer.

The MoonEP pages describe one pass as: router output -> planning -> (weight prefetch
and dispatch) -> grouped GEMM -> combine, then reduce_grad of replica gradients in
training [thakicloud.com "The Busiest Rank Sets Your Step Time", "What the technique
is" flowchart].  Every buffer has a fixed shape (the receive buffer is always S*K rows
per rank), so it is allocated once and reused each step with no host synchronisation
[twodots.gr "MoonEP balances AI experts in MoE models", architecture].

This module only allocates device memory through torch and calls the library's entry
points in that order; all arithmetic runs in the HIP kernels.
"""
from __future__ import annotations

import torch

from . import (Dims, GradList, moonep_combine, moonep_dispatch, moonep_grad_clip, moonep_grad_norm,
               moonep_grad_norm_workspace_bytes, moonep_grouped_ffn, moonep_grouped_ffn_backward,
               moonep_layer_norm, moonep_layer_norm_backward, moonep_layer_norm_workspace_bytes,
               moonep_plan, moonep_plan_workspace_bytes, moonep_prefetch, moonep_quantize_w4,
               moonep_reduce_grad, moonep_w4_code_bytes, moonep_w4_ffn, moonep_w4_ffn_workspace_bytes,
               moonep_w4_scale_bytes, NSTATS)


def _slot_shapes(R, B, H, I):
    return (R, B, H, 2 * I), (R, B, I, H)


def _nbytes(shape, itemsize):
    n = itemsize
    for v in shape:
        n *= v
    return n


def _within(x, buf) -> bool:
    """Whether x begins in the memory of buf, a whole allocation."""
    return 0 <= x.data_ptr() - buf.data_ptr() < buf.nbytes


def _aligned(t):
    """t, or where its rows begin between 16-byte addresses (later tokens of a batch) a copy."""
    return t if t.data_ptr() % 16 == 0 else t.clone()


class MoonEPPool:
    """Process-global prefetch slots shared by every layer [AT, TL;DR; TD, memory contract].

    Layers run one after another, so one set of B weight slots per rank (and, in training,
    one fp32 reduce buffer [R, B, ...]) serves all of them: the extra memory does not grow
    with depth.  A layer whose slots were overwritten by later layers prefetches its replicas
    again before its backward (its plan stays in its own workspace).
    """

    def __init__(self, R, B, H, I, training=False, device="cuda"):
        dev = torch.device(device)
        s13, s2 = _slot_shapes(R, B, H, I)
        self.R, self.B, self.H, self.I, self.training = R, B, H, I, training
        self.w13_slot = torch.zeros(s13, dtype=torch.bfloat16, device=dev) if B else None
        self.w2_slot = torch.zeros(s2, dtype=torch.bfloat16, device=dev) if B else None
        self.dw13_red = torch.zeros(s13, dtype=torch.float32, device=dev) if B and training else None
        self.dw2_red = torch.zeros(s2, dtype=torch.float32, device=dev) if B and training else None
        self.owner = None     # the layer whose replicas the slots hold

    @staticmethod
    def nbytes(R, B, H, I, training=False) -> dict:
        s13, s2 = _slot_shapes(R, B, H, I)
        slots = _nbytes(s13, 2) + _nbytes(s2, 2) if B else 0
        red = _nbytes(s13, 4) + _nbytes(s2, 4) if B and training else 0
        return {"prefetch": slots, "reduce": red, "total": slots + red}


def stack_slot_bytes(R, B, H, I, layers, pooled, training=False) -> int:
    """Bytes of prefetch slots (and reduce buffers) for `layers` layers, pooled or one set each."""
    per = MoonEPPool.nbytes(R, B, H, I, training)["total"]
    return per if pooled else layers * per


class MoonEPLayer:
    """One emulated EP layer: R ranks as R static partitions of one GPU's memory.

    ``w13`` [E, H, 2I] and ``w2`` [E, I, H] are the home expert weights (bf16, on the
    device).  With ``I == 0`` the layer has no expert FFN (identity experts): only
    planning, dispatch and combine run.

    With ``norm_weight`` [H] (float32; ``norm_bias`` [H] or None) the rows are layer-normed before
    they are dispatched, and ``backward`` returns the gradient of the rows before the norm; it also
    writes ``dnorm_weight`` and ``dnorm_bias``.  A router that reads the normed rows calls ``norm(x)``
    itself; ``forward`` given what that returned does not norm again, and given a copy of it does not
    with ``normed=True``.  ``backward`` goes back to the rows of the last ``norm(x)``.
    """

    def __init__(self, dims: Dims, w13=None, w2=None, training: bool = False, device="cuda", pool=None,
                 norm_weight=None, norm_bias=None, norm_eps: float = 1e-5):
        if norm_bias is not None and norm_weight is None:
            raise ValueError("norm_bias needs norm_weight")
        self.d = dims
        self.training = training
        self.pool = pool
        dev = torch.device(device)
        self.device = dev
        R, E, B, S, K, H, I = dims.R, dims.E, dims.B, dims.S, dims.K, dims.H, dims.I
        M = R * S * K
        rt = torch.float32 if dims.flags & 2 else torch.bfloat16
        i32 = torch.int32
        self.ws = torch.empty(moonep_plan_workspace_bytes(dims), dtype=torch.uint8, device=dev)
        self.cu = torch.empty((R, E + B + 1), dtype=i32, device=dev)
        self.dest = torch.empty((R, S, K), dtype=i32, device=dev)
        self.stats = torch.empty((NSTATS,), dtype=i32, device=dev)
        self.recv = torch.empty((M, H), dtype=rt, device=dev)
        self.out = torch.empty((R, S, H), dtype=rt, device=dev)
        self.w13, self.w2 = w13, w2
        self.norm_weight, self.norm_bias, self.norm_eps = norm_weight, norm_bias, norm_eps
        if norm_weight is not None:
            f32 = torch.float32
            self.normed = torch.empty((R, S, H), dtype=rt, device=dev)
            self.mean = torch.empty((R * S,), dtype=f32, device=dev) if training else None
            self.rstd = torch.empty((R * S,), dtype=f32, device=dev) if training else None
            self.x = None         # the rows of the last norm(), which its backward reads
            if training:
                self.dnorm_weight = torch.zeros((H,), dtype=f32, device=dev)
                self.dnorm_bias = torch.zeros((H,), dtype=f32, device=dev) if norm_bias is not None else None
                self.norm_ws = torch.empty(moonep_layer_norm_workspace_bytes(dims), dtype=torch.uint8, device=dev)
                self.dx_in = torch.empty((R, S, H), dtype=rt, device=dev)
        if I > 0:
            bf = torch.bfloat16
            if pool is not None:
                if (pool.R, pool.B, pool.H, pool.I) != (R, B, H, I) or (training and not pool.training):
                    raise ValueError("the pool's shapes do not match the layer")
                self.w13_slot, self.w2_slot = pool.w13_slot, pool.w2_slot
            else:
                self.w13_slot = torch.zeros((R, B, H, 2 * I), dtype=bf, device=dev) if B else None
                self.w2_slot = torch.zeros((R, B, I, H), dtype=bf, device=dev) if B else None
            self.gu = torch.empty((M, 2 * I), dtype=bf, device=dev)
            self.act = torch.empty((M, I), dtype=bf, device=dev)
            self.y = torch.empty((M, H), dtype=bf, device=dev)
            if training:
                f32 = torch.float32
                self.dy = torch.empty((M, H), dtype=bf, device=dev)
                self.drecv = torch.empty((M, H), dtype=bf, device=dev)
                self.dx = torch.empty((R, S, H), dtype=bf, device=dev)
                self.dw13 = torch.zeros((E, H, 2 * I), dtype=f32, device=dev)
                self.dw2 = torch.zeros((E, I, H), dtype=f32, device=dev)
                if pool is not None:
                    self.dw13_red, self.dw2_red = pool.dw13_red, pool.dw2_red
                else:
                    self.dw13_red = torch.zeros((R, B, H, 2 * I), dtype=f32, device=dev) if B else None
                    self.dw2_red = torch.zeros((R, B, I, H), dtype=f32, device=dev) if B else None
        else:
            self.y = self.recv          # identity experts

    # -- steps ---------------------------------------------------------------
    def norm(self, x):
        """Layer norm of the rows [R, S, H] (a static buffer, replaced by the next call); x must stay as
        it is until the backward."""
        if _within(x, self.normed):
            raise ValueError("norm of rows that norm() returned: it would write over what it reads")
        moonep_layer_norm(self.d, x, self.norm_weight, self.norm_bias, self.norm_eps, self.normed, self.mean,
                          self.rstd)
        self.x = x
        return self.normed

    def plan(self, topk):
        moonep_plan(self.d, topk, self.ws, self.cu, self.dest, self.stats)

    def prefetch(self):
        if self.d.I > 0 and self.d.B > 0:
            moonep_prefetch(self.d, self.ws, self.w13, self.w2, self.w13_slot, self.w2_slot)
            if self.pool is not None:
                self.pool.owner = self

    def dispatch(self, x):
        moonep_dispatch(self.d, self.dest, x, None, self.recv)

    def expert_ffn(self):
        if self.d.I > 0:
            moonep_grouped_ffn(self.d, self.ws, self.cu, self.recv, self.w13, self.w2,
                               self.w13_slot, self.w2_slot, self.gu, self.act, self.y)

    def combine(self, gates):
        moonep_combine(self.d, self.dest, self.y, gates, self.out)

    def forward(self, x, topk, gates, normed=False):
        """Returns the [R, S, H] output (a view of a static buffer, replaced by the next call).

        ``normed``: x is a copy of what norm() returned last (what it returned itself need not say so)."""
        if self.norm_weight is not None:
            if not normed and not _within(x, self.normed):
                x = self.norm(x)
            elif self.training and self.x is None:
                raise ValueError("normed rows without a call of norm(), whose rows the backward goes back to")
        self.plan(topk)
        self.prefetch()
        self.dispatch(x)
        self.expert_ffn()
        self.combine(gates)
        return self.out

    def backward(self, dout, gates):
        """Gradient of forward(): returns dx [R, S, H]; writes dw13 / dw2 (fp32; added to them
        with MOONEP_GRAD_ACCUM), slot replicas' gradients reduced into their home experts.

        The saved gate|up activations are overwritten by their gradients."""
        assert self.training and self.d.I > 0
        if self.pool is not None and self.pool.owner is not self:
            self.prefetch()       # a later layer reused the shared slots
        moonep_dispatch(self.d, self.dest, dout, gates, self.dy)
        moonep_grouped_ffn_backward(self.d, self.ws, self.cu, self.recv, self.gu, self.act, self.dy,
                                    self.w13, self.w2, self.w13_slot, self.w2_slot, self.drecv,
                                    self.dw13, self.dw2, self.dw13_red, self.dw2_red)
        moonep_combine(self.d, self.dest, self.drecv, None, self.dx)
        moonep_reduce_grad(self.d, self.ws, self.dw13, self.dw2, self.dw13_red, self.dw2_red)
        if self.norm_weight is None:
            return self.dx
        moonep_layer_norm_backward(self.d, self.dx, self.x, self.norm_weight, self.mean, self.rstd, self.dx_in,
                                   self.dnorm_weight, self.dnorm_bias, self.norm_ws)
        return self.dx_in

    # -- round the step --------------------------------------------------------
    def grads(self) -> list:
        """The weights' gradients that backward() leaves behind."""
        if not self.training or self.d.I == 0:
            raise ValueError("only a training layer with experts has gradients")
        norm = [self.dnorm_weight, self.dnorm_bias] if self.norm_weight is not None else []
        return [g for g in [self.dw13, self.dw2, *norm] if g is not None]

    def decoder(self, max_tokens: int) -> "W4Experts":
        """The same norm and experts for decoding, with 4-bit weights made from the present ones."""
        if self.d.I == 0:
            raise ValueError("a layer without experts has nothing to decode with")
        return W4Experts(self.w13, self.w2, self.d.K, max_tokens, self.norm_weight, self.norm_bias, self.norm_eps)


class GradClipper:
    """Clips the gradients of one or more layers by their global norm."""

    def __init__(self, layers):
        self.list = GradList(g for layer in layers for g in layer.grads())
        dev = self.list.device
        self.ws = torch.empty(moonep_grad_norm_workspace_bytes(self.list), dtype=torch.uint8, device=dev)
        self.norm = torch.empty((1,), dtype=torch.float32, device=dev)

    def clip(self, max_norm):
        """Scales the gradients so that their norm is at most max_norm; returns the norm they had, a
        [1] float32 tensor on the GPU (a static buffer, replaced by the next call)."""
        moonep_grad_norm(self.list, self.ws, self.norm)
        moonep_grad_clip(self.list, self.norm, max_norm)
        return self.norm


class W4Experts:
    """A layer's experts for decoding: up to max_tokens tokens a call, weights in 4 bits.

    ``w13`` [E, H, 2I] and ``w2`` [E, I, H] bf16 are quantised here, once, and not kept.  All buffers
    are static, so a call can be captured; a call replaces the output of the one before.
    """

    def __init__(self, w13, w2, K: int, max_tokens: int, norm_weight=None, norm_bias=None, norm_eps: float = 1e-5):
        E, H, I = w13.shape[0], w13.shape[1], w2.shape[1]
        dev, u8 = w13.device, torch.uint8
        self.E, self.H, self.I, self.K, self.max_tokens = E, H, I, K, max_tokens
        self.norm_weight, self.norm_bias, self.norm_eps = norm_weight, norm_bias, norm_eps
        self.packed = []
        for w, kin, n in ((w13, H, 2 * I), (w2, I, H)):
            codes = torch.empty((E, moonep_w4_code_bytes(kin, n)), dtype=u8, device=dev)
            scales = torch.empty((E, moonep_w4_scale_bytes(kin, n)), dtype=u8, device=dev)
            moonep_quantize_w4(w, codes, scales)
            self.packed += [codes, scales]
        self.ws = torch.empty(moonep_w4_ffn_workspace_bytes(self._dims(max_tokens)), dtype=u8, device=dev)
        self.normed = torch.empty((max_tokens, H), dtype=torch.bfloat16, device=dev)
        self.out = torch.empty((max_tokens, H), dtype=torch.bfloat16, device=dev)

    def _dims(self, T):
        return Dims.make(1, self.E, 0, T, self.K, self.H, self.I)

    def norm(self, x):
        """Layer norm of the tokens x [T, H] (a view of a static buffer, replaced by the next call)."""
        if _within(x, self.normed):
            raise ValueError("norm of rows that norm() returned: it would write over what it reads")
        T = x.shape[0]
        d = Dims.make(1, 1, 0, T, 1, self.H)
        moonep_layer_norm(d, x.unsqueeze(0), self.norm_weight, self.norm_bias, self.norm_eps,
                          self.normed[:T].unsqueeze(0))
        return self.normed[:T]

    def forward(self, x, topk, gates, normed=False):
        """x [T, H] bf16, topk [T, K] int32 (-1: nothing), gates [T, K] float32 -> [T, H] bf16 (a view of a
        static buffer).  x is what comes before the norm, or what norm() returned or some of its tokens,
        or with ``normed`` a copy of such."""
        T = x.shape[0]
        if not 1 <= T <= self.max_tokens:
            raise ValueError(f"{T} tokens: this decoder takes 1 to {self.max_tokens}")
        if self.norm_weight is not None and not normed and not _within(x, self.normed):
            x = self.norm(x)
        d = self._dims(T)
        ws = self.ws[:moonep_w4_ffn_workspace_bytes(d)]
        out = self.out[:T]
        moonep_w4_ffn(d, _aligned(topk).unsqueeze(0), _aligned(gates).unsqueeze(0), x.unsqueeze(0), *self.packed, ws,
                      out.unsqueeze(0))
        return out
