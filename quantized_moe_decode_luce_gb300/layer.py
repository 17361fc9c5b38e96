"""One MoE-FFN decode step through the C ABI, with torch-owned buffers.

:class:`MoEStep` allocates (once, with torch) every intermediate buffer of
the step for a fixed token count and runs the five calls of the step in the
pages' order on one stream: route select + weights, q8_1 quantization of
the FFN input, expert grouping (one fused launch for the first three when
it fits one CTA), gate/up pair + SwiGLU, down + combine.
Allocation is torch's; all arithmetic is in libluce_moe's kernels.

:class:`LinearI8` is an int8 projection with its weights, :class:`GreedyHead`
the end of a decode or verify step: final norm, vocabulary product, penalties
and masks, greedy tokens.
"""
from __future__ import annotations

import torch

from . import binding as B
from .workloads import QK, Q8_1_BYTES


class MoEStep:
    def __init__(self, T: int, H: int, I: int, E: int, k: int, shared: bool, clamp: float, device="cuda"):
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.shared, self.clamp = shared, float(clamp)
        dev = torch.device(device)
        rows = T * k + (T if shared else 0)
        self.ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.weights = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.xq = torch.empty((T, H // QK, Q8_1_BYTES), dtype=torch.uint8, device=dev)
        self.counts = torch.empty(E, dtype=torch.int32, device=dev)
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        self.routes = torch.empty(max(1, T * k), dtype=torch.int32, device=dev)
        self.h = torch.empty((max(1, rows), I), dtype=torch.float32, device=dev)
        self.hq = torch.empty((max(1, rows), I // QK, Q8_1_BYTES), dtype=torch.uint8, device=dev)
        self.out = torch.empty((T, H), dtype=torch.float32, device=dev)
        # luce_moe_layer's workspace: its barrier count (first 8 bytes, zero) and scratch
        self.workspace = torch.zeros(B.luce_moe_layer_workspace_bytes(T, k, H, I), dtype=torch.uint8, device=dev)
        self.fused_prep = True
        # "layer": luce_moe_layer -- one cooperative launch for T <= 8, T*k <= 64,
        # E <= 256 (bitwise the results of the split launches), the grouped
        # tensor-core path for more tokens; "split": the separate launches.
        self.path = "split" if (T <= 8 and T * k <= 64 and E > 256) else "layer"

    def run(self, layer, x, logits, bias=None, stream=None, out=None) -> torch.Tensor:
        """layer: object with wg, wu, wd (+ wsg, wsu, wsd) uint8 CUDA tensors.
        Writes the layer output into `out` (default: this step's own buffer)."""
        out = self.out if out is None else out
        T, H, I, E, k = self.T, self.H, self.I, self.E, self.k
        wsg = layer.wsg if self.shared else None
        wsu = layer.wsu if self.shared else None
        wsd = layer.wsd if self.shared else None
        if self.path == "layer":
            try:
                B.luce_moe_layer(logits, bias, x, k, I, layer.wg, layer.wu, layer.wd, wsg, wsu, wsd, self.clamp,
                                 self.ids, self.weights, self.xq, self.counts, self.offsets, self.routes, self.h,
                                 self.hq, out, self.workspace, stream)
                return out
            except B.LuceError as err:
                if err.status != B.LUCE_ERR_UNSUPPORTED:
                    raise
                self.path = "split"  # beyond the one-launch limits: the split launches (nothing ran)
        if self.fused_prep:
            B.luce_moe_prep(logits, bias, x, k, self.ids, self.weights, self.xq, self.counts, self.offsets,
                            self.routes, stream)
        else:
            B.luce_route_topk(logits, bias, k, self.ids, self.weights, stream)
            B.luce_quantize_q8_1(x, self.xq, stream)
            B.luce_moe_group(self.ids, E, self.counts, self.offsets, self.routes, stream)
        B.luce_moe_glu_pair(layer.wg, layer.wu, wsg, wsu, self.xq, self.offsets, self.routes, T, k, E, H, I,
                            self.clamp, self.h, self.hq, 0, stream)
        B.luce_moe_down_combine(layer.wd, wsd, self.hq, self.ids, self.weights, self.offsets, self.routes,
                                T, k, E, H, I, out, 0, stream)
        return out


class Argmax:
    """Greedy argmax over [R, V] logits with its own zero-filled workspace."""

    def __init__(self, R: int, V: int, device="cuda"):
        self.R, self.V = R, V
        n = max(16, B.luce_argmax_workspace_bytes(R, V))
        self.workspace = torch.zeros(n, dtype=torch.uint8, device=device)
        self.idx = torch.empty(R, dtype=torch.int32, device=device)
        self.val = torch.empty(R, dtype=torch.float32, device=device)

    def run(self, logits, stream=None):
        B.luce_argmax(logits, self.idx, self.val, self.workspace, stream)
        return self.idx, self.val


class LinearI8:
    """An int8 projection: weights [N, K] with a scale per output channel, and an optional bias."""

    def __init__(self, wq: torch.Tensor, w_scale: torch.Tensor, bias: torch.Tensor | None = None):
        self.wq, self.w_scale, self.bias = wq, w_scale, bias
        self.N, self.K = wq.shape

    @classmethod
    def from_float(cls, w: torch.Tensor, bias: torch.Tensor | None = None) -> "LinearI8":
        """Quantizes w [N, K] (fp32, bf16 or fp16), a channel to a row, by the rule of luce_quantize_i8."""
        wq = torch.empty(w.shape, dtype=torch.int8, device=w.device)
        scale = torch.empty(w.shape[0], dtype=torch.float32, device=w.device)
        B.luce_quantize_i8(w, wq, scale)
        return cls(wq, scale, bias)

    def run(self, xq, x_scale, out, stream=None) -> torch.Tensor:
        B.luce_linear_i8(xq, x_scale, self.wq, self.w_scale, self.bias, out, stream)
        return out


class GreedyHead:
    """The end of a step for R rows (tokens, or the columns of a verify step): the residual sum's
    RMS norm in int8, the vocabulary product, penalties, biases and masks, the greedy tokens.

    Owns every buffer, so one head runs on one stream at a time (a captured graph of it among them);
    `run` makes four calls and returns (idx [R] int32, val [R] fp32).

    val says whether a row has a token: it is -inf where the row's mask allows nothing (idx is 0), and
    NaN or -inf where the row of x (or of the sum) holds a NaN or an infinity, which makes all its logits
    NaN that are not masked (idx then is in range, and no pick)."""

    def __init__(self, R: int, gamma: torch.Tensor, eps: float, head: LinearI8):
        if head.K != gamma.numel():
            raise ValueError(f"the head takes {head.K} values, the norm gives {gamma.numel()}")
        dev = gamma.device
        self.R, self.gamma, self.eps, self.head = R, gamma, float(eps), head
        self.q = torch.empty((R, head.K), dtype=torch.int8, device=dev)
        self.scale = torch.empty(R, dtype=torch.float32, device=dev)
        self.logits = torch.empty((R, head.N), dtype=torch.float32, device=dev)
        self.argmax = Argmax(R, head.N, device=dev)

    def run(self, x, residual=None, x_sum=None, stream=None, **process):
        """x (+ residual) [R, K]; `process` are the keyword arguments of luce_logits_process.
        Runs on the head's device, on its current stream unless one is given."""
        dev = self.q.get_device()
        if dev != torch.cuda.current_device():
            with torch.cuda.device(dev):
                return self.run(x, residual, x_sum, stream, **process)
        if residual is None and x_sum is not None:
            raise ValueError("x_sum is the sum with a residual, and there is none")
        if residual is not None:
            B.luce_add_rmsnorm_i8(x, residual, x_sum, self.gamma, self.eps, self.q, self.scale, stream)
        else:
            B.luce_rmsnorm_i8(x, self.gamma, self.eps, self.q, self.scale, stream)
        self.head.run(self.q, self.scale, self.logits, stream)
        if process:
            B.luce_logits_process(self.logits, self.logits, stream=stream, **process)
        return self.argmax.run(self.logits, stream)
