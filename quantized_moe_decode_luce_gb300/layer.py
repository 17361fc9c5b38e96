"""One MoE-FFN decode step through the C ABI, with torch-owned buffers.

:class:`MoEStep` allocates (once, with torch) every intermediate buffer of
the step for a fixed token count and runs the five calls of the step in the
pages' order on one stream: route select + weights, q8_1 quantization of
the FFN input, expert grouping (one fused launch for the first three when
it fits one CTA), gate/up pair + SwiGLU, down + combine.
Allocation is torch's; all arithmetic is in libluce_moe's kernels.

:class:`LinearI8` and :class:`LinearW4` are projections with their int8 or 4-bit
weights, :class:`GreedyHead` and :class:`SampleHead` the end of a decode or
verify step: final norm, vocabulary product, penalties and masks, greedy or
drawn tokens.
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


class LinearW4:
    """A projection of 4-bit weights with a scale, and optionally a zero point, per `group` values of a channel:
    wq [N, row bytes] packed, w_scale [N, ceil(K / group)] fp16 or bf16, zeros of its shape or None, bias [N] or None."""

    def __init__(self, wq: torch.Tensor, w_scale: torch.Tensor, K: int, group: int, zeros: torch.Tensor | None = None,
                 bias: torch.Tensor | None = None):
        if wq.shape[1] != B.w4_row_bytes(K):
            raise ValueError(f"rows of {K} codes take {B.w4_row_bytes(K)} bytes, got {wq.shape[1]}")
        self.wq, self.w_scale, self.zeros, self.bias = wq, w_scale, zeros, bias
        self.N, self.K, self.group = wq.shape[0], K, group

    @classmethod
    def from_float(cls, w: torch.Tensor, group: int = 128, zero_points: bool = False, scale_dtype=torch.float16,
                   bias: torch.Tensor | None = None) -> "LinearW4":
        """Quantizes w [N, K] (fp32, bf16 or fp16) by the rule of luce_quantize_w4."""
        N, K = w.shape
        shape = (N, -(-K // group))
        wq = torch.empty((N, B.w4_row_bytes(K)), dtype=torch.uint8, device=w.device)
        scale = torch.empty(shape, dtype=scale_dtype, device=w.device)
        zeros = torch.empty(shape, dtype=torch.uint8, device=w.device) if zero_points else None
        B.luce_quantize_w4(w, group, wq, scale, zeros)
        return cls(wq, scale, K, group, zeros, bias)

    @classmethod
    def from_codes(cls, codes: torch.Tensor, w_scale: torch.Tensor, group: int, zeros: torch.Tensor | None = None,
                   bias: torch.Tensor | None = None) -> "LinearW4":
        """Codes [N, K] of any origin, a byte each."""
        N, K = codes.shape
        wq = torch.empty((N, B.w4_row_bytes(K)), dtype=torch.uint8, device=codes.device)
        B.luce_pack_w4(codes, wq)
        return cls(wq, w_scale, K, group, zeros, bias)

    def run(self, x, x_scale, out, stream=None) -> torch.Tensor:
        """x [T, K] int8 with x_scale [T], or fp32, bf16 or fp16 with None."""
        if x.shape[-1] != self.K:  # (rows of packed codes do not tell K: they are whole chunks)
            raise ValueError(f"the projection takes {self.K} values, got {x.shape[-1]}")
        B.luce_linear_w4(x, x_scale, self.wq, self.w_scale, self.zeros, self.group, self.bias, out, stream)
        return out


class _Head:
    """What stands before the pick of a step's tokens, for R rows: final norm, vocabulary product (LinearI8 or LinearW4),
    penalties and masks."""

    def __init__(self, R: int, gamma: torch.Tensor, eps: float, head):
        if head.K != gamma.numel():
            raise ValueError(f"the head takes {head.K} values, the norm gives {gamma.numel()}")
        dev = gamma.device
        self.R, self.gamma, self.eps, self.head = R, gamma, float(eps), head
        self.q = torch.empty((R, head.K), dtype=torch.int8, device=dev)
        self.scale = torch.empty(R, dtype=torch.float32, device=dev)
        self.logits = torch.empty((R, head.N), dtype=torch.float32, device=dev)

    def _run_logits(self, x, residual, x_sum, stream, process) -> None:
        if residual is None and x_sum is not None:
            raise ValueError("x_sum is the sum with a residual, and there is none")
        if residual is not None:
            B.luce_add_rmsnorm_i8(x, residual, x_sum, self.gamma, self.eps, self.q, self.scale, stream)
        else:
            B.luce_rmsnorm_i8(x, self.gamma, self.eps, self.q, self.scale, stream)
        self.head.run(self.q, self.scale, self.logits, stream)
        if process:
            B.luce_logits_process(self.logits, self.logits, stream=stream, **process)


class GreedyHead(_Head):
    """The end of a step for R rows (tokens, or the columns of a verify step): the residual sum's
    RMS norm in int8, the vocabulary product, penalties, biases and masks, the greedy tokens.

    Owns every buffer, so one head runs on one stream at a time (a captured graph of it among them);
    `run` makes four calls and returns (idx [R] int32, val [R] fp32).

    val says whether a row has a token: it is -inf where the row's mask allows nothing (idx is 0), and
    NaN or -inf where the row of x (or of the sum) holds a NaN or an infinity, which makes all its logits
    NaN that are not masked (idx then is in range, and no pick)."""

    def __init__(self, R: int, gamma: torch.Tensor, eps: float, head):
        super().__init__(R, gamma, eps, head)
        self.argmax = Argmax(R, head.N, device=gamma.device)

    def run(self, x, residual=None, x_sum=None, stream=None, **process):
        """x (+ residual) [R, K]; `process` are the keyword arguments of luce_logits_process.
        Runs on the head's device, on its current stream unless one is given."""
        dev = self.q.get_device()
        if dev != torch.cuda.current_device():
            with torch.cuda.device(dev):
                return self.run(x, residual, x_sum, stream, **process)
        self._run_logits(x, residual, x_sum, stream, process)
        return self.argmax.run(self.logits, stream)


class SampleHead(_Head):
    """GreedyHead with a draw at its end: a token per row from its logits, at the row's temperature and with its top-k,
    top-p and min-p, by a given random number.

    `run` returns (idx [R] int32, prob [R] fp32); prob is 0 where the row's mask allows nothing (idx is 0), and NaN
    where the row of x (or of the sum) holds a NaN or an infinity (idx is 0 as well), unless the mask allows nothing."""

    def __init__(self, R: int, gamma: torch.Tensor, eps: float, head):
        super().__init__(R, gamma, eps, head)
        self.idx = torch.empty(R, dtype=torch.int32, device=gamma.device)
        self.prob = torch.empty(R, dtype=torch.float32, device=gamma.device)

    def run(self, x, u, residual=None, x_sum=None, temperature=None, top_k=None, top_p=None, min_p=None, stream=None,
            **process):
        """x (+ residual) [R, K]; u [R] in [0, 1) and the four per-row parameters as luce_sample takes them;
        `process` are the keyword arguments of luce_logits_process.
        Runs on the head's device, on its current stream unless one is given."""
        dev = self.q.get_device()
        if dev != torch.cuda.current_device():
            with torch.cuda.device(dev):
                return self.run(x, u, residual, x_sum, temperature, top_k, top_p, min_p, stream, **process)
        self._run_logits(x, residual, x_sum, stream, process)
        B.luce_sample(self.logits, u, self.idx, self.prob, temperature, top_k, top_p, min_p, stream)
        return self.idx, self.prob
