"""Plain definitions of the int8 decode-head operators, on the CPU in 64 bits.

Written from the formulas in include/luce_moe.h: sums and products in 64 bits
(or whole numbers), rounded to 32 bits at exactly the places where the
formulas round.  Where a formula rounds every step the results are bits to
compare with; the row scale holds a sum of squares, whose order is free, and
is compared within a bound.  Test infrastructure only; shares nothing with
the CUDA library.
"""
from __future__ import annotations

import math

import torch

f64, f32 = torch.float64, torch.float32
INF = math.inf


def _fl(v: torch.Tensor) -> torch.Tensor:
    """Rounded to fp32, held in 64 bits."""
    return v.to(f32).to(f64)


def round_half_away(v: torch.Tensor) -> torch.Tensor:
    return torch.sign(v) * torch.floor(v.abs() + 0.5)  # exact: v holds 24 bits, the sum at most 53


def rows_i8(x: torch.Tensor, gamma=None, eps: float = 0.0, residual=None):
    """(q int8, scale fp64, x_sum in x's type or None) of rows x (+ residual)."""
    s = None
    if residual is not None:
        s = (x.to(f32) + residual.to(f32)).to(x.dtype)  # one fp32 addition, rounded to the type
        x = s
    v = x.to(f64)
    p = v if gamma is None else _fl(v * gamma.to(f64))
    finite = torch.isfinite(p).all(dim=1)
    m = p.abs().amax(dim=1)
    d = _fl(m / 127.0)
    live = finite & (d > 0)
    dd = torch.where(live, d, torch.ones_like(d))[:, None]
    q = round_half_away(_fl(torch.where(live[:, None], p, torch.zeros_like(p)) / dd)).clamp(-127, 127)
    scale = d
    if gamma is not None:
        r2 = v.square().mean(dim=1) + float(torch.tensor(eps, dtype=f32))
        scale = torch.where(d > 0, d / torch.sqrt(r2), d)  # (a row whose d is zero has scale zero, without 0 / 0)
    scale = torch.where(finite, scale, torch.full_like(scale, math.nan))
    return q.to(torch.int8), scale, s


def linear_i8(xq, x_scale, wq, w_scale, bias, dtype):
    """out of luce_linear_i8, bit for bit."""
    isum = xq.to(f64) @ wq.to(f64).t()  # whole numbers below 2^53: exact
    y = _fl(_fl(isum) * _fl(x_scale.to(f64)[:, None] * w_scale.to(f64)[None, :]))
    if bias is not None:
        y = _fl(y + bias.to(f64))
    return y.to(f32).to(dtype)


def logits_process(logits, hist=None, hist_len=None, prompt_len=None, repetition=None, frequency=None, presence=None,
                   bias_ids=None, bias_vals=None, mask=None, mask_rows=None):
    """out of luce_logits_process, bit for bit, token by token; CPU tensors or None."""
    out = logits.to(f64).clone()
    R, V = out.shape
    for r in range(R):
        if hist is not None:
            n = min(max(int(hist_len[r]), 0), hist.shape[1])
            np_ = int(prompt_len[r]) if prompt_len is not None else 0
            counts = {}
            for i in range(n):
                v = int(hist[r, i])
                if 0 <= v < V:
                    counts[v] = counts.get(v, 0) + (1 if i >= np_ else 0)
            rep = repetition[r].to(f64) if repetition is not None else torch.tensor(1.0, dtype=f64)
            fr = frequency[r].to(f64) if frequency is not None else torch.tensor(0.0, dtype=f64)
            pr = presence[r].to(f64) if presence is not None else torch.tensor(0.0, dtype=f64)
            for v, c in counts.items():
                l = out[r, v]
                l = _fl(l / rep) if l > 0 else _fl(l * rep)
                if c:
                    l = _fl(l - _fl(_fl(_fl(torch.tensor(float(c), dtype=f64)) * fr) + pr))
                out[r, v] = l
        if bias_ids is not None:
            last = {int(v): j for j, v in enumerate(bias_ids[r]) if 0 <= int(v) < V}
            for v, j in last.items():
                out[r, v] = _fl(out[r, v] + bias_vals[r, j].to(f64))
        if mask is not None:
            m = int(mask_rows[r]) if mask_rows is not None else r
            if 0 <= m < mask.shape[0]:
                words = mask[m].to(torch.int64) & 0xFFFFFFFF
                v = torch.arange(V)
                allowed = (words[v // 32] >> (v % 32)) & 1
                out[r, allowed == 0] = -INF
    return out.to(f32)
