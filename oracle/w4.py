"""Definitions of the 4-bit products in 64 bits (test infrastructure; shares nothing with the library).

Plain torch on any device, written from the formulas: the order of packed codes, the rule that makes codes and scales
of a matrix, and the product with group scales and zero points.
"""
from __future__ import annotations

import torch

CHUNK = 128


def row_bytes(K: int) -> int:
    return (K + CHUNK - 1) // CHUNK * 64


def _places(K: int, device) -> tuple[torch.Tensor, torch.Tensor]:
    """Of every value of a row: the byte that holds its code, and whether it is the byte's upper half."""
    k = torch.arange(K, device=device)
    chunk, j, t, i = k // 128, k % 128 // 32, k % 32 // 8, k % 8
    bit = 4 * (i // 2) + 16 * (i % 2)
    return chunk * 64 + (4 * t + j) * 4 + bit // 8, bit % 8 == 4


def pack(codes: torch.Tensor) -> torch.Tensor:
    """Codes [N, K] (0..15) -> packed rows [N, row_bytes(K)]; zero where no value is."""
    N, K = codes.shape
    out = torch.zeros((N, row_bytes(K)), dtype=torch.uint8, device=codes.device)
    byte, upper = _places(K, codes.device)
    out[:, byte[~upper]] = codes[:, ~upper].to(torch.uint8)
    out[:, byte[upper]] += codes[:, upper].to(torch.uint8) * 16
    return out


def unpack(wq: torch.Tensor, K: int) -> torch.Tensor:
    byte, upper = _places(K, wq.device)
    v = wq[:, byte]
    return torch.where(upper, v // 16, v % 16)


def _away(v: torch.Tensor) -> torch.Tensor:
    """Nearest whole number, halves away from zero (fp32)."""
    t = torch.trunc(v)
    return t + torch.sign(v) * ((v - t).abs() >= 0.5)


def quantize(w: torch.Tensor, group: int, scale_dtype, zero_points: bool):
    """(codes [N, K] uint8, scale [N, G], zeros [N, G] uint8 or None) of w [N, K], every operation in fp32."""
    N, K = w.shape
    G = (K + group - 1) // group
    codes = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    scale = torch.empty((N, G), dtype=scale_dtype, device=w.device)
    zeros = torch.empty((N, G), dtype=torch.uint8, device=w.device) if zero_points else None
    most = torch.finfo(scale_dtype).max
    for g in range(G):
        v = w[:, g * group:(g + 1) * group].float()
        odd = ~torch.isfinite(v).all(dim=1)
        v = torch.where(odd[:, None], torch.zeros_like(v), v)
        lo, hi = v.amin(1).clamp(max=0.0), v.amax(1).clamp(min=0.0)
        # (tensors as divisors: torch multiplies by the reciprocal of a number on a GPU)
        d = (hi - lo) / torch.full_like(lo, 15.0) if zero_points else torch.maximum(hi, -lo) / torch.full_like(lo, 7.0)
        s = torch.clamp(d.to(scale_dtype).double(), max=most).to(scale_dtype)
        sf = s.float()
        flat = sf == 0
        one = torch.where(flat, torch.ones_like(sf), sf)
        if zero_points:
            z = torch.where(flat, torch.zeros_like(sf), _away(-lo / one).clamp(max=15.0))
            zeros[:, g] = torch.where(odd, torch.zeros_like(z), z).to(torch.uint8)
        else:
            z = torch.full_like(sf, 8.0)
        q = _away(v / one[:, None]) + z[:, None]
        q = torch.where(flat[:, None], z[:, None], q).clamp(0.0 if zero_points else 1.0, 15.0)
        q = torch.where(odd[:, None], (torch.zeros_like(z) if zero_points else z)[:, None], q)
        codes[:, g * group:(g + 1) * group] = q.to(torch.uint8)
        scale[:, g] = torch.where(odd, torch.full_like(sf, float("nan")).to(scale_dtype), s)
    return codes, scale, zeros


def _spread(t: torch.Tensor, group: int, K: int) -> torch.Tensor:
    return t.double().repeat_interleave(group, dim=1)[:, :K]


def linear(x, x_scale, codes, scale, zeros, group, bias=None):
    """(y [T, N], terms [T, N], rest [T, N]) in 64 bits: the product, the sum of its terms' sizes with the codes taken
    as they are (|x| s (q + z)), and that of the chunks' largest activations with the weights' sizes."""
    K = codes.shape[1]
    s = _spread(scale, group, K)
    z = torch.full_like(s, 8.0) if zeros is None else _spread(zeros, group, K)
    q = codes.double()
    w = (q - z) * s
    xd = x.double()
    f = torch.ones(x.shape[0], 1, dtype=torch.float64, device=x.device) if x_scale is None else x_scale.double()[:, None]
    y = (xd @ w.T) * f
    terms = (xd.abs() @ ((q + z) * s.abs()).T) * f.abs()
    pad = -K % CHUNK
    xa = torch.nn.functional.pad(xd.abs(), (0, pad)).view(x.shape[0], -1, CHUNK).amax(2)
    wa = torch.nn.functional.pad(w.abs(), (0, pad)).view(codes.shape[0], -1, CHUNK).sum(2)
    rest = (xa @ wa.T) * f.abs()
    if bias is not None:
        y = y + bias.double()
        terms = terms + bias.double().abs()
    return y, terms, rest
