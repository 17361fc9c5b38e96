"""GPU: draws and 4-bit products at the ends of their ranges: top-p just below 1 over long flat tails, small
temperatures, activations and scales near fp32's smallest numbers, sums of bf16 activations for fp32 outputs."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import draw as D
from oracle import w4 as O
from quantized_moe_decode_luce_gb300 import binding as B
from test_gpu_head import _lib, _no_device_faults, bf16, f16, f32, gen  # noqa: F401 (the fixtures hold here)

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------- draws in whole units
# The weights of a row whose largest logit is 0, at temperature 1, are whole multiples of 2^-L, rounded down: 2^L for the
# largest. Where no weight is near a whole number (the library's are within 2^-29 of theirs) every sum is known, and so is
# every decision: nothing is left to a margin.
def units_of(l):
    V = l.size
    L = min(62, 63 - (V - 1).bit_length())
    with np.errstate(divide="ignore"):
        w = np.exp2(L + l.astype(np.float64) / math.log(2.0))
    rest = np.abs(w - np.rint(w))
    assert np.all((l == 0) | (w == 0) | (rest > 1e-6 * np.maximum(w, 1.0)))
    return np.where(l == 0, 1 << L, np.floor(w).astype(np.int64)).astype(np.int64)


def draw_in_units(l, us, top_p, top_k=0):
    """[(id, weight / total)] for every u."""
    w = units_of(l)
    order = np.lexsort((np.arange(l.size), -l))
    if 0 < top_k < l.size:
        order = order[:top_k]
    upto = np.cumsum(w[order])
    want = max(1, math.ceil(Fraction(float(np.float32(top_p))) * int(upto[-1])))
    ids = np.sort(order[upto - w[order] < want])
    upto = np.cumsum(w[ids])
    total, out = int(upto[-1]), []
    for u in us:
        f = float(np.float32(u))
        target = total - 1 if f >= 1 else math.floor(Fraction(f) * total)
        i = int(np.searchsorted(upto, target, side="right"))
        out.append((int(ids[i]), int(w[ids[i]]) / total))
    return out


def check_units(row, top_p, top_k=0, copies=1):
    """One row for every random number, and that `copies` times over, in one call; the same bits in ten calls."""
    us = [0.0, 0.25, 0.5, 0.999, 1.0 - 2.0 ** -23, 1.0 - 2.0 ** -24, 1.0] * copies
    want = draw_in_units(row.float().numpy(), us[:7], top_p, top_k) * copies
    R = len(us)
    l, u = row.cuda().expand(R, -1).contiguous(), torch.tensor(us, device="cuda")
    p = torch.full((R,), top_p, device="cuda")
    k = torch.full((R,), top_k, dtype=torch.int32, device="cuda") if top_k else None
    for _ in range(10):
        idx, prob = torch.full((R,), -9, dtype=torch.int32, device="cuda"), torch.full((R,), -9.0, device="cuda")
        B.luce_sample(l, u, idx, prob, None, k, p)
        torch.cuda.synchronize()
        assert idx.tolist() == [i for i, _ in want]
        # the weight and the total are rounded to fp32, and so is their quotient: 3 2^-24
        assert all(abs(a - q) <= q * 2.0 ** -22 for a, (_, q) in zip(prob.tolist(), want))


def tail_row(V, parts, first_at, seed):
    """A token at 0, and for each (n, w) n tokens whose weight is w units, at places of their own; no others."""
    L = min(62, 63 - (V - 1).bit_length())
    l = torch.full((V,), -math.inf)
    places = torch.randperm(V, generator=gen(seed))
    places = places[places != first_at]
    at = 0
    for n, w in parts:
        l[places[at:at + n]] = math.log(w) - L * math.log(2.0)
        at += n
    l[first_at] = 0.0
    return l


# The weights stand a little below whole numbers: counted by their real size, a bin holds fewer tokens than it does.
# (Clusters of 16 CTAs and of eight; CTAs of 512 threads for the first two, of 256 for the last two.)
@pytest.mark.parametrize("copies", [1, 3])
@pytest.mark.parametrize("first_at", [0, 77777, -1])
@pytest.mark.parametrize("V,parts,top_p", [
    (393216, [(1200, 3.95), (349000, 3.1)], 1.0 - 2.0 ** -24), (393216, [(1500, 3.97), (349400, 3.1)], 1.0 - 2.0 ** -24),
    (129280, [(518, 33.95), (127000, 33.05)], 1.0 - 2.0 ** -24), (129280, [(3000, 34.9), (125000, 33.9)], 1.0 - 2.0 ** -24)])
def test_top_p_over_a_flat_tail(V, parts, top_p, first_at, copies):
    check_units(tail_row(V, parts, first_at % V, 1), top_p, copies=copies)


@pytest.mark.parametrize("dtype", [f32, bf16, f16])
@pytest.mark.parametrize("most", [1.9, 8.0, 100.0])
@pytest.mark.parametrize("bits", [20, 22, 23, 24])
@pytest.mark.parametrize("V", [393216, 250000, 129280])
def test_top_p_over_a_tail_of_few_units(V, bits, most, dtype):
    L = 63 - (V - 1).bit_length()
    units = torch.exp(torch.rand(V, generator=gen(bits)) * math.log(most)) * 1.01
    l = (units.log() - L * math.log(2.0)).to(dtype)
    w = np.exp2(L + l.double().numpy() / math.log(2.0))
    l[torch.from_numpy(np.abs(w - np.rint(w)) < 1e-4)] = -math.inf
    l[V // 3] = 0.0
    check_units(l, 1.0 - 2.0 ** -bits)
    check_units(l, 1.0 - 2.0 ** -bits, top_k=V // 2)


# ----------------------------------------------------------------------------- small temperatures
@pytest.mark.parametrize("M,t", [(100.0, 1e-3), (-37.0, 1e-3), (5.0, 1e-4), (3e4, 0.5), (12345.0, 1e-1)])
def test_probabilities_at_small_temperatures(M, t):
    # two tokens 1 to 38 octaves of weight apart; u = 1 draws the second
    R = 64
    l = torch.empty((R, 2))
    l[:, 0] = M
    l[:, 1] = torch.from_numpy(M - np.linspace(1.0, 38.0, R) * math.log(2.0) * t).float()
    assert torch.all(l[:, 1] < M)
    idx, prob = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda")
    B.luce_sample(l.cuda(), torch.ones(R, device="cuda"), idx, prob, torch.full((R,), t, device="cuda"))
    torch.cuda.synchronize()
    for r in range(R):
        i, q, _ = D.draw(l[r].double().numpy(), 1.0, float(np.float32(t)))
        # weights within 2^-29 of theirs, or a unit of 2^-62 of weights above 2^-39; three roundings to fp32 of 2^-24
        assert int(idx[r]) == i == 1 and abs(prob[r].item() - q) <= q * 2.0 ** -22, (r, prob[r].item() / q - 1)


# ----------------------------------------------------------------------------- products
@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("T", [5, 8, 12, 40])
@pytest.mark.parametrize("x_dtype,x_size,s_size", [(bf16, -98, -20), (bf16, -100, -16), (f16, -16, -96)])
def test_small_activations_and_scales(T, x_dtype, x_size, s_size, zero_points):
    N, K, group = 60, 512, 64
    x = (torch.randn((T, K), generator=gen(T)).clamp(-4, 4) * 2.0 ** x_size).to(x_dtype)
    q = torch.randint(0, 16, (N, K), generator=gen(1), dtype=torch.uint8)
    s = ((torch.rand((N, K // group), generator=gen(2)) + 0.5) * 2.0 ** s_size).to(bf16)
    z = torch.randint(0, 16, (N, K // group), generator=gen(3), dtype=torch.uint8) if zero_points else None
    out = torch.empty((T, N), dtype=bf16, device="cuda")
    B.luce_linear_w4(x.cuda(), None, O.pack(q).cuda(), s.cuda(), None if z is None else z.cuda(), group, None, out)
    torch.cuda.synchronize()
    y, terms, _ = O.linear(x, None, q, s, z, group)
    # the output's rounding, half a step of 2^-7 of it; 2^-19 of the terms for the tensor cores' sums, 2^-24 for each of
    # eight groups and 24 further operations; sums of groups are kept 2^-14 of their size, good to 2^-150 2^14 each
    tol = 1.001 * 2.0 ** -8 * y.abs() + (2.0 ** -19 + 32 * 2.0 ** -24) * terms + 8 * 2.0 ** -136
    assert terms.max() < 2.0 ** -90 and torch.all((out.cpu().double() - y).abs() <= tol)


# Sums of bf16 activations for fp32 outputs: without the fixed point of others, so that nothing is left of an activation
# itself. Eight steps of the tensor cores may each cut off 2^-22 of the sizes added so far, 2^-19 of a group's terms; a
# rounding of 2^-24 for each of G groups and for 24 further additions, factors and conversions; the output's, 2^-24.
@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,N,K", [(20, 300, 128), (70, 200, 2064), (300, 1000, 4096)])
def test_sums_of_bf16_for_fp32_outputs(T, N, K, group, zero_points):
    # activations over forty octaves, and some that outweigh their chunk a thousandfold
    x = torch.randn((T, K), generator=gen(T)) * 2.0 ** torch.randint(-20, 21, (T, K), generator=gen(T + 1))
    x = torch.where(torch.rand((T, K), generator=gen(T + 2)) < 0.6, torch.randn((T, K), generator=gen(T + 3)), x).to(bf16)
    G = -(-K // group)
    q = torch.randint(0, 16, (N, K), generator=gen(1), dtype=torch.uint8)
    s = (torch.rand((N, G), generator=gen(2)) + 0.5).to(f16)
    z = torch.randint(0, 16, (N, G), generator=gen(3), dtype=torch.uint8) if zero_points else None
    out = torch.empty((T, N), device="cuda")
    B.luce_linear_w4(x.cuda(), None, O.pack(q).cuda(), s.cuda(), None if z is None else z.cuda(), group, None, out)
    torch.cuda.synchronize()
    y, terms, _ = O.linear(x.cuda(), None, q.cuda(), s.cuda(), None if z is None else z.cuda(), group)
    tol = 1.001 * 2.0 ** -24 * y.abs() + (2.0 ** -19 + (G + 24) * 2.0 ** -24) * terms
    assert torch.all((out.double() - y).abs() <= tol)
