"""GPU: 4-bit weights, their products, and draws from logits against their definitions in 64 bits (oracle/w4.py,
oracle/draw.py), one by one and as a decode step's end uses them together.

Codes, scales and zero points are compared bit for bit.  A product's error is bounded by what its parts may leave:
  * whole-number operands (int8; fp32 activations; 16-bit ones for fp32 outputs): each activation is off by at most 2^-23
    of its chunk's largest, and the sums of a group are exact;
  * fp16 operands (16-bit activations and outputs): the tensor cores add 128 products in eight steps, each of which may cut
    off 2^-22 of the sizes added so far: 2^-19 of the terms, codes taken as they are;
  * fp32 sums over the groups: a rounding of 2^-24 for each of G groups, for 24 further additions, factors and
    conversions, relative to the terms' sizes;
  * the output's rounding: half a step.
A drawn token has to be the definition's wherever no decision that leads to it (a sum against top-p's share or the
random number's, a weight against min-p) is closer than 2^-26: the library's weights are within 2^-29 of theirs, or one
unit of 2^-44 or less of the largest, of which even 393,216 make less than 2^-25.4 of it.
"""
import math

import numpy as np
import pytest
import torch

from oracle import draw as D
from oracle import head as OH
from oracle import w4 as O
from quantized_moe_decode_luce_gb300 import binding as B
from quantized_moe_decode_luce_gb300.layer import GreedyHead, LinearI8, LinearW4, SampleHead
from test_gpu_head import _lib, _no_device_faults, bf16, f16, f32, gen, same, shifted  # noqa: F401 (the fixtures hold here)

pytestmark = pytest.mark.gpu
i8 = torch.int8
MARGIN = 2.0 ** -26


@pytest.fixture
def pdl():
    B.luce_set_pdl(True)
    yield
    torch.cuda.synchronize()
    B.luce_set_pdl(False)


# ----------------------------------------------------------------------------- codes
def check_quantize(w, group, sdt, zero_points, shift=0):
    N, K = w.shape
    q, s, z = O.quantize(w, group, sdt, zero_points)
    wq = torch.full((N, O.row_bytes(K)), 255, dtype=torch.uint8, device="cuda")
    sc = torch.full(s.shape, 7.0, dtype=sdt, device="cuda")
    ze = torch.full(s.shape, 99, dtype=torch.uint8, device="cuda") if zero_points else None
    B.luce_quantize_w4(shifted(w, shift), group, wq, sc, ze)
    torch.cuda.synchronize()
    same(sc, s)
    if zero_points:
        same(ze, z)
    same(O.unpack(wq.cpu(), K), q)


@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("sdt", [f16, bf16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(1, 16), (3, 48), (5, 128), (7, 144), (33, 1040), (129, 4096)])
def test_quantize(N, K, group, sdt, zero_points):
    w = torch.randn((N, K), generator=gen(N + K)) * torch.rand((N, 1), generator=gen(1)) * 0.1
    for dt, shift in ((f32, 0), (bf16, 1), (f16, 3)):
        check_quantize(w.to(dt), group, sdt, zero_points, shift)


@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("sdt", [f16, bf16])
def test_quantize_of_unusual_groups(sdt, zero_points):
    w = torch.randn((14, 128), generator=gen(3))
    w[0, :32] = 0.0
    w[1, 40] = math.nan
    w[2, 70] = -math.inf
    w[3] = 1e30       # beyond an fp16 scale
    w[4] = 1e-30      # below it
    w[5] = -w[5].abs()
    w[6] = w[6].abs()
    w[7] = 3.0e38
    w[8] = -3.0e38
    w[9, ::2], w[9, 1::2] = 3.0e38, -3.0e38  # their distance leaves fp32
    w[10] = 2.0 ** -149
    w[11] = -0.0
    w[12] = torch.arange(128) - 64.0
    w[13] = torch.arange(128) * 0.5 + 100.0
    for group in (32, 64, 128):
        check_quantize(w, group, sdt, zero_points)


# codes at and beside half way between two, of rows aligned for wide loads and not, and of scales that their type holds down
@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("dt,shift", [(f32, 0), (f32, 1), (bf16, 0), (bf16, 1), (f16, 0), (f16, 8)])
def test_quantize_half_way(dt, shift, zero_points):
    N, K = 65, 272
    half = torch.randint(-14, 15, (N, K), generator=gen(5)).float() * 0.5
    half[:, ::16] = 7.0
    w = half * 2.0 ** torch.randint(-12, 5, (N, 1), generator=gen(6)).float()
    w[::5] *= 1.0 + 2.0 ** -9
    w[1::5] *= torch.rand((13, K), generator=gen(7)) * 2.0 ** -7 + 1.0
    w = w.to(dt)
    if dt != f16:
        w[2::5] *= 2.0 ** torch.randint(16, 48, (13, K), generator=gen(8)).to(dt)
    for group in (32, 64, 128):
        for sdt in (f16, bf16):
            check_quantize(w, group, sdt, zero_points, shift)


@pytest.mark.parametrize("N,K", [(1, 32), (17, 144)])
def test_pack_aligned(N, K):
    q = torch.randint(0, 16, (N, K), generator=gen(K), dtype=torch.uint8)
    wq = torch.full((N, O.row_bytes(K)), 77, dtype=torch.uint8, device="cuda")
    B.luce_pack_w4(q.cuda(), wq)
    same(wq, O.pack(q))


@pytest.mark.parametrize("N,K", [(1, 16), (9, 112), (40, 400)])
def test_pack(N, K):
    q = torch.randint(0, 256, (N, K), generator=gen(K), dtype=torch.uint8)  # (of other bits the low four count)
    wq = torch.full((N + 2, O.row_bytes(K)), 77, dtype=torch.uint8, device="cuda")
    B.luce_pack_w4(shifted(q, 1), wq[1:N + 1])
    same(wq[1:N + 1], O.pack(q & 15))
    assert torch.all(wq[0] == 77) and torch.all(wq[N + 1] == 77)


# ----------------------------------------------------------------------------- products
def activations(T, K, dtype, seed):
    if dtype == i8:
        return torch.randint(-128, 128, (T, K), generator=gen(seed), dtype=torch.int32).to(i8)
    x = torch.randn((T, K), generator=gen(seed))
    x[:, :: max(1, K // 3)] *= 30.0
    if T > 2:
        x[T - 1] = 0.0  # a padding row
    return x.to(dtype)


def weights(N, K, group, zero_points, sdt, seed):
    G = -(-K // group)
    q = torch.randint(0, 16, (N, K), generator=gen(seed), dtype=torch.uint8)
    s = (torch.randn((N, G), generator=gen(seed + 1)) * 0.01).to(sdt)  # (a scale may be negative)
    z = torch.randint(0, 16, (N, G), generator=gen(seed + 2), dtype=torch.uint8) if zero_points else None
    return q, s, z


def tolerance(y, terms, rest, group, K, x_dtype, out_dtype):
    whole = x_dtype in (i8, f32) or out_dtype == f32
    sums = (-(-K // group) + 24) * 2.0 ** -24 + (0.0 if whole else 2.0 ** -19)
    left = 2.0 ** -23 * rest if whole and x_dtype != i8 else 0.0
    tiny = {f32: 2.0 ** -126, bf16: 2.0 ** -126, f16: 2.0 ** -24}[out_dtype]
    return torch.finfo(out_dtype).eps / 2 * y.abs() * 1.001 + sums * terms + left + tiny


def check_linear(T, N, K, group=128, zero_points=False, x_dtype=bf16, out_dtype=f32, sdt=f16, bias=False, seed=1, x=None, xgap=0, gap=0, stream=None,
                 device_oracle=False):
    x = activations(T, K, x_dtype, seed) if x is None else x
    q, s, z = weights(N, K, group, zero_points, sdt, seed + 10)
    xs = torch.rand(T, generator=gen(seed + 20)) * 0.01 if x_dtype == i8 else None
    b = torch.randn(N, generator=gen(seed + 21)) if bias else None
    wide_x = torch.zeros((T, K + xgap), dtype=x_dtype, device="cuda")
    wide_x[:, :K] = x.cuda()
    wide = torch.full((T, N + gap), 77.0, dtype=out_dtype, device="cuda")
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    B.luce_linear_w4(wide_x[:, :K], cuda(xs), O.pack(q).cuda(), s.cuda(), cuda(z), group, cuda(b), wide[:, :N], stream)
    torch.cuda.synchronize()
    at = "cuda" if device_oracle else "cpu"
    args = [None if t is None else t.to(at) for t in (x, xs, q, s, z)]
    y, terms, rest = O.linear(*args, group, None if b is None else b.to(at))
    tol = tolerance(y, terms, rest, group, K, x_dtype, out_dtype)
    off = (wide[:, :N].to(at).double() - y).abs()
    bad = ~(off <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off, first at {i}: by {off[i]:.3g}, bound {tol[i]:.3g}, of {y[i]:.3g}")
    assert torch.all(wide[:, N:] == 77.0)
    return wide[:, :N]


TS = [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 24, 31, 33, 47, 48, 49, 64, 65, 96, 97, 128, 130, 300]
SHAPES = [(1, 16), (15, 48), (16, 112), (17, 128), (129, 144), (300, 1040), (1000, 400), (40, 4096)]


@pytest.mark.parametrize("x_dtype", [f32, bf16, f16, i8])
@pytest.mark.parametrize("T", TS)
def test_products(T, x_dtype):
    for i, (N, K) in enumerate(SHAPES):
        v = TS.index(T) + i
        check_linear(T, N, K, (32, 64, 128)[v % 3], v % 2 == 1, x_dtype, (f32, bf16, f16)[(v // 2) % 3], (f16, bf16)[(v // 3) % 2], v % 5 == 0, seed=v + 1)


@pytest.mark.parametrize("x_dtype,out_dtype", [(f32, f32), (bf16, bf16), (bf16, f32), (f16, f16), (f16, f32), (i8, f32)])
@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 6, 20, 70])
def test_every_kind_of_group(T, group, zero_points, x_dtype, out_dtype):
    check_linear(T, 200, 2064, group, zero_points, x_dtype, out_dtype, seed=T)


# many tiles to a CTA, and more stages than its shared memory holds: every place is used again
@pytest.mark.parametrize("T,N,K,group,zero_points,x_dtype", [
    (3, 30240, 11696, 64, True, i8), (2, 60000, 4096, 32, False, bf16), (5, 40001, 4096, 64, True, f32), (100, 20001, 4096, 32, True, bf16),
    (300, 8192, 4096, 64, False, bf16), (40, 25000, 3088, 128, True, f16), (130, 20480, 2048, 32, True, i8), (90, 20480, 2048, 64, True, f32),
    (1, 60001, 2048, 128, False, bf16), (1, 129280, 1024, 32, True, i8)])
def test_many_tiles(T, N, K, group, zero_points, x_dtype):
    first = check_linear(T, N, K, group, zero_points, x_dtype, f32, device_oracle=True)
    for _ in range(3):
        same(check_linear(T, N, K, group, zero_points, x_dtype, f32, device_oracle=True), first)


# more tiles than SMs, so that those of the last round may be split along K by a second launch
@pytest.mark.parametrize("T,N,K,group,zero_points,x_dtype", [
    (200, 4096, 4112, 64, True, bf16), (210, 14001, 1040, 64, False, f16), (515, 4000, 1552, 32, True, bf16), (161, 10000, 2064, 32, True, f32),
    (300, 8100, 2048, 64, False, i8), (700, 3000, 2080, 128, True, bf16), (97, 20479, 1056, 64, True, bf16), (2049, 1300, 528, 128, False, i8)])
def test_the_last_tiles(T, N, K, group, zero_points, x_dtype):
    first = check_linear(T, N, K, group, zero_points, x_dtype, f32, bias=True, gap=5, device_oracle=True)
    same(check_linear(T, N, K, group, zero_points, x_dtype, f32, bias=True, gap=5, device_oracle=True), first)


def test_the_last_tiles_started_early():
    # each product's activations are the one's before, two launches each: the same bits with programmatic launch as without
    T, N = 200, 4096
    q, s, z = weights(N, N, 64, True, f16, 3)
    w = LinearW4(O.pack(q).cuda(), (s * 0.05).cuda(), N, 64, z.cuda())
    x = activations(T, N, bf16, 4).cuda()

    def chain():
        outs = [x] + [torch.zeros((T, N), dtype=bf16, device="cuda") for _ in range(4)]
        for a, b in zip(outs, outs[1:]):
            w.run(a, None, b)
        torch.cuda.synchronize()
        return outs[1:]

    want = chain()
    B.luce_set_pdl(True)
    try:
        for _ in range(10):
            for a, b in zip(chain(), want):
                same(a, b)
    finally:
        B.luce_set_pdl(False)


@pytest.mark.parametrize("T,K", [(1, 16384), (4, 16384), (2, 65536), (20, 65536), (64, 14336), (1, 65520)])
@pytest.mark.parametrize("x_dtype", [f32, bf16, i8])
def test_long_rows(T, K, x_dtype):
    check_linear(T, 70, K, 64, True, x_dtype, f32, seed=K % 100)


@pytest.mark.parametrize("T", [1, 5, 33, 130])
@pytest.mark.parametrize("x_dtype", [f32, bf16, i8])
def test_rows_apart(T, x_dtype):
    xgap = 64 // torch.empty(0, dtype=x_dtype).element_size()
    check_linear(T, 100, 512, 32, False, x_dtype, bf16, xgap=xgap, gap=3)
    check_linear(T, 257, 272, 64, True, x_dtype, f32, xgap=xgap, gap=1, bias=True)


@pytest.mark.parametrize("T", [2, 3, 12, 40])
@pytest.mark.parametrize("x_dtype", [f32, bf16])
def test_activations_of_any_size(T, x_dtype):
    x = activations(T, 512, x_dtype, 5).float()
    x[0] *= 1e30
    x[1] *= 1e-30
    x[0, 128:256] = 2.0 ** -130  # subnormal ones beside them
    x[1, 256:384] = 0.0
    check_linear(T, 60, 512, 64, True, x_dtype, f32, x=x.to(x_dtype))


@pytest.mark.parametrize("T", [3, 12, 40])
@pytest.mark.parametrize("x_dtype", [f32, bf16, f16])
def test_nan_and_infinity_stay_in_their_rows(T, x_dtype):
    x = activations(T, 512, x_dtype, 6)
    clean = check_linear(T, 100, 512, 64, True, x_dtype, f32, x=x)
    for value in (math.nan, math.inf, -math.inf):
        dirty = x.clone()
        dirty[1, 300] = value
        q, s, z = weights(100, 512, 64, True, f16, 11)
        out = torch.zeros((T, 100), device="cuda")
        B.luce_linear_w4(dirty.cuda(), None, O.pack(q).cuda(), s.cuda(), z.cuda(), 64, None, out)
        assert not torch.isfinite(out[1]).any()
        keep = [t for t in range(T) if t != 1]
        same(out[keep], clean[keep])


def test_scales_of_zero_infinity_and_nan():
    q, s, z = weights(8, 256, 64, False, f16, 4)
    s[1, 2], s[2, 0], s[3] = math.nan, math.inf, 0.0
    for T in (1, 20):
        x = activations(T, 256, bf16, 9)
        out = torch.zeros((T, 8), device="cuda")
        B.luce_linear_w4(x.cuda(), None, O.pack(q).cuda(), s.cuda(), None, 64, None, out)
        live = [t for t in range(T) if x[t].any()]
        assert torch.isnan(out[:, 1]).all() and torch.all(out[:, 3] == 0) and not torch.isfinite(out[live, 2]).any()
        assert torch.isfinite(out[:, 4:]).all()


def test_no_tokens():
    q, s, _ = weights(8, 64, 32, False, f16, 1)
    B.luce_linear_w4(torch.zeros((0, 64), device="cuda"), None, O.pack(q).cuda(), s.cuda(), None, 32, None, torch.zeros((0, 8), device="cuda"))
    B.luce_quantize_w4(torch.zeros((0, 64), device="cuda"), 32, torch.zeros((0, 64), dtype=torch.uint8, device="cuda"),
                       torch.zeros((0, 2), dtype=f16, device="cuda"))


@pytest.mark.parametrize("T,N,K", [(1, 2048, 1024), (5, 1000, 4096), (20, 4000, 1024), (300, 8000, 512)])
def test_weights_quantized_just_before_their_product(T, N, K, pdl):
    # the launch before the product writes its weights, the same buffers take two matrices in turn
    ws = [torch.randn((N, K), generator=gen(s)).cuda() for s in (1, 2)]
    x = activations(T, K, bf16, 3)
    wq, sc, ze = torch.empty((N, O.row_bytes(K)), dtype=torch.uint8, device="cuda"), torch.empty((N, K // 64), dtype=f16, device="cuda"), \
        torch.empty((N, K // 64), dtype=torch.uint8, device="cuda")
    outs, xd = torch.empty((20, T, N), device="cuda"), x.cuda()
    torch.cuda.synchronize()
    for i in range(20):
        B.luce_quantize_w4(ws[i % 2], 64, wq, sc, ze)
        B.luce_linear_w4(xd, None, wq, sc, ze, 64, None, outs[i])
    torch.cuda.synchronize()
    for i in range(2):
        q, s, z = O.quantize(ws[i], 64, f16, True)
        y, terms, rest = O.linear(xd, None, q, s, z, 64)
        assert torch.all((outs[i].double() - y).abs() <= tolerance(y, terms, rest, 64, K, bf16, f32))
        for j in range(i + 2, 20, 2):
            same(outs[j], outs[i])


@pytest.mark.parametrize("T", [1, 30])
def test_products_on_streams_and_in_graphs(T):
    N, K = 3000, 1024
    xs = [activations(T, K, bf16, s).cuda() for s in (1, 2, 3)]
    q, s, z = weights(N, K, 64, True, f16, 9)
    wq, s, z = O.pack(q).cuda(), s.cuda(), z.cuda()
    want = [torch.empty((T, N), device="cuda") for _ in xs]
    for x, w in zip(xs, want):
        B.luce_linear_w4(x, None, wq, s, z, 64, None, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [torch.empty((T, N), device="cuda") for _ in xs]
    for _ in range(5):
        for x, o, st in zip(xs, got, streams):
            B.luce_linear_w4(x, None, wq, s, z, 64, None, o, st)
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        same(o, w)
    # two graphs that replay side by side, with new inputs in their places
    graphs, ins, outs = [], [], []
    for _ in range(2):
        x, o = torch.zeros_like(xs[0]), torch.empty((T, N), device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.luce_linear_w4(x, None, wq, s, z, 64, None, o)
        graphs.append(g), ins.append(x), outs.append(o)
    for a, b in ((0, 1), (2, 0), (1, 2)):
        ins[0].copy_(xs[a]), ins[1].copy_(xs[b])
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        same(outs[0], want[a]), same(outs[1], want[b])


def test_products_that_are_refused():
    q, s, _ = weights(8, 64, 32, False, f16, 1)
    wq, s, x, out = O.pack(q).cuda(), s.cuda(), torch.zeros((3, 72), dtype=bf16, device="cuda"), torch.zeros((3, 8), device="cuda")
    B.luce_linear_w4(x[:, :64], None, wq, s, None, 32, None, out)
    with pytest.raises(B.LuceError):  # rows that do not start on 16 bytes
        B.luce_linear_w4(x[:, 1:65], None, wq, s, None, 32, None, out)
    with pytest.raises(B.LuceError):  # the output over the weights
        B.luce_linear_w4(x[:1, :64], None, wq, s, None, 32, None, wq.view(-1)[:32].view(f32).view(1, 8))
    for bad in (lambda: B.luce_linear_w4(x[:, :64], out[:, 0], wq, s, None, 32, None, out), lambda: B.luce_linear_w4(x, None, wq, s, None, 32, None, out),
                lambda: B.luce_linear_w4(x[:, :64], None, wq, s[:, :1].contiguous(), None, 32, None, out),
                lambda: B.luce_linear_w4(x[:, :64], None, wq, s, None, 32, None, out[:2]),
                lambda: B.luce_linear_w4(x[:, :64], None, wq, s, None, 16, None, out),
                lambda: B.luce_linear_w4(torch.zeros((3, 64), dtype=i8, device="cuda"), None, wq, s, None, 32, None, out)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(TypeError):
        B.luce_linear_w4(x[:, :64], None, wq, s.float(), None, 32, None, out)


# ----------------------------------------------------------------------------- draws
def logits_of(kind, R, V, seed):
    g = gen(seed)
    return {"normal": lambda: torch.randn((R, V), generator=g) * 3, "flat": lambda: torch.zeros((R, V)),
            "two values": lambda: torch.randint(0, 2, (R, V), generator=g).float(), "whole": lambda: torch.randint(-3, 4, (R, V), generator=g).float(),
            "uniform": lambda: torch.rand((R, V), generator=g), "wide": lambda: torch.randn((R, V), generator=g) * 100,
            "tiny": lambda: torch.randn((R, V), generator=g) * 1e-30, "below": lambda: -50 - torch.rand((R, V), generator=g) * 5,
            "huge": lambda: torch.randn((R, V), generator=g) * 1e37,
            "masked": lambda: torch.where(torch.rand((R, V), generator=g) < 0.6, torch.tensor(-math.inf), torch.randn((R, V), generator=g) * 2),
            "peaked": lambda: torch.randn((R, V), generator=g) * 2 + 14 * (torch.rand((R, V), generator=g) < 20 / max(V, 40))}[kind]()


def check_draws(l, u, t=None, k=None, p=None, m=None, gap=0, front=0, stream=None, prob=True):
    """Every row against the definition; returns how many rows were too close to call."""
    R, V = l.shape
    wide = torch.full((R, front + V + gap), 6e4, dtype=l.dtype, device="cuda")
    wide[:, front:front + V] = l.cuda()
    column = lambda x, dt: None if x is None else torch.as_tensor(x, dtype=dt).expand(R).contiguous().cuda()  # noqa: E731
    idx = torch.full((R + 2,), -9, dtype=torch.int32, device="cuda")
    pr = torch.full((R + 2,), -9.0, device="cuda")
    tt, kk, pp, mm = column(t, f32), column(k, torch.int32), column(p, f32), column(m, f32)
    B.luce_sample(wide[:, front:front + V], u.cuda(), idx[1:R + 1], pr[1:R + 1] if prob else None, tt, kk, pp, mm, stream)
    torch.cuda.synchronize()
    assert idx[0] == -9 and idx[R + 1] == -9 and pr[0] == -9 and pr[R + 1] == -9
    close = 0
    at = lambda x, r, off: off if x is None else x[r].item()  # noqa: E731
    for r in range(R):
        i, q, margin = D.draw(l[r].double().numpy(), u[r].item(), at(tt, r, 1.0), at(kk, r, 0), at(pp, r, 1.0), at(mm, r, 0.0))
        if margin < MARGIN:
            close += 1
            continue
        assert int(idx[r + 1]) == i, (r, int(idx[r + 1]), i, margin)
        if prob:
            got = pr[r + 1].item()
            assert (math.isnan(got) and math.isnan(q)) or abs(got - q) <= q * 2.0 ** -21 + 2.0 ** -40, (r, got, q)
    return close


PARAMS = [dict(), dict(t=0.7, k=1), dict(t=1.3, k="half", p=0.9), dict(t=0.5, p=0.5), dict(t=2.0, p=0.999, m=0.01), dict(k=7, p=0.3, m=0.5),
          dict(k="all but one"), dict(t=math.inf, p=0.7), dict(t=0.0, k=3, p=0.5, m=0.1), dict(t=1e-6, k=20, p=0.9), dict(t=50.0, k=1500, p=0.99),
          dict(p=0.0), dict(m=1.0), dict(t=0.9, k=40, p=0.95, m=0.02), dict(t=1.0, k=600), dict(t=-1.0), dict(t=math.nan), dict(k=-3, p=math.nan, m=math.nan)]


@pytest.mark.parametrize("kind", ["normal", "flat", "two values", "whole", "uniform", "wide", "tiny", "below", "huge", "masked", "peaked"])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 5003, 40000, 131073])
def test_draws(V, kind):
    close = rows = 0
    for n, prm in enumerate(PARAMS):
        dt = f32 if kind == "huge" else (f32, bf16, f16)[n % 3]
        l, u = logits_of(kind, 2, V, V + n).to(dt), torch.rand(2, generator=gen(n + V))
        prm = dict(prm, **({"k": max(1, V // 2 if prm["k"] == "half" else V - 1)} if isinstance(prm.get("k"), str) else {}))
        close += check_draws(l, u, **prm)
        rows += 2
    # Rows that the definition itself leaves open, whatever the kernel gave. Where the first n logits are equal, a share p
    # of them lies on a token's edge if p n is whole: 0.9 V/2, 0.5 V, 0.999 V, 0.7 V (all weights are 1 at an infinite
    # temperature), 0.9 * 20, 0.99 * 1500 and 0.95 * 40 can be, 0.3 * 7 = 2.1 can't: 7 of the 18, two rows each, 14 rows.
    # Values of a narrow range are equal at the top in 16 bits. Otherwise a sum comes as near to one of V edges by a
    # chance of 2 V 2^-26, at most 0.4 %.
    assert close <= (14 if kind in ("flat", "two values", "tiny", "whole", "uniform", "below") or V <= 33 else 0.06 * rows)


@pytest.mark.parametrize("dtype", [f32, bf16, f16])
@pytest.mark.parametrize("R,V", [(1, 129280), (5, 129279), (10, 50001), (64, 32000), (200, 4097), (40, 129280)])
def test_draws_of_batches(R, V, dtype):
    g = gen(R + V)
    l = logits_of("peaked", R, V, R).to(dtype)
    l[:, ::7] = -math.inf
    t = torch.rand(R, generator=g) * 1.2 + 0.3
    t[::5] = 0.0
    k = torch.tensor([0, 1, 40, 7, 1000, 0, 20000, 64], dtype=torch.int32).repeat(R // 8 + 1)[:R]
    p = torch.tensor([0.9, 1.0, 0.5, 0.99, 0.95]).repeat(R // 5 + 1)[:R]
    m = torch.tensor([0.0, 0.05, 0.001]).repeat(R // 3 + 1)[:R]
    assert check_draws(l, torch.rand(R, generator=g), t, k, p, m) <= 1 + R // 50


@pytest.mark.parametrize("dtype", [f32, bf16, f16])
@pytest.mark.parametrize("front,gap", [(1, 0), (3, 2), (0, 5), (8, 8), (7, 1)])
def test_draws_from_rows_apart(front, gap, dtype):
    for V in (1, 100, 4099):
        l = logits_of("normal", 5, V, V)
        check_draws(l.to(dtype), torch.rand(5, generator=gen(V)), 0.8, 30, 0.9, gap=gap, front=front)
        check_draws(l.to(dtype), torch.rand(5, generator=gen(V)), 0.8, gap=gap, front=front, prob=False)


@pytest.mark.parametrize("V", [393216, 393213])
@pytest.mark.parametrize("dtype", [f32, bf16])
def test_draws_from_the_largest_vocabularies(V, dtype):
    l, u = logits_of("normal", 3, V, 2).to(dtype), torch.tensor([0.1, 0.5, 0.999])
    for prm in (dict(t=0.8), dict(t=0.8, k=50, p=0.9), dict(t=1.2, p=0.9), dict(k=200000, p=0.99)):
        assert check_draws(l, u, **prm) <= 1
    l, u = logits_of("normal", 20, V, 3).to(dtype), torch.rand(20, generator=gen(3))  # (rows for clusters of eight CTAs)
    assert check_draws(l, u, t=0.9, k=40, p=0.95) <= 1
    with pytest.raises(B.LuceError) as e:
        B.luce_sample(torch.zeros((1, 393217), device="cuda"), torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert e.value.status == B.LUCE_ERR_UNSUPPORTED


def test_rows_without_a_token():
    l = torch.randn((7, 3000), generator=gen(1))
    l[0] = -math.inf
    l[1, 2999] = math.nan
    l[2, 0] = math.inf
    l[3], l[3, 5] = -math.inf, -3.0e38
    l[4, 100:] = -math.inf
    l[5], l[5, 7] = -math.inf, math.nan
    for prm in (dict(), dict(t=0.0), dict(k=5), dict(p=0.5), dict(t=1.5, k=1500, p=0.9, m=0.1)):
        for dt in (f32, bf16):
            check_draws(l.to(dt), torch.full((7,), 0.5), **prm)


def test_random_numbers_at_their_ends():
    l = logits_of("normal", 8, 2000, 4)
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -0.5, math.nan, 2.0 ** -149, math.inf])
    for prm in (dict(), dict(k=10), dict(p=0.9), dict(t=30.0, p=0.99)):
        check_draws(l, u, **prm)


@pytest.mark.parametrize("prm", [dict(), dict(k=30), dict(p=0.8), dict(t=2.0, k=900, p=0.95)])
def test_a_larger_number_draws_a_larger_id(prm):
    R = 513
    l = logits_of("peaked", 1, 3000, 8).expand(R, -1).contiguous()
    u = torch.arange(R) / R
    check_draws(l, u, **prm)
    idx = torch.empty(R, dtype=torch.int32, device="cuda")
    column = {n: torch.full((R,), v, dtype=torch.int32 if n == "top_k" else f32, device="cuda")
              for n, v in (("temperature", prm.get("t", 1.0)), ("top_k", prm.get("k", 0)), ("top_p", prm.get("p", 1.0)))}
    B.luce_sample(l.cuda(), u.cuda(), idx, None, **column)
    assert torch.all(idx[1:] >= idx[:-1])


def test_equal_logits_by_exact_counts():
    # n equal logits of V stay, by id: of m = 2^j n draws, every one of them m / n times
    V, n, R = 5000, 64, 256
    l = torch.full((R, V), -1.0)
    l[:, 3::7] = 2.0
    ids = list(range(3, V, 7))[:n]
    idx = torch.empty(R, dtype=torch.int32, device="cuda")
    u = (torch.arange(R) + 0.5) / R
    B.luce_sample(l.cuda(), u.cuda(), idx, None, top_k=torch.full((R,), n, dtype=torch.int32, device="cuda"))
    assert idx.tolist() == [ids[r * n // R] for r in range(R)]
    share = (n - 0.5) * math.exp(0.0) / (len(range(3, V, 7)) + (V - len(range(3, V, 7))) * math.exp(-3.0))
    B.luce_sample(l.cuda(), u.cuda(), idx, None, top_p=torch.full((R,), share, device="cuda"))
    assert idx.tolist() == [ids[r * n // R] for r in range(R)]


def test_draws_on_streams_in_graphs_and_early(pdl):
    R, V = 6, 20000
    ls = [logits_of("peaked", R, V, s).cuda() for s in range(3)]
    u = torch.rand(R, generator=gen(1)).cuda()
    k, p = torch.tensor([0, 5, 50, 900, 0, 64], dtype=torch.int32, device="cuda"), torch.tensor([0.9, 1.0, 0.5, 0.95, 1.0, 0.9], device="cuda")
    want = []
    for l in ls:
        i, q = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda")
        B.luce_sample(l, u, i, q, None, k, p)
        torch.cuda.synchronize()
        want.append((i, q))
    for _ in range(20):
        outs = []
        for l in ls:
            i, q = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda")
            B.luce_sample(l, u, i, q, None, k, p, None, torch.cuda.Stream())
            outs.append((i, q))
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            same(a[0], b[0]), same(a[1], b[1])
    l, i, q = torch.zeros_like(ls[0]), torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.luce_sample(l, u, i, q, None, k, p)
    for n in (2, 0, 1):
        l.copy_(ls[n])
        g.replay()
        torch.cuda.synchronize()
        same(i, want[n][0]), same(q, want[n][1])


def test_draws_that_are_refused():
    l, u, i = torch.zeros((2, 8), device="cuda"), torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    B.luce_sample(l, u, i)
    B.luce_sample(l[:0], u[:0], i[:0])
    for bad in (lambda: B.luce_sample(l, u[:1], i), lambda: B.luce_sample(l.t(), u, i), lambda: B.luce_sample(l, u, u), lambda: B.luce_sample(l.double(), u, i),
                lambda: B.luce_sample(l, u, i, top_k=u), lambda: B.luce_sample(l, u, i, top_p=i), lambda: B.luce_sample(l, u.cpu(), i),
                lambda: B.luce_sample(l, u, i, temperature=0.7)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(B.LuceError):
        B.luce_sample(l, u, l.view(torch.int32).view(-1)[:2])


# ----------------------------------------------------------------------------- together
@pytest.mark.parametrize("weights_of", ["w4", "w4 with zero points", "i8"])
@pytest.mark.parametrize("R,K,N", [(1, 512, 3000), (5, 1024, 4099), (33, 272, 1000)])
def test_a_steps_end(R, K, N, weights_of):
    g = gen(R + K)
    w = torch.randn((N, K), generator=g) * 0.05
    gamma = torch.rand(K, generator=g) + 0.5
    x, res = torch.randn((R, K), generator=g).to(bf16), torch.randn((R, K), generator=g).to(bf16)
    x[R - 1, 0] = math.nan if R > 1 else x[R - 1, 0]
    bias = torch.randn(N, generator=g)
    if weights_of == "i8":
        head = LinearI8.from_float(w.cuda(), bias.cuda())
    else:
        head = LinearW4.from_float(w.cuda(), 64, weights_of != "w4", bias=bias.cuda())
    hist = torch.randint(0, N, (R, 50), generator=g, dtype=torch.int32)
    mask = torch.randint(-2**31, 2**31, (R, (N + 31) // 32), generator=g, dtype=torch.int64).to(torch.int32)
    process = dict(hist=hist.cuda(), hist_len=torch.full((R,), 50, dtype=torch.int32, device="cuda"), repetition=torch.full((R,), 1.3, device="cuda"),
                   mask=mask.cuda())
    sample, greedy = SampleHead(R, gamma.cuda(), 1e-6, head), GreedyHead(R, gamma.cuda(), 1e-6, head)
    u = torch.rand(R, generator=g)
    t, k = torch.full((R,), 0.7), torch.full((R,), 40, dtype=torch.int32)
    summed = torch.empty_like(x, device="cuda")
    idx, prob = sample.run(x.cuda(), u.cuda(), res.cuda(), summed, t.cuda(), k.cuda(), **process)
    gi, gv = greedy.run(x.cuda(), res.cuda(), **process)
    torch.cuda.synchronize()
    q, sc, s = OH.rows_i8(x, gamma, 1e-6, res)
    same(summed, s)
    same(sample.q, q)
    if weights_of == "i8":
        y = torch.nn.functional.linear(q.double() * sample.scale.cpu().double()[:, None], head.wq.cpu().double() * head.w_scale.cpu().double()[:, None]) + bias.double()
        terms = (q.double().abs() * sample.scale.cpu().double()[:, None]) @ (head.wq.cpu().double().abs() * head.w_scale.cpu().double()[:, None]).T + bias.abs()
    else:
        codes = O.unpack(head.wq.cpu(), K)
        zeros = None if head.zeros is None else head.zeros.cpu()
        y, terms, _ = O.linear(q, sample.scale.cpu(), codes, head.w_scale.cpu(), zeros, 64, bias)
    live = [r for r in range(R) if torch.isfinite(sample.scale[r])]
    assert len(live) == (R - 1 if R > 1 else 1)
    # penalties and mask by their own definition, on the product's rows
    raw = torch.empty((R, N), device="cuda")
    head.run(sample.q, sample.scale, raw)
    tol = (K // 64 + 26) * 2.0 ** -24 * terms + 2.0 ** -24 * y.abs()
    assert torch.all(((raw.cpu().double() - y).abs() <= tol)[live])
    want = OH.logits_process(raw.cpu(), hist, torch.full((R,), 50, dtype=torch.int32), None, torch.full((R,), 1.3), None, None, None, None, mask, None)
    same(sample.logits, want)
    same(greedy.logits, want)
    for r in live:
        i, p, margin = D.draw(want[r].double().numpy(), u[r].item(), t[r].item(), 40)
        assert margin < MARGIN or (int(idx[r]) == i and abs(prob[r].item() - p) <= p * 2.0 ** -21)
        assert int(gi[r]) == int(want[r].argmax()) and gv[r].item() == want[r].max().item()
    for r in set(range(R)) - set(live):
        assert math.isnan(prob[r].item()) and int(idx[r]) == 0
    # the same in a graph, on new rows
    x2 = torch.randn((R, K), generator=g).to(bf16).cuda()
    ud, td, kd, buf = u.cuda(), t.cuda(), k.cuda(), x.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sample.run(buf, ud, temperature=td, top_k=kd)
    buf.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    got = idx.clone(), prob.clone()
    sample.run(x2, ud, temperature=td, top_k=kd)
    same(got[0], idx), same(got[1], prob)


def test_weights_of_other_programs_codes():
    codes = torch.randint(0, 16, (50, 400), generator=gen(1), dtype=torch.uint8)
    s, z = torch.rand((50, 4), generator=gen(2)).to(bf16) * 0.1, torch.randint(0, 16, (50, 4), generator=gen(3), dtype=torch.uint8)
    lin = LinearW4.from_codes(codes.cuda(), s.cuda(), 128, z.cuda())
    x = torch.randn((6, 400), generator=gen(4))
    out = lin.run(x.cuda(), None, torch.empty((6, 50), device="cuda"))
    y, terms, rest = O.linear(x, None, codes, s, z, 128)
    assert torch.all((out.cpu().double() - y).abs() <= tolerance(y, terms, rest, 128, 400, f32, f32))
