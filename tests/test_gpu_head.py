"""GPU: the int8 decode-head operators against their definitions in 64 bits
(oracle/head.py), one by one and as they are used together.

Codes, products and processed logits are compared bit for bit: their formulas
round at named places and hold no sum whose order is free (the int8 product's
sum is exact).  A row scale holds a sum of squares in fp32: with at most 256
squares added one after the other and 16 levels of partial sums, its relative
error is at most 272 halves of a step (2^-24 each), of which the square root
keeps half, and six more roundings follow: 142 * 2^-24.
"""
import math

import pytest
import torch

from oracle import head as O
from quantized_moe_decode_luce_gb300 import binding as B
from quantized_moe_decode_luce_gb300 import build as BLD
from quantized_moe_decode_luce_gb300.layer import GreedyHead, LinearI8

pytestmark = pytest.mark.gpu
f32, bf16, f16 = torch.float32, torch.bfloat16, torch.float16
SCALE_TOL = 142 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    BLD.build()
    B.lib()
    yield


@pytest.fixture(autouse=True)
def _no_device_faults(request):
    yield
    faults = B.luce_get_fault()
    if "allow_fault" not in request.keywords:
        assert faults == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def same(a, b):
    """Equal bits, NaNs (of any payload) in the same places."""
    a, b = a.cpu(), b.cpu()
    assert a.shape == b.shape and a.dtype == b.dtype
    na, nb = torch.isnan(a), torch.isnan(b)
    assert torch.equal(na, nb), "NaNs in other places"
    bad = (a != b) & ~na
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} differ, first at {i}: {a[i]!r} against {b[i]!r}")


def shifted(t, n):
    """A contiguous copy of t on the GPU that starts n elements into its storage."""
    buf = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")
    out = buf[n:].view(t.shape)
    out.copy_(t)
    return out


# ----------------------------------------------------------------------------- rows to int8
def rows_input(T, H, dtype, seed):
    x = torch.randn((T, H), generator=gen(seed))
    x[:, :: max(1, H // 3)] *= 30.0
    if T > 1:
        x[T - 1] = 0.0  # a padding row
    return x.to(dtype)


def check_rows(x, gamma=None, eps=0.0, residual=None, shift=(0, 0, 0, 0), in_place=None, stream=None):
    T, H = x.shape
    q_ref, s_ref, sum_ref = O.rows_i8(x, gamma, eps, residual)
    xd = shifted(x, shift[0])
    q = shifted(torch.full((T, H), 99, dtype=torch.int8), shift[2])
    scale = torch.full((T,), 99.0, device="cuda")
    if gamma is None:
        B.luce_quantize_i8(xd, q, scale, stream)
    elif residual is None:
        B.luce_rmsnorm_i8(xd, shifted(gamma, shift[3]), eps, q, scale, stream)
    else:
        rd = shifted(residual, shift[1])
        xs = {"x": xd, "residual": rd, None: None}.get(in_place, shifted(torch.zeros_like(x), shift[0]))
        B.luce_add_rmsnorm_i8(xd, rd, xs, shifted(gamma, shift[3]), eps, q, scale, stream)
        if xs is not None:
            same(xs, sum_ref)
    torch.cuda.synchronize()
    same(q, q_ref)
    sc = scale.cpu().double()
    assert torch.equal(torch.isnan(sc), torch.isnan(s_ref))
    ok = (sc - s_ref).abs() <= SCALE_TOL * s_ref.abs() + 2.0 ** -149
    assert torch.all(ok | torch.isnan(s_ref))
    if gamma is None:
        same(scale, s_ref.to(f32))  # no sum: the same bits


HS = [1, 2, 7, 31, 32, 33, 64, 100, 255, 516, 1000, 1024, 1025, 2048, 4096, 4099, 5000, 8192, 8200, 12288, 16384, 16391,
      32768, 65536]


# every number of chunks to a thread: few and many rows of short and long ones
MANY = [(60, 1000), (700, 1000), (2300, 1001), (330, 758), (3600, 758), (150, 4099), (400, 4099), (900, 4099), (1100, 4096),
        (900, 4728), (300, 6319), (260, 8192), (700, 8192), (300, 14336), (300, 16390)]


@pytest.mark.parametrize("dtype", [f32, bf16])
@pytest.mark.parametrize("T,H", MANY)
def test_many_rows_of_every_width(T, H, dtype):
    x, gamma = rows_input(T, H, dtype, T + H), torch.randn(H, generator=gen(H))
    check_rows(x)
    check_rows(x, gamma, 1e-6)
    check_rows(x, gamma, 1e-6, rows_input(T, H, dtype, T), in_place="x" if T % 2 else None)


@pytest.mark.parametrize("dtype", [f32, bf16, f16])
@pytest.mark.parametrize("H", HS)
def test_quantize_rows(H, dtype):
    for T in (1, 5):
        check_rows(rows_input(T, H, dtype, H + T))


@pytest.mark.parametrize("dtype", [f32, bf16, f16])
@pytest.mark.parametrize("H", HS)
def test_rmsnorm_rows(H, dtype):
    gamma = torch.rand(H, generator=gen(5)) + 0.5
    check_rows(rows_input(3, H, dtype, H), gamma, 1e-6)
    res = (torch.randn((3, H), generator=gen(H)) * 2).to(dtype)
    res[2] = 0
    check_rows(rows_input(3, H, dtype, H + 1), gamma, 1e-6, res, in_place="new")
    check_rows(rows_input(3, H, dtype, H + 1), gamma, 1e-6, res, in_place=None)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 151, 153, 700, 2049])
@pytest.mark.parametrize("H", [64, 1000, 2048])
def test_many_rows(T, H):
    gamma = torch.rand(H, generator=gen(5)) + 0.5
    check_rows(rows_input(T, H, bf16, T), gamma, 1e-5, rows_input(T, H, bf16, T + 1), in_place="new")


@pytest.mark.parametrize("dtype", [f32, bf16])
@pytest.mark.parametrize("shift", [(1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1), (1, 1, 3, 1), (3, 2, 5, 1),
                                   (8, 8, 16, 4), (7, 7, 0, 0)])
@pytest.mark.parametrize("H", [100, 2048, 4099])
def test_rows_at_any_alignment(H, shift, dtype):
    gamma = torch.rand(H, generator=gen(6)) + 0.5
    res = torch.randn((3, H), generator=gen(7)).to(dtype)
    check_rows(rows_input(3, H, dtype, 8), gamma, 1e-6, res, shift=shift, in_place="new")
    check_rows(rows_input(3, H, dtype, 9), shift=shift)


@pytest.mark.parametrize("which", ["x", "residual"])
@pytest.mark.parametrize("H", [516, 4096, 4099, 20000, 40000])
def test_residual_stream_in_place(H, which):
    gamma = torch.rand(H, generator=gen(6)) + 0.5
    check_rows(rows_input(6, H, bf16, 3), gamma, 1e-6, torch.randn((6, H), generator=gen(7)).to(bf16), in_place=which)


@pytest.mark.parametrize("H", [48, 2048, 4099, 40000])
def test_rows_with_infinities_nans_and_tiny_values(H):
    x = rows_input(8, H, f32, 11)
    x[0, H // 2] = math.inf
    x[1, 0] = math.nan
    x[2, H - 1] = -math.inf
    x[3] = 2.0 ** -149       # the step rounds to zero
    x[4] = 190 * 2.0 ** -149  # the step rounds down: codes are kept within 127
    x[5] = 0.0
    x[5, 1] = -3.0e38
    x[6] = -0.0
    check_rows(x)
    x[5, 1] = -1.0e18  # (its square is finite)
    check_rows(x, torch.ones(H), 1e-6)


def test_gammas_of_zero_and_negative():
    x, gamma = rows_input(3, 256, f32, 12), torch.randn(256, generator=gen(13))
    gamma[::3] = 0.0
    check_rows(x, gamma, 1e-6)
    check_rows(x, torch.zeros(256), 1e-6)


def test_rows_around_are_left_alone():
    T, H = 5, 77
    x = rows_input(T, H, bf16, 14)
    q = torch.full((T + 2, H), 55, dtype=torch.int8, device="cuda")
    s = torch.full((T + 2,), 55.0, device="cuda")
    B.luce_quantize_i8(x.cuda(), q[1:T + 1], s[1:T + 1])
    assert torch.all(q[0] == 55) and torch.all(q[T + 1] == 55) and s[0] == 55 and s[T + 1] == 55
    same(q[1:T + 1], O.rows_i8(x)[0])
    B.luce_quantize_i8(x.cuda()[:0], q[:0], s[:0])  # no rows: nothing


# ----------------------------------------------------------------------------- the int8 product
def codes(rows, cols, seed, lo=-127, hi=127):
    return torch.randint(lo, hi + 1, (rows, cols), generator=gen(seed), dtype=torch.int32).to(torch.int8)


def check_linear(T, N, K, dtype=f32, bias=True, seed=1, xq=None, wq=None, gap=0, stream=None):
    xq = codes(T, K, seed) if xq is None else xq
    wq = codes(N, K, seed + 1) if wq is None else wq
    xs, ws = torch.rand(T, generator=gen(seed + 2)) * 0.01, torch.rand(N, generator=gen(seed + 3)) * 0.01
    b = torch.randn(N, generator=gen(seed + 4)) if bias else None
    ref = O.linear_i8(xq, xs, wq, ws, b, dtype)
    wide = torch.full((T, N + gap), 77.0, dtype=dtype, device="cuda")
    out = wide[:, :N]
    B.luce_linear_i8(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), None if b is None else b.cuda(), out, stream)
    torch.cuda.synchronize()
    same(out, ref)
    assert torch.all(wide[:, N:] == 77.0)
    return out


TS = [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 31, 33, 61, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300, 513]


@pytest.mark.parametrize("N,K", [(1, 16), (7, 48), (127, 64), (128, 1024), (129, 1040), (257, 2064), (1000, 112)])
@pytest.mark.parametrize("T", TS)
def test_linear_sizes(T, N, K):
    check_linear(T, N, K, [f32, bf16, f16][(T + N) % 3], bias=(T + N) % 2 == 0, seed=T * 7 + N)


@pytest.mark.parametrize("dtype", [f32, bf16, f16])
@pytest.mark.parametrize("T,N,K", [(1, 2048, 2048), (5, 3001, 4096), (61, 4096, 4096), (140, 5000, 2048), (512, 4096, 1024),
                                   (1030, 640, 4096), (6, 100, 9184), (40, 300, 9184), (300, 300, 9184)])
def test_linear_working_sizes(T, N, K, dtype):
    check_linear(T, N, K, dtype, bias=T % 2 == 0)


# few and many tiles of every width, with and without a split of K
TILES = [(37, 165, 16), (22, 39, 352), (17, 10421, 16), (373, 19, 1936), (1281, 398, 16), (465, 18, 2752), (810, 2188, 16),
         (697, 19, 3216), (50, 10020, 3616), (51, 4875, 5200), (475, 14942, 16), (1219, 165, 2848), (354, 16147, 16),
         (1395, 137, 4864), (137, 13219, 800), (130, 3554, 3952), (325, 6638, 1696), (210, 12862, 1296), (232, 13600, 2128),
         (223, 620, 16), (9, 3957, 1344), (17, 1759, 2160), (639, 58, 2224), (680, 36, 4768)]


@pytest.mark.parametrize("T,N,K", TILES)
def test_linear_tiles_of_every_width(T, N, K):
    check_linear(T, N, K, f32, bias=True, seed=T)
    full = lambda r, v: torch.full((r, K), v, dtype=torch.int8)  # noqa: E731
    check_linear(T, N, K, f32, xq=full(T, 127), wq=full(N, 125))


@pytest.mark.parametrize("T,N,K", [(9, 21891, 10240), (32, 20480, 5120), (70, 20480, 6144), (260, 9800, 8192)])
def test_linear_a_last_round_of_few_tiles(T, N, K):
    # the channels behind the whole rounds of tiles, in their own launch: bias, scales and stride go with them
    check_linear(T, N, K, bf16, bias=True, gap=6, seed=T)
    assert B.luce_get_fault() == 0


@pytest.mark.parametrize("T,N,K", [(9, 1, 16), (16, 33, 4096), (17, 500, 1040), (70, 130, 9184), (250, 64, 8192),
                                   (524280, 2, 16), (524281, 3, 16)])
def test_linear_eight_tokens_at_a_time(T, N, K):
    # few weights: the last tokens fill an eighth, or all; as many eights as a grid holds, and more
    check_linear(T, N, K, bf16, bias=True, seed=T)


@pytest.mark.parametrize("K", [1008, 1024, 1040, 2048, 4096, 16384, 65536])
@pytest.mark.parametrize("T", [1, 7, 20, 100, 300])
def test_linear_sums_are_exact_at_the_largest_codes(T, K):
    # every product is 127^2 or 128^2 with one sign: the largest sums there are
    N = 130
    full = lambda r, v: torch.full((r, K), v, dtype=torch.int8)  # noqa: E731
    check_linear(T, N, K, xq=full(T, 127), wq=full(N, 127))
    check_linear(T, N, K, xq=full(T, -128), wq=full(N, -128))
    x, w = full(T, 127), full(N, -128)
    x[:, ::2], w[:, 1::3] = -127, 125  # and sums that end near zero, of low bits
    check_linear(T, N, K, xq=x, wq=w)


@pytest.mark.parametrize("T,N,K", [(3, 40, 512), (100, 3000, 512), (100, 3000, 1040), (300, 12000, 512), (300, 12000, 1024)])
def test_linear_sums_of_nothing_are_positive_zeros(T, N, K):
    # zeros times negative codes: the sum's sign is an int32's, whatever the kernel
    out = torch.empty((T, N), device="cuda")
    ones = torch.ones(max(T, N), device="cuda")
    x = torch.zeros((T, K), dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -7, dtype=torch.int8, device="cuda")
    for xq, wq in ((x, w), (torch.full_like(x, -3), torch.zeros_like(w))):
        B.luce_linear_i8(xq, ones[:T], wq, ones[:N], None, out)
        assert torch.all(out == 0) and not torch.any(torch.signbit(out))


@pytest.mark.parametrize("T", [1, 6, 30, 130, 280])
def test_linear_into_a_slice_of_wider_rows(T):
    check_linear(T, 260, 512, f32, gap=12)
    check_linear(T, 131, 512, bf16, gap=5)
    check_linear(T, 128, 512, f16, gap=128)


@pytest.mark.parametrize("T", [5, 40, 100, 300])
def test_linear_many_tiles_and_launches(T):
    # several tiles per CTA, launches back to back: stages, slots and accumulators
    # go round many times (weights from memory, whose tiles land in any order)
    N, K, n = 60000, 2048, 4
    g = torch.Generator(device="cuda").manual_seed(T)
    wq = torch.empty((n, N, K), dtype=torch.int8, device="cuda").random_(-127, 128, generator=g)
    xq = codes(T, K, 3).cuda()
    xs, ws = torch.rand(T, generator=gen(5)).cuda(), torch.rand(N, generator=gen(6)).cuda()
    out = torch.empty((n, T, N), device="cuda")
    for r in range(20):
        for i in range(n):
            B.luce_linear_i8(xq, xs, wq[i], ws, None, out[i])
        if r in (0, 19):
            first = out.clone() if r == 0 else first
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    for i in range(n):
        at = torch.randint(0, N, (200,), generator=gen(i)).cuda()
        at[:4] = torch.tensor([0, 127, 128, N - 1])
        same(out[i][:, at], O.linear_i8(xq.cpu(), xs.cpu(), wq[i][at].cpu(), ws[at].cpu(), None, f32))


def test_linear_rows_do_not_depend_on_the_batch():
    N, K, T = 700, 2048, 300
    xq, wq = codes(T, K, 3), codes(N, K, 4)
    xs, ws = torch.rand(T, generator=gen(5)).cuda(), torch.rand(N, generator=gen(6)).cuda()
    xq, wq = xq.cuda(), wq.cuda()
    whole = torch.empty((T, N), device="cuda")
    B.luce_linear_i8(xq, xs, wq, ws, None, whole)
    for n in (1, 4, 8, 13, 64, 100, 256):
        part = torch.empty((n, N), device="cuda")
        B.luce_linear_i8(xq[:n], xs[:n], wq, ws, None, part)
        same(part, whole[:n])


def test_linear_scales_that_are_zero_or_nan():
    T, N, K = 20, 64, 256
    xq, wq = codes(T, K, 3).cuda(), codes(N, K, 4).cuda()
    xs, ws = torch.ones(T, device="cuda"), torch.ones(N, device="cuda")
    xs[3], xs[4] = math.nan, 0.0
    out = torch.empty((T, N), device="cuda")
    B.luce_linear_i8(xq, xs, wq, ws, None, out)
    assert torch.all(torch.isnan(out[3])) and torch.all(out[4] == 0) and torch.isfinite(out[5:]).all()


def test_linear_large_offsets():
    # weights beyond 2^31 bytes: the last channels are those of a small product
    N, K, T = 40000, 65536, 3
    wq = torch.empty((N, K), dtype=torch.int8, device="cuda")
    wq.random_(-127, 128, generator=torch.Generator(device="cuda").manual_seed(9))
    xq = codes(T, K, 10).cuda()
    xs, ws = torch.ones(T, device="cuda"), torch.rand(N, device="cuda")
    for t in (T, 40):
        x = xq[:1].repeat(t, 1) if t > T else xq
        s = torch.ones(t, device="cuda")
        out, tail = torch.empty((t, N), device="cuda"), torch.empty((t, 64), device="cuda")
        B.luce_linear_i8(x, s, wq, ws, None, out)
        B.luce_linear_i8(x, s, wq[-64:].clone(), ws[-64:].clone(), None, tail)
        same(out[:, -64:], tail)
        same(tail, O.linear_i8(x.cpu(), s.cpu(), wq[-64:].cpu(), ws[-64:].cpu(), None, f32))


# ----------------------------------------------------------------------------- logits
def logits_case(R, V, dtype=f32, hist=50, prompt=20, bias=0, mask=False, seed=1):
    g = gen(seed)
    c = dict(logits=(torch.randn((R, V), generator=g) * 3).to(dtype))
    if hist is not None:
        h = (torch.rand((R, hist), generator=g) ** 3 * V).to(torch.int32).clamp_(0, V - 1)
        if hist > 3:
            h[:, 1] = -1  # padding inside a history
            h[:, 2] = V - 1
        c["hist"] = h
        c["hist_len"] = torch.tensor([hist - (7 * r) % (hist + 1) for r in range(R)], dtype=torch.int32)
        c["prompt_len"] = torch.full((R,), prompt, dtype=torch.int32)
        c["repetition"], c["frequency"], c["presence"] = (torch.rand(R, generator=g) + o for o in (0.7, -0.3, -0.2))
    if bias:
        ids = torch.randint(-1, V, (R, bias), generator=g, dtype=torch.int32)
        if bias > 2:
            ids[:, 0] = ids[:, bias - 1]  # listed twice: the last entry counts
        c["bias_ids"], c["bias_vals"] = ids, torch.randn((R, bias), generator=g) * 5
    if mask:
        m = max(1, R // 2 + 1)
        c["mask"] = torch.randint(-2**31, 2**31, (m, (V + 31) // 32), generator=g).to(torch.int32)
        c["mask"][m - 1] = 0  # allows nothing
        c["mask_rows"] = torch.tensor([(r % (m + 1)) - 1 for r in range(R)], dtype=torch.int32)
    return c


def run_logits(c, gap_in=0, gap_out=0, in_place=False, shift=0):
    R, V = c["logits"].shape
    wide = torch.full((R, V + gap_in + shift), 9.0, dtype=c["logits"].dtype, device="cuda")
    l = wide[:, shift:V + shift]
    l.copy_(c["logits"])
    wide_out = torch.full((R, V + gap_out), 33.0, device="cuda")
    out = l if in_place else wide_out[:, :V]
    kw = {k: v.cuda() for k, v in c.items() if k != "logits"}
    B.luce_logits_process(l, out, **kw)
    torch.cuda.synchronize()
    assert torch.all(wide_out[:, V:] == 33.0) and torch.all(wide[:, V + shift:] == 9.0)
    return out


def check_logits(c, **how):
    same(run_logits(c, **how), O.logits_process(**c))


VS = [1, 2, 5, 31, 32, 33, 64, 100, 1000, 1023, 4096, 4097, 8191, 16384, 16389, 33000]


@pytest.mark.parametrize("V", VS)
@pytest.mark.parametrize("dtype", [f32, bf16, f16])
def test_logits_sizes(V, dtype):
    check_logits(logits_case(3, V, dtype, hist=40, bias=5, mask=True, seed=V))
    check_logits(logits_case(1, V, dtype, hist=7, seed=V + 1))


@pytest.mark.parametrize("hist", [None, 0, 1, 2, 255, 1024, 1025, 5000])
@pytest.mark.parametrize("V", [50, 5000, 40001])
def test_logits_histories(V, hist):
    check_logits(logits_case(2, V, hist=hist, prompt=(hist or 0) // 2, bias=3))


@pytest.mark.parametrize("groups", [(), ("hist",), ("bias",), ("mask",), ("hist", "bias"), ("hist", "mask"), ("bias", "mask")])
@pytest.mark.parametrize("V", [777, 20000])
def test_logits_groups_may_be_left_out(groups, V):
    check_logits(logits_case(4, V, hist=30 if "hist" in groups else None, bias=9 if "bias" in groups else 0,
                             mask="mask" in groups))
    c = logits_case(4, V, hist=30)
    for drop in (("prompt_len",), ("repetition",), ("frequency", "presence"), ("repetition", "frequency", "presence")):
        check_logits({k: v for k, v in c.items() if k not in drop})


@pytest.mark.parametrize("R", [1, 2, 5, 40, 300])
def test_logits_rows(R):
    check_logits(logits_case(R, 3001, bf16, hist=64, prompt=13, bias=7, mask=True, seed=R))


@pytest.mark.parametrize("how", [dict(gap_in=3), dict(gap_out=5), dict(gap_in=4, gap_out=8), dict(gap_in=8, gap_out=3, shift=1),
                                 dict(gap_in=3, shift=1), dict(in_place=True), dict(in_place=True, gap_in=7, shift=2)])
@pytest.mark.parametrize("V", [1000, 4099, 20000])
def test_logits_strides_and_in_place(how, V):
    check_logits(logits_case(3, V, hist=40, bias=5, mask=True), **how)


def test_logits_infinities_and_nans_under_a_mask():
    c = logits_case(4, 400, hist=60, bias=4, mask=True)
    c["logits"][:, ::5] = math.nan
    c["logits"][:, 1::5] = -math.inf
    c["logits"][:, 2::7] = math.inf
    c["logits"][:, 3::7] = torch.finfo(f32).min
    c["mask_rows"] = torch.tensor([0, 1, 2, -1], dtype=torch.int32)
    check_logits(c)
    out = run_logits(c).cpu()
    assert torch.all(out[2] == -math.inf)  # a mask that allows nothing, whatever stood there


@pytest.mark.parametrize("V,hist", [(300, 30000), (129280, 30000)])
def test_logits_one_token_again_and_again(V, hist):
    # a history of a single token (every count in one word), and one with all lengths out of bounds
    c = logits_case(2, V, hist=hist, prompt=100)
    c["hist"][:] = 5
    c["hist_len"] = torch.tensor([hist + 1000, -3], dtype=torch.int32)
    check_logits(c)


@pytest.mark.parametrize("hist", [32767, 32768, 32769, 40000])
@pytest.mark.parametrize("V", [200, 60001])
def test_logits_the_longest_histories_of_either_slot_width(V, hist):
    # sixteen-bit slots count 32,767 of a token: rows of one token alone, and of all others
    c = logits_case(3, V, hist=hist, prompt=0, bias=2)
    c["hist"][0] = V - 1
    c["hist"][1] = torch.arange(hist) % V
    c["hist_len"][:] = hist
    check_logits(c)
    c["prompt_len"] = torch.tensor([hist, hist - 1, hist + 5], dtype=torch.int32)
    check_logits(c)


@pytest.mark.parametrize("V,nbias,hist", [(300, 2000, 5), (50000, 2000, None), (140000, 40, 9), (3000, 65534, 5), (3000, 65535, None)])
def test_logits_many_biases_and_no_room_for_their_places(V, nbias, hist):
    # ids many times over: the last entry counts, in either slot width, beside the counts or behind them
    R = 320 if V == 140000 else 2
    check_logits(logits_case(R, V, bf16 if V == 140000 else f32, hist=hist, prompt=2, bias=nbias, mask=True))


def test_logits_repetition_of_extreme_values():
    V = 64
    l = torch.tensor([1e-44, 3e-39, 1.2e-38, 3e38, 1.0, -1e-44, -3e38, 7.0] * 8)
    for rep in (1e-30, 0.3, 3.0, 1e30, 0.0, math.inf):
        c = logits_case(1, V, hist=V, prompt=V)
        c["logits"][0], c["hist"][0] = l, torch.arange(V, dtype=torch.int32)
        c["hist_len"][:] = V
        c["repetition"] = torch.tensor([rep])
        check_logits({k: v for k, v in c.items() if k not in ("frequency", "presence")})


@pytest.mark.parametrize("e", [-130, -126, -64, -63, -40, 0, 40, 64, 65, 127])
def test_logits_repetition_at_every_magnitude(e):
    # all four logits of a step of one magnitude, over penalties on both sides of 2^-40 and 2^40
    V = 4096
    reps = [2.0**-40, math.nextafter(2.0**-40, 0), 2.0**40, 2.0**40 * (1 + 2.0**-23), 1.3, 0.77, 1 + 2.0**-23, 2 - 2.0**-23]
    c = logits_case(len(reps), V, hist=V, prompt=V // 2, seed=e + 200)
    c["logits"] = torch.ldexp(1 + torch.rand((len(reps), V), generator=gen(e + 300)), torch.tensor(e))
    c["logits"][:, ::97] *= -1
    c["logits"][:, 5] = 0.0
    c["hist"][:] = torch.arange(V, dtype=torch.int32)
    c["hist_len"][:] = V
    c["repetition"] = torch.tensor(reps)
    check_logits(c)


@pytest.mark.parametrize("dtype", [f32, bf16, f16])
@pytest.mark.parametrize("V", [3, 4, 6, 7, 8, 9, 13])
def test_logits_rows_of_a_few_steps(V, dtype):
    # rows that start at every place between boundaries of four, whole steps or none in them
    c = logits_case(9, V, dtype, hist=20, bias=4, mask=True, seed=V)
    check_logits(c)
    check_logits(c, gap_in=4, gap_out=8)
    check_logits(c, gap_in=1, gap_out=1)


@pytest.mark.allow_fault
def test_logits_ids_out_of_range_are_skipped_and_raise_the_fault_bit():
    V = 5000
    for where in ("hist", "bias_ids", "mask_rows"):
        assert B.luce_get_fault() == 0
        c = logits_case(3, V, hist=40, bias=5, mask=True)
        c["hist_len"][:] = 40
        if where == "mask_rows":
            c[where][1] = c["mask"].shape[0]
        else:
            c[where][1, 3] = V
            c[where][2, 3] = 2**31 - 1
        check_logits(c)
        assert B.luce_get_fault() == B.LUCE_FAULT_BAD_ID
    c = logits_case(3, V, hist=40)
    c["hist_len"][:] = 20
    c["hist"][:, 30] = V  # behind the length: not read as a token
    check_logits(c)
    assert B.luce_get_fault() == 0


def test_logits_own_mask_row_by_row():
    c = logits_case(4, 700, hist=None, mask=True)
    c["mask"] = torch.randint(-2**31, 2**31, (5, 25), generator=gen(4)).to(torch.int32)  # wider than needed
    del c["mask_rows"]
    check_logits(c)


# ----------------------------------------------------------------------------- streams, graphs, the whole head
def make_head(R, V, H, seed=1):
    g = gen(seed)
    w = torch.randn((V, H), generator=g) * 0.02
    gamma = torch.rand(H, generator=g) + 0.5
    head = GreedyHead(R, gamma.cuda(), 1e-6, LinearI8.from_float(w.cuda()))
    return head, w, gamma


def head_reference(x, res, gamma, w, head, kw):
    wq, ws, _ = O.rows_i8(w)
    same(head.head.wq, wq)
    same(head.head.w_scale, ws.to(f32))
    q, s, xsum = O.rows_i8(x, gamma, 1e-6, res)
    same(head.q, q)
    sc = head.scale.cpu()
    assert torch.all((sc.double() - s).abs() <= SCALE_TOL * s)
    # the product and what follows, from the scales as they are (their sum's order is free)
    l = O.logits_process(O.linear_i8(q, sc, wq, ws.to(f32), None, f32), **kw)
    return l, xsum


@pytest.mark.parametrize("R", [1, 5, 40])
def test_greedy_head_is_its_parts(R):
    V, H = 3001, 512
    head, w, gamma = make_head(R, V, H)
    x, res = (torch.randn((R, H), generator=gen(k)).to(bf16) for k in (2, 3))
    kw = {k: v for k, v in logits_case(R, V, hist=40, bias=3, mask=True).items() if k != "logits"}
    if kw["mask_rows"].numel() > 1:
        kw["mask_rows"].clamp_(max=kw["mask"].shape[0] - 2)  # (a mask that allows nothing has no greedy token)
    xsum = torch.empty_like(x, device="cuda")
    idx, val = head.run(x.cuda(), res.cuda(), xsum, **{k: v.cuda() for k, v in kw.items()})
    torch.cuda.synchronize()
    l, sum_ref = head_reference(x, res, gamma, w, head, kw)
    same(xsum, sum_ref)
    same(head.logits, l)
    top = l.max(dim=1)
    same(val, top.values)
    assert torch.equal(idx.cpu().long(), (l == top.values[:, None]).int().argmax(dim=1))
    idx2, val2 = head.run(x.cuda(), None)  # without a residual and without processing
    torch.cuda.synchronize()
    l2, _ = head_reference(x, None, gamma, w, head, {})
    same(val2, l2.max(dim=1).values)


def test_head_captured_and_replayed_on_two_streams():
    R, V, H = 4, 2000, 256
    kw = {k: v.cuda() for k, v in logits_case(R, V, hist=40, bias=3, mask=True).items() if k != "logits"}
    heads = [make_head(R, V, H, seed=s)[0] for s in (1, 2)]
    xs = [torch.randn((R, H), generator=gen(9 + k)).cuda() for k in (0, 1)]
    want = []
    for hd, x in zip(heads, xs):
        hd.run(x, **kw)
        torch.cuda.synchronize()
        want.append((hd.logits.clone(), hd.argmax.idx.clone()))
    streams, graphs = [torch.cuda.Stream() for _ in heads], []
    for hd, x, st in zip(heads, xs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            hd.run(x, **kw)
        graphs.append(g)
    for hd in heads:
        hd.logits.zero_()
        hd.q.zero_()
    torch.cuda.synchronize()
    for _ in range(3):  # both graphs in flight at once
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for hd, (l, i) in zip(heads, want):
        same(hd.logits, l)
        assert torch.equal(hd.argmax.idx, i)


@pytest.mark.parametrize("T", [3, 20, 100, 300])
def test_linear_captured_with_split_products(T):
    # clusters that split K, captured without a warm-up call of this shape and replayed
    xq, wq = codes(T, 4096, 1).cuda(), codes(384, 4096, 2).cuda()
    xs, ws = torch.rand(T, generator=gen(3)).cuda(), torch.rand(384, generator=gen(4)).cuda()
    out = torch.zeros((T, 384), dtype=f16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.luce_linear_i8(xq, xs, wq, ws, None, out)
    ref = O.linear_i8(xq.cpu(), xs.cpu(), wq.cpu(), ws.cpu(), None, f16)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        same(out, ref)


@pytest.mark.parametrize("T", [1, 20, 300])
def test_calls_on_a_given_stream_and_under_programmatic_launch(T):
    st = torch.cuda.Stream()
    gamma = torch.rand(512, generator=gen(1)) + 0.5
    B.luce_set_pdl(True)
    try:
        check_rows(rows_input(T, 512, bf16, 2), gamma, 1e-6, rows_input(T, 512, bf16, 3), in_place="new", stream=st)
        check_linear(T, 300, 512, stream=st.cuda_stream)
        # back to back, each reading what the one before wrote
        x = rows_input(T, 512, f32, 4)
        w = codes(333, 512, 5)
        ws = torch.rand(333, generator=gen(6))
        q, s = torch.empty((T, 512), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        out, l = torch.empty((T, 333), device="cuda"), torch.empty((T, 333), device="cuda")
        kw = {k: v.cuda() for k, v in logits_case(T, 333, hist=9).items() if k != "logits"}
        xd, wd, wsd = x.cuda(), w.cuda(), ws.cuda()
        torch.cuda.synchronize()
        for _ in range(20):
            B.luce_quantize_i8(xd, q, s)
            B.luce_linear_i8(q, s, wd, wsd, None, out)
            B.luce_logits_process(out, l, **kw)
        torch.cuda.synchronize()
    finally:
        B.luce_set_pdl(False)
    qr, sr, _ = O.rows_i8(x)
    ref = O.linear_i8(qr, sr.to(f32), w, ws, None, f32)
    same(out, ref)
    same(l, O.logits_process(ref, **{k: v.cpu() for k, v in kw.items()}))


def test_both_ways_of_calling_are_one(monkeypatch):
    # the call module takes the common call, the Python code the others: the same results
    x, gamma = rows_input(5, 200, bf16, 1).cuda(), (torch.rand(200, generator=gen(2)) + 0.5).cuda()
    res = rows_input(5, 200, bf16, 3).cuda()
    wq, ws = codes(64, 208, 4).cuda(), torch.rand(64, generator=gen(5)).cuda()
    xq, xs = codes(5, 208, 6).cuda(), torch.rand(5, generator=gen(7)).cuda()
    c = {k: v.cuda() for k, v in logits_case(5, 64, hist=9, bias=3, mask=True).items()}
    logits = c.pop("logits")

    def everything():
        new = lambda *s, dt=f32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        outs = [new(5, 200, dt=torch.int8), new(5), new(5, 200, dt=torch.int8), new(5), new(5, 200, dt=bf16),
                new(5, 200, dt=torch.int8), new(5), new(5, 64), new(5, 70, dt=f16)[:, :64], new(5, 64), new(5, 64)]
        B.luce_quantize_i8(x, outs[0], outs[1])
        B.luce_rmsnorm_i8(x, gamma, 1e-5, outs[2], outs[3])
        B.luce_add_rmsnorm_i8(x, res, outs[4], gamma, 1e-5, outs[5], outs[6])
        B.luce_linear_i8(xq, xs, wq, ws, None, outs[7])
        B.luce_linear_i8(xq, xs, wq, ws, ws, outs[8])
        B.luce_logits_process(logits, outs[9], **c)
        B.luce_logits_process(logits, outs[10])
        torch.cuda.synchronize()
        return outs

    calls = []
    fast = B._fast
    assert fast is not None

    class Counting:
        def __getattr__(self, name):
            def call(*a):
                calls.append(getattr(fast, name)(*a))
                return calls[-1]
            return call

    monkeypatch.setattr(B, "_fast", Counting())
    first = everything()
    assert calls == [0] * 7  # every one of these is a common call
    monkeypatch.setattr(B, "_fast", None)
    for a, b in zip(first, everything()):
        same(a, b)
    monkeypatch.setattr(B, "_fast", fast)
    # what the module leaves alone: other kinds, shapes and layouts
    s = torch.zeros(5, device="cuda")
    q = torch.zeros((5, 200), dtype=torch.int8, device="cuda")
    assert fast.quantize_i8(x, q, s[:4]) == -1 and fast.quantize_i8(x.cpu(), q, s) == -1
    assert fast.quantize_i8(x.t(), q, s) == -1 and fast.quantize_i8(x, q.float(), s) == -1
    assert fast.quantize_i8(None, q, s) == -1 and fast.quantize_i8(x, q) == -1
    assert fast.rmsnorm_i8(x, gamma, 1, q, s) == -1 and fast.rmsnorm_i8(x, gamma[:9], 1e-5, q, s) == -1
    assert fast.linear_i8(xq, xs, wq[:, :192], ws, None, first[7]) == -1
    assert fast.logits_process(logits, logits, *[None] * 9, s.int()) == -1
    assert fast.rmsnorm_i8(x, gamma, -1.0, q, s) == B.LUCE_ERR_INVALID_ARG  # the library's own refusals come through
    with pytest.raises(B.LuceError):
        B.luce_rmsnorm_i8(x, gamma, -1.0, q, s)


def test_bindings_check_shapes():
    x = torch.zeros((4, 64), device="cuda")
    q, s = torch.zeros((4, 64), dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    out = torch.zeros((4, 4), device="cuda")
    for call in (lambda: B.luce_quantize_i8(x, q[:3], s), lambda: B.luce_quantize_i8(x, q, s[:3]),
                 lambda: B.luce_quantize_i8(x.t(), q, s), lambda: B.luce_rmsnorm_i8(x, s, 1e-6, q, s),
                 lambda: B.luce_linear_i8(q, s, q[:, :32], s, None, out), lambda: B.luce_linear_i8(q, s, q, s, x[0], out),
                 lambda: B.luce_linear_i8(q, s, q, s, None, out.t()[:, :3].t()),
                 lambda: B.luce_logits_process(x, x[:, :32]), lambda: B.luce_logits_process(x, x, hist=q.int()),
                 lambda: B.luce_logits_process(x, x, hist_len=s.int()), lambda: B.luce_logits_process(x, x, bias_vals=x),
                 lambda: B.luce_logits_process(x, x, repetition=s[:2]), lambda: B.luce_logits_process(x, x, mask_rows=s.int())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: B.luce_quantize_i8(q, q, s), lambda: B.luce_linear_i8(q, s.half(), q, s, None, out),
                 lambda: B.luce_add_rmsnorm_i8(x, x.half(), None, x[0], 1e-6, q, s), lambda: B.luce_logits_process(x, x.half())):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(B.LuceError):
        B.luce_logits_process(x, x, mask=torch.zeros((2, 2), dtype=torch.int32, device="cuda"))  # masks for two rows of four
    with pytest.raises(B.LuceError):
        B.luce_linear_i8(q[:, :40].contiguous(), s, q[:, :40].contiguous(), s, None, out)  # K
