"""The definitions of the int8 decode-head operators (oracle/head.py), pinned
to hand-worked values and closed forms, and the refusals of their entry points
(host checks only: nothing here reaches a kernel)."""
import ctypes
import math

import pytest
import torch

from oracle import head as O
from quantized_moe_decode_luce_gb300 import binding as Bd
from quantized_moe_decode_luce_gb300 import build as B

f32 = torch.float32


# ----------------------------------------------------------------------------- definitions
def test_quantize_hand_worked_row():
    # m = 127, d = 1: the codes are the values, halves away from zero
    x = torch.tensor([[127.0, -127.0, 0.5, -0.5, 1.5, -2.5, 0.49999997, 63.5]])
    q, s, _ = O.rows_i8(x)
    assert q.tolist() == [[127, -127, 1, -1, 2, -3, 0, 64]] and s.tolist() == [1.0]


def test_quantize_is_the_nearest_code_and_negation_mirrors():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((7, 300), generator=g)
    q, s, _ = O.rows_i8(x)
    assert torch.all((x.double() - q.double() * s[:, None]).abs() <= s[:, None] * (0.5 + 127 * 2.0 ** -23))
    q2, s2, _ = O.rows_i8(-x)
    assert torch.equal(q2, -q) and torch.equal(s, s2)
    assert torch.equal(q.abs().amax(dim=1), torch.full((7,), 127, dtype=torch.int8))


def test_norm_of_constant_rows_and_scale_invariance():
    x = torch.full((1, 64), 3.0)
    q, s, _ = O.rows_i8(x, torch.ones(64), 0.0)
    assert torch.all(q == 127) and abs(float(s[0]) * 127 - 1.0) < 1e-6  # a constant row norms to ones
    g = torch.Generator().manual_seed(2)
    y, gam = torch.randn((3, 96), generator=g), torch.rand(96, generator=g) + 0.5
    qa, sa, _ = O.rows_i8(y, gam, 0.0)
    qb, sb, _ = O.rows_i8(y * 8.0, gam, 0.0)  # a power of two moves neither codes nor scale
    assert torch.equal(qa, qb) and torch.allclose(sa, sb, rtol=1e-12)
    # the values stand for the norm
    n = y.double() / y.double().square().mean(dim=1, keepdim=True).sqrt() * gam.double()
    assert torch.all((qa.double() * sa[:, None] - n).abs() <= sa[:, None] * 0.5001)


def test_rows_with_nothing_or_with_infinities():
    x = torch.zeros((4, 32))
    x[1, 3], x[2, 5] = math.inf, math.nan
    x[3, 0] = 1.0
    q, s, _ = O.rows_i8(x, torch.ones(32), 1e-6)
    assert torch.all(q[:3] == 0) and s[0] == 0.0 and math.isnan(s[1]) and math.isnan(s[2])
    assert q[3, 0] == 127
    tiny = torch.full((1, 2), 2.0 ** -149)  # d rounds to zero
    q, s, _ = O.rows_i8(tiny)
    assert torch.all(q == 0) and s[0] == 0.0
    some = torch.full((1, 2), 190 * 2.0 ** -149)  # d rounds down to 2^-149: codes stay within 127
    q, s, _ = O.rows_i8(some)
    assert torch.all(q == 127)


def test_residual_sum_is_rounded_to_the_type_before_the_norm():
    x, r = torch.tensor([[1.0, 256.0]], dtype=torch.bfloat16), torch.tensor([[0.0, 1.0]], dtype=torch.bfloat16)
    _, _, s = O.rows_i8(x, torch.ones(2), 0.0, r)
    assert s.tolist() == [[1.0, 256.0]]  # 257 has nine bits: half way, to even


def test_linear_hand_worked():
    xq = torch.tensor([[1, -2, 3, 4]], dtype=torch.int8)
    wq = torch.tensor([[5, 6, 7, 8], [-128, 127, 0, 1]], dtype=torch.int8)
    y = O.linear_i8(xq, torch.tensor([0.5]), wq, torch.tensor([2.0, 0.25]), torch.tensor([1.0, 0.0]), f32)
    assert y.tolist() == [[46.0 + 1.0, (-128 - 254 + 4) * 0.125]]


def test_logits_hand_worked_row():
    l = torch.tensor([[2.0, -2.0, 1.0, 0.0, 5.0, math.nan]])
    hist = torch.tensor([[0, 1, 2, 2, -1, 4]], dtype=torch.int32)
    kw = dict(hist=hist, hist_len=torch.tensor([5]), prompt_len=torch.tensor([2]), repetition=torch.tensor([2.0]),
              frequency=torch.tensor([0.25]), presence=torch.tensor([0.5]))
    out = O.logits_process(l, **kw)
    # 0 and 1 are the prompt's; 2 came twice; the padding and the id behind the length count for nothing
    assert out[0, :5].tolist() == [1.0, -4.0, 0.5 - (2 * 0.25 + 0.5), 0.0, 5.0] and math.isnan(out[0, 5])
    out = O.logits_process(l, **kw, bias_ids=torch.tensor([[4, 4, -1]], dtype=torch.int32),
                           bias_vals=torch.tensor([[9.0, 1.0, 7.0]]),
                           mask=torch.tensor([[0b010100]], dtype=torch.int32))
    assert out[0].tolist() == [-math.inf, -math.inf, -0.5, -math.inf, 6.0, -math.inf]


# ----------------------------------------------------------------------------- refusals of the C entry points
GOOD, FAR, FAR2, FAR3 = 0x10000, 0x20000000, 0x40000000, 0x60000000  # aligned addresses that nothing is launched with
vp, ci, cf, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int64


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(B.build())


def test_quantize_i8_refusals(lib):
    f = lib.luce_quantize_i8
    f.argtypes = [vp, ci, ci, ci, vp, vp, vp]
    ok = [GOOD, 0, 4, 64, FAR, FAR2, None]

    def bad(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)
    assert bad(a1=3) == 1 and bad(a1=-1) == 1                       # dtype
    assert bad(a2=-1) == 1 and bad(a3=0) == 1 and bad(a3=65537) == 1
    assert bad(a0=None) == 1 and bad(a4=None) == 1 and bad(a5=None) == 1
    assert bad(a0=GOOD + 2) == 1 and bad(a1=1, a0=GOOD + 1) == 1    # alignment to the element
    assert bad(a5=FAR2 + 2) == 1
    assert bad(a4=GOOD + 16) == 1 and bad(a5=GOOD) == 1 and bad(a5=FAR) == 1  # outputs over an input, or over each other
    assert bad(a2=0, a0=None) == 0                                  # an empty call


def test_rmsnorm_i8_refusals(lib):
    f = lib.luce_rmsnorm_i8
    f.argtypes = [vp, ci, vp, cf, ci, ci, vp, vp, vp]
    G2 = GOOD + (1 << 20)
    assert f(GOOD, 0, None, 1e-6, 4, 64, FAR, FAR2, None) == 1      # gamma missing
    assert f(GOOD, 0, G2, -1.0, 4, 64, FAR, FAR2, None) == 1
    assert f(GOOD, 0, G2, math.nan, 4, 64, FAR, FAR2, None) == 1
    assert f(GOOD, 0, G2, math.inf, 4, 64, FAR, FAR2, None) == 1
    assert f(GOOD, 0, G2 + 1, 1e-6, 4, 64, FAR, FAR2, None) == 1
    assert f(GOOD, 0, G2, 1e-6, 4, 64, G2, FAR2, None) == 1         # codes over gamma
    assert f(GOOD, 0, None, 1e-6, 0, 64, FAR, FAR2, None) == 0
    a = lib.luce_add_rmsnorm_i8
    a.argtypes = [vp, vp, vp, ci, vp, cf, ci, ci, vp, vp, vp]
    R = FAR3
    assert a(GOOD, None, None, 0, G2, 1e-6, 4, 64, FAR, FAR2, None) == 1            # residual missing
    assert a(GOOD, R, GOOD + 16, 0, G2, 1e-6, 4, 64, FAR, FAR2, None) == 1          # the sum half over x
    assert a(GOOD, R, R + 4, 0, G2, 1e-6, 4, 64, FAR, FAR2, None) == 1              # ... over the residual
    assert a(GOOD, R, FAR, 0, G2, 1e-6, 4, 64, FAR, FAR2, None) == 1                # ... over the codes
    assert a(GOOD, R, G2, 0, G2, 1e-6, 4, 64, FAR, FAR2, None) == 1                 # ... over gamma
    assert a(GOOD, R + 1, None, 1, G2, 1e-6, 4, 64, FAR, FAR2, None) == 1
    assert a(GOOD, None, None, 0, None, 1e-6, 0, 64, FAR, FAR2, None) == 0


def test_linear_i8_refusals(lib):
    f = lib.luce_linear_i8
    f.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, vp, ci, i64, vp]
    XS, WS, BI = FAR3, FAR3 + 4096, FAR3 + 8192
    ok = [GOOD, XS, FAR, WS, BI, 4, 32, 64, FAR2, 0, 32, None]

    def bad(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)
    assert bad(a7=40) == 1 and bad(a7=0) == 1 and bad(a7=65552) == 1   # K
    assert bad(a5=-1) == 1 and bad(a6=0) == 1 and bad(a5=1 << 24) == 1 and bad(a6=1 << 24) == 1
    assert bad(a9=5) == 1 and bad(a10=31) == 1
    assert bad(a0=GOOD + 8) == 1 and bad(a2=FAR + 4) == 1              # codes 16-byte aligned
    assert bad(a8=FAR2 + 2) == 1 and bad(a8=FAR2 + 1, a9=1) == 1
    for i in (0, 1, 2, 3, 8):
        assert bad(**{f"a{i}": None}) == 1
    assert bad(a8=GOOD) == 1 and bad(a8=FAR) == 1 and bad(a8=XS) == 1 and bad(a8=WS) == 1 and bad(a8=BI) == 1
    assert bad(a4=BI + 2) == 1
    assert bad(a5=0, a0=None) == 0


def test_logits_process_refusals(lib):
    f = lib.luce_logits_process
    f.argtypes = [vp, ci, ci, i64, i64, vp, i64, vp, vp, vp, vp, vp, vp, vp, ci, vp, ci, i64, vp, vp, i64, vp]
    S = FAR3
    #     0     1  2  3     4     5  6  7          8          9  10 11 12         13        14 15        16 17 18 19   20    21
    ok = [GOOD, 0, 2, 1000, 1000, S, 8, S + 4096, S + 8192, S, S, S, S + 12288, S + 16384, 4, S + 20480, 2, 32, None,
          FAR, 1000, None]

    def bad(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)
    assert bad(a1=3) == 1 and bad(a2=-1) == 1 and bad(a2=65536) == 1
    assert bad(a3=0) == 1 and bad(a3=1 << 31, a4=1 << 31, a20=1 << 31) == 1
    assert bad(a4=999) == 1 and bad(a20=999) == 1                # rows that overlap
    assert bad(a7=None) == 1 and bad(a5=None) == 1               # a history without lengths, lengths without one
    assert bad(a6=-1) == 1 and bad(a14=-1) == 1
    assert bad(a12=None) == 1 and bad(a13=None) == 1
    assert bad(a17=31) == 1 and bad(a16=1) == 1 and bad(a16=0) == 1  # words a mask, masks for the rows
    assert bad(a15=None, a18=S) == 1                             # mask rows without masks
    assert bad(a0=GOOD + 2) == 1 and bad(a19=FAR + 2) == 1 and bad(a5=S + 1) == 1
    assert bad(a0=None) == 1 and bad(a19=None) == 1
    assert bad(a19=GOOD + 4) == 1                                # half over the logits
    assert bad(a1=1, a19=GOOD) == 1                              # in place needs fp32 logits
    assert bad(a19=GOOD, a20=1001) == 1                          # ... and their row stride
    assert bad(a19=S) == 1 and bad(a19=S + 20480) == 1           # over the history, over the masks
    assert bad(a2=0, a0=None) == 0


def test_bindings_refuse_what_is_not_theirs():
    x = torch.zeros((2, 64))
    with pytest.raises(TypeError):
        Bd.luce_quantize_i8(x, torch.zeros((2, 64), dtype=torch.int8), torch.zeros(2))  # not on a GPU
    with pytest.raises(TypeError):
        Bd.luce_linear_i8(x, None, x, None, None, x)
    with pytest.raises(TypeError):
        Bd.luce_logits_process(x, x)
