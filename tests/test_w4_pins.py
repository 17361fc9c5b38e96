"""The definitions behind the 4-bit products and the draw, on hand-worked cases, and the calls that the library refuses
(no GPU needed: nothing is launched)."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import draw as D
from oracle import w4 as O
from quantized_moe_decode_luce_gb300 import binding as Bd
from quantized_moe_decode_luce_gb300 import build as B
from quantized_moe_decode_luce_gb300.layer import GreedyHead, LinearI8, LinearW4, SampleHead

vp, ci, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64


# ----------------------------------------------------------------------------- packed codes
@pytest.mark.parametrize("K", [16, 128, 144, 400])
def test_packed_codes_come_back(K):
    q = torch.randint(0, 16, (5, K), generator=torch.Generator().manual_seed(K), dtype=torch.uint8)
    p = O.pack(q)
    assert p.shape == (5, O.row_bytes(K)) and O.row_bytes(K) == Bd.w4_row_bytes(K)
    assert torch.equal(O.unpack(p, K), q)


@pytest.mark.parametrize("k,byte,upper", [(0, 0, False), (1, 2, False), (2, 0, True), (3, 2, True), (4, 1, False), (7, 3, True),
                                          (8, 16, False), (31, 51, True), (32, 4, False), (127, 63, True), (128, 64, False)])
def test_where_a_code_is(k, byte, upper):
    # word 4 t + j of a chunk holds the values 32 j + 8 t + i, value i in its bits 4 (i / 2) + 16 (i % 2) .. + 3
    q = torch.zeros((1, 256), dtype=torch.uint8)
    q[0, k] = 9
    p = O.pack(q)[0]
    assert p.nonzero().flatten().tolist() == [byte] and int(p[byte]) == (9 * 16 if upper else 9)


def test_a_group_by_hand():
    w = torch.zeros((1, 32))
    w[0, :4] = torch.tensor([7.0, -3.5, 0.4, -7.0])
    q, s, z = O.quantize(w, 32, torch.float16, False)
    assert float(s[0, 0]) == 1.0 and z is None and q[0, :5].tolist() == [15, 4, 8, 1, 8]  # -3.5 goes away from zero
    w[0, :3] = torch.tensor([10.0, -5.0, 2.5])
    w[0, 3] = 0.0
    q, s, z = O.quantize(w, 32, torch.float16, True)
    assert float(s[0, 0]) == 1.0 and int(z[0, 0]) == 5 and q[0, :4].tolist() == [15, 0, 8, 5]
    w[0, 1] = math.inf
    q, s, z = O.quantize(w, 32, torch.bfloat16, False)
    assert torch.isnan(s[0, 0]) and torch.all(q == 8)


def test_products_by_hand():
    codes = torch.tensor([[8, 9, 7, 8] * 8 + [15] * 16], dtype=torch.uint8)
    scale = torch.tensor([[0.5, 2.0]], dtype=torch.float16)
    x = torch.arange(48, dtype=torch.float32)[None]
    want = sum(Fraction(k) * (int(codes[0, k]) - 8) * (Fraction(1, 2) if k < 32 else 2) for k in range(48))
    y, terms, rest = O.linear(x, None, codes, scale, None, 32)
    assert y.item() == float(want) and terms.item() >= abs(y.item()) and rest.item() > 0
    zeros = torch.tensor([[9, 15]], dtype=torch.uint8)
    want = sum(Fraction(k) * (int(codes[0, k]) - (9 if k < 32 else 15)) * (Fraction(1, 2) if k < 32 else 2) for k in range(48))
    assert O.linear(x, torch.tensor([0.25]), codes, scale, zeros, 32, torch.tensor([1.0]))[0].item() == float(want / 4 + 1)


# ----------------------------------------------------------------------------- the draw
def test_draws_by_hand():
    l = np.log([1.0, 2.0, 4.0, 1.0])
    for u, want in ((0.0, 0), (0.1249, 0), (0.126, 1), (0.374, 1), (0.376, 2), (0.874, 2), (0.876, 3), (1.0, 3), (math.nan, 0), (-1.0, 0)):
        i, p, _ = D.draw(l, u)
        assert (i, round(p, 9)) == (want, [0.125, 0.25, 0.5, 0.125][want])
    assert D.draw(l, 0.4, top_k=3)[0] == 1  # the first of the two equal ones stays: weights 1, 2, 4
    assert D.draw(l, 0.99, top_k=3)[0] == 2 and D.draw(l, 0.01, top_k=3)[0] == 0
    assert D.draw(l, 0.01, top_k=2)[0] == 1 and D.draw(l, 0.5, top_k=1)[:2] == (2, 1.0)
    assert D.draw(l, 0.99, top_p=0.5)[:2] == (2, 1.0)   # 0 < 4 <= 8 / 2: nothing after it
    assert D.draw(l, 0.01, top_p=0.51)[0] == 1          # 4 < 4.08
    assert D.draw(l, 0.01, top_p=0.0)[0] == 2
    assert D.draw(l, 0.01, min_p=0.5)[0] == 1 and D.draw(l, 0.01, min_p=0.51)[0] == 2
    assert D.draw(l, 0.9, temperature=0.0)[:2] == (2, 1.0)
    assert D.draw([2.0, 5.0, 5.0], 0.9, temperature=0.0)[0] == 1
    i, p, _ = D.draw(l, 0.9, temperature=math.inf)
    assert (i, p) == (3, 0.25)
    assert D.draw([-math.inf, 1.0, -math.inf], 0.99)[:2] == (1, 1.0)
    assert D.draw([-math.inf] * 3, 0.5)[:2] == (0, 0.0)
    for bad in (math.nan, math.inf):
        i, p, _ = D.draw([1.0, bad, 2.0], 0.5)
        assert i == 0 and math.isnan(p)


# ----------------------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(B.build())


W, Q, S, Z, X, OUT, XS, BIAS = (0x10000000 * (i + 1) for i in range(8))  # addresses that nothing reads


def test_quantize_and_pack_refusals(lib):
    f, g = lib.luce_quantize_w4, lib.luce_pack_w4
    f.argtypes, g.argtypes = [vp, ci, ci, ci, ci, vp, vp, ci, vp, vp], [vp, ci, ci, vp, vp]
    ok = dict(w=W, dtype=0, N=0, K=64, group=32, wq=Q, scale=S, sdt=2, zeros=None)

    def call(**kw):
        return f(*{**ok, **kw}.values(), None)
    assert call() == 0 and call(sdt=1, zeros=Z, dtype=1) == 0  # no rows: nothing is launched
    for kw in (dict(N=-1), dict(N=1 << 24), dict(K=24), dict(K=0), dict(K=65552), dict(group=16), dict(group=0), dict(group=256), dict(dtype=3),
               dict(sdt=0), dict(sdt=3), dict(N=4, w=None), dict(N=4, wq=None), dict(N=4, scale=None), dict(N=4, wq=Q + 8),
               dict(N=4, w=W + 2), dict(N=4, scale=S + 1), dict(N=4, wq=W), dict(N=4, scale=Q + 64), dict(N=4, zeros=S + 8)):
        assert call(**kw) == 1, kw
    assert g(W, 0, 64, Q, None) == 0
    for a in ((W, -1, 64, Q), (W, 4, 24, Q), (None, 4, 64, Q), (W, 4, 64, None), (W, 4, 64, Q + 4), (W, 4, 64, W + 240)):
        assert g(*a, None) == 1, a


def test_linear_refusals(lib):
    f = lib.luce_linear_w4
    f.argtypes = [vp, ci, i64, vp, vp, vp, ci, vp, ci, vp, ci, ci, ci, vp, ci, i64, vp]
    ok = dict(x=X, xdt=1, ldx=64, xs=None, wq=Q, ws=S, sdt=2, zeros=None, group=32, bias=None, T=0, N=8, K=64, out=OUT, odt=0, ldo=8)

    def call(**kw):
        return f(*{**ok, **kw}.values(), None)
    assert call() == 0 and call(xdt=3, xs=XS) == 0 and call(zeros=Z, bias=BIAS, odt=2) == 0
    for kw in (dict(T=-1), dict(T=1 << 24), dict(N=0), dict(N=1 << 24), dict(K=72, ldx=72), dict(K=0), dict(K=65552, ldx=65552), dict(group=48),
               dict(sdt=0), dict(odt=3), dict(xdt=4), dict(xdt=-1), dict(ldx=63), dict(ldo=7)):
        assert call(**kw) == 1, kw
    for kw in (dict(x=None), dict(wq=None), dict(ws=None), dict(out=None), dict(x=X + 8), dict(wq=Q + 4), dict(ws=S + 1), dict(out=OUT + 2),
               dict(bias=BIAS + 2), dict(xdt=3), dict(xs=XS), dict(xdt=3, xs=XS + 1), dict(T=2, ldx=68), dict(xdt=3, xs=XS, T=2, ldx=72),
               dict(out=X), dict(out=Q + 480), dict(out=S), dict(zeros=Z, out=Z), dict(bias=BIAS, out=BIAS + 28), dict(xdt=3, xs=OUT)):
        assert call(**{"T": 1, **kw}) == 1, kw


def test_sample_refusals(lib):
    f = lib.luce_sample
    f.argtypes = [vp, ci, ci, i64, i64] + [vp] * 8
    ok = dict(logits=W, dtype=0, R=0, V=100, ld=100, u=Q, t=None, k=None, p=None, m=None, idx=S, prob=Z)

    def call(**kw):
        return f(*{**ok, **kw}.values(), None)
    assert call() == 0 and call(prob=None, dtype=2) == 0 and call(V=393216, ld=393216) == 0
    assert call(V=393217, ld=393217, R=1) == 2 and call(V=(1 << 31) - 1, ld=1 << 31) == 2
    for kw in (dict(R=-1), dict(R=65536), dict(V=0), dict(V=1 << 31, ld=1 << 31), dict(ld=99), dict(ld=(1 << 33) + 1), dict(dtype=3), dict(dtype=-1)):
        assert call(**kw) == 1, kw
    for kw in (dict(logits=None), dict(u=None), dict(idx=None), dict(logits=W + 2), dict(idx=S + 2), dict(prob=Z + 1), dict(u=Q + 1), dict(t=X + 2),
               dict(k=X + 1), dict(p=X + 3), dict(m=X + 2), dict(prob=S + 4), dict(idx=W + 8), dict(prob=W), dict(u=S), dict(t=Z + 4), dict(k=S), dict(m=Z)):
        assert call(**{"R": 2, **kw}) == 1, kw


def test_bindings_look_at_their_arguments(lib):
    x = torch.zeros((2, 64))
    for call in (lambda: Bd.luce_quantize_w4(x, 32, x, x), lambda: Bd.luce_pack_w4(x, x), lambda: Bd.luce_sample(x, x, x),
                 lambda: Bd.luce_linear_w4(x, None, x, x, None, 32, None, x)):
        with pytest.raises(TypeError):  # no CUDA tensor
            call()
    assert Bd.w4_row_bytes(1) == 64 and Bd.w4_row_bytes(128) == 64 and Bd.w4_row_bytes(129) == 128
    with pytest.raises(ValueError):
        Bd._groups(64, 48)
    with pytest.raises(ValueError):
        LinearW4(torch.zeros((4, 64), dtype=torch.uint8), x, 130, 32)


# ----------------------------------------------------------------------------- heads
@pytest.fixture
def calls(monkeypatch, lib):
    made = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # (the device of tensors on the CPU)
    for name in ("luce_rmsnorm_i8", "luce_add_rmsnorm_i8", "luce_linear_i8", "luce_linear_w4", "luce_logits_process", "luce_argmax", "luce_sample"):
        monkeypatch.setattr(Bd, name, lambda *a, name=name, **kw: made.append(name))
    return made


def test_heads_take_either_weights(calls):
    w4 = LinearW4(torch.zeros((100, 64), dtype=torch.uint8), torch.zeros((100, 1)), 32, 32)
    i8 = LinearI8(torch.zeros((100, 32), dtype=torch.int8), torch.zeros(100))
    x, u = torch.zeros((2, 32)), torch.zeros(2)
    for head, product in ((w4, "luce_linear_w4"), (i8, "luce_linear_i8")):
        del calls[:]
        GreedyHead(2, torch.ones(32), 1e-6, head).run(x, x)
        h = SampleHead(2, torch.ones(32), 1e-6, head)
        idx, prob = h.run(x, u, hist=None, top_k=u)
        assert calls == ["luce_add_rmsnorm_i8", product, "luce_argmax", "luce_rmsnorm_i8", product, "luce_logits_process", "luce_sample"]
        assert idx is h.idx and prob is h.prob
        del calls[:]
        with pytest.raises(ValueError):
            h.run(x, u, None, torch.zeros((2, 32)))
        assert calls == []
    with pytest.raises(ValueError):
        SampleHead(2, torch.ones(48), 1e-6, w4)
