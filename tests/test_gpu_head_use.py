"""GPU: the int8 decode head as programs use it -- weights made on the GPU,
launches that start early, streams and threads, the tile of every product --
against the definitions in 64 bits (oracle/head.py), with the helpers and
bounds of test_gpu_head.py.
"""
import pytest
import torch

from oracle import head as O
from quantized_moe_decode_luce_gb300 import binding as B
from quantized_moe_decode_luce_gb300.layer import LinearI8
from test_gpu_head import (_lib, _no_device_faults, bf16, check_rows, codes, f16, f32, gen,  # noqa: F401
                           logits_case, rows_input, same)  # (the fixtures hold for every test here)

pytestmark = pytest.mark.gpu


@pytest.fixture
def pdl():
    B.luce_set_pdl(True)
    yield
    torch.cuda.synchronize()
    B.luce_set_pdl(False)


# ----------------------------------------------------------------------------- launches that start early
@pytest.mark.parametrize("T,N,K", [(1, 2048, 1024), (5, 1000, 4096), (20, 4000, 1024), (300, 8000, 512)])
def test_weights_quantized_just_before_their_product(T, N, K, pdl):
    # the launch before the product writes its weights; the tokens' codes are older
    ws = [torch.randn((N, K), generator=gen(s)) for s in (1, 2)]
    xq, xs = codes(T, K, 3), torch.rand(T, generator=gen(4))
    refs = []
    for w in ws:
        wq, s, _ = O.rows_i8(w)
        refs.append(O.linear_i8(xq, xs, wq, s.to(f32), None, f32))
    wd, xqd, xsd = [w.cuda() for w in ws], xq.cuda(), xs.cuda()
    wq, s = torch.empty((N, K), dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    outs = torch.empty((20, T, N), device="cuda")
    torch.cuda.synchronize()
    for i in range(20):  # the same buffer takes the two weights in turn
        B.luce_quantize_i8(wd[i % 2], wq, s)
        B.luce_linear_i8(xqd, xsd, wq, s, None, outs[i])
    last = LinearI8.from_float(wd[0]).run(xqd, xsd, torch.empty((T, N), device="cuda"))
    torch.cuda.synchronize()
    for i in range(20):
        same(outs[i], refs[i % 2])
    same(last, refs[0])


# ----------------------------------------------------------------------------- masks
@pytest.fixture(params=["call module", "python"])
def both_ways(request, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(B, "_fast", None)


def test_logits_masks_that_hold_nothing_are_refused(both_ways):
    # an empty tensor is a mask all the same: a step with a grammar does not run without it
    x, out = torch.randn((3, 64), generator=gen(1)).cuda(), torch.full((3, 64), 7.0, device="cuda")
    rows = torch.zeros(3, dtype=torch.int32, device="cuda")
    for shape, mask_rows in (((0, 2), None), ((0, 0), None), ((3, 0), None), ((3, 0), rows), ((3, 1), rows), ((2, 2), None)):
        mask = torch.zeros(shape, dtype=torch.int32, device="cuda")
        with pytest.raises(B.LuceError):
            B.luce_logits_process(x, out, mask=mask, mask_rows=mask_rows)
    torch.cuda.synchronize()
    assert torch.all(out == 7.0)
    B.luce_logits_process(x[:0], out[:0], mask=torch.zeros((0, 2), dtype=torch.int32, device="cuda"))  # no rows: nothing


@pytest.mark.allow_fault
@pytest.mark.parametrize("groups", [(), ("hist", "bias")])
def test_logits_rows_without_a_mask_need_no_masks(groups, both_ways):
    V = 5000
    c = logits_case(3, V, hist=30 if "hist" in groups else None, bias=4 if "bias" in groups else 0)
    want = O.logits_process(**c)
    kw = {k: v.cuda() for k, v in c.items()}
    out = torch.empty((3, V), device="cuda")
    for words in ((V + 31) // 32, 0):
        none = torch.zeros((0, words), dtype=torch.int32, device="cuda")
        for rows, fault in (([-1, -1, -1], 0), ([-1, 0, -1], B.LUCE_FAULT_BAD_ID)):
            out.fill_(9.0)
            B.luce_logits_process(out=out, mask=none, mask_rows=torch.tensor(rows, dtype=torch.int32, device="cuda"), **kw)
            same(out, want)
            assert B.luce_get_fault() == fault


# ----------------------------------------------------------------------------- rows
@pytest.mark.parametrize("dtype", [f32, bf16, f16])
@pytest.mark.parametrize("H", [32, 100, 2048, 4099, 20000, 65536])
def test_rows_of_zeros_without_an_epsilon(H, dtype):
    # codes and scale are zero; the row's neighbours are what they are anyway
    x = rows_input(5, H, dtype, H)
    x[1], x[3] = 0.0, -0.0
    gamma = torch.rand(H, generator=gen(5)) + 0.5
    check_rows(x, gamma, 0.0)
    check_rows(x, gamma, 0.0, -x, in_place="new")  # every sum is a zero
    check_rows(x, torch.zeros(H), 0.0)
    q, s = torch.empty((5, H), dtype=torch.int8, device="cuda"), torch.empty(5, device="cuda")
    B.luce_rmsnorm_i8(x.cuda(), gamma.cuda(), 0.0, q, s)
    assert torch.all(s[[1, 3, 4]] == 0) and not torch.any(q[[1, 3, 4]]) and torch.all(s[[0, 2]] > 0)


@pytest.mark.parametrize("in_place", ["x", "residual", "new", None])
@pytest.mark.parametrize("dtype", [f32, bf16])
@pytest.mark.parametrize("H", [32, 100, 2048, 4099, 20000, 65536])
def test_rows_whose_squares_fall_out_of_range(H, dtype, in_place):
    # values on both sides of where their squares leave the normal range (2^-63) and vanish
    # (2^-75), and down to the smallest numbers: the scale is the definition's whatever eps is
    es = [-20, -58, -60, -62, -64, -70, -74, -76, -90, -110, -120]
    x, r = (torch.ldexp(rows_input(len(es) + 2, H, f32, s), torch.tensor(es + [0, -100])[:, None]).to(dtype)
            for s in (H, H + 1))
    gamma = torch.rand(H, generator=gen(5)) + 0.5
    for eps in (0.0, 1e-42, 2.0 ** -121, 2.0 ** -119, 1e-30):
        check_rows(x, gamma, eps)
        check_rows(x, gamma, eps, r, in_place=in_place)
