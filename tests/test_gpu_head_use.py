"""GPU: the int8 decode head as programs use it -- weights made on the GPU,
launches that start early, streams and threads, the tile of every product --
against the definitions in 64 bits (oracle/head.py), with the helpers and
bounds of test_gpu_head.py.
"""
import ctypes
import importlib.machinery
import importlib.util
import math
import shutil
import subprocess
import threading
import time

import pytest
import torch

from oracle import head as O
from quantized_moe_decode_luce_gb300 import binding as B
from quantized_moe_decode_luce_gb300 import build as BLD
from quantized_moe_decode_luce_gb300.layer import GreedyHead, LinearI8
from test_gpu_head import (_lib, _no_device_faults, bf16, check_rows, codes, f16, f32, gen,  # noqa: F401
                           logits_case, make_head, rows_input, same)  # (the fixtures hold for every test here)

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


# ----------------------------------------------------------------------------- threads
WAITER = r"""
#include <unistd.h>
static volatile int flag;
void set_flag(void) { flag = 1; }
int wait_for_flag(void) /* two seconds at most */
{
    for (int i = 0; i < 2000 && !flag; i++)
        usleep(1000);
    return flag ? 0 : 3;
}
"""


def test_other_threads_run_while_a_call_waits(tmp_path):
    # a launch may have to wait (a full queue, a host function that needs Python): the call
    # module's function stands still here until another Python thread has run
    source, helper, copy = tmp_path / "w.c", tmp_path / "w.so", tmp_path / "luce_call.so"
    source.write_text(WAITER)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", str(source), "-o", str(helper)], check=True)
    w = ctypes.CDLL(str(helper))
    shutil.copy(BLD.call_path(), copy)  # (a module of its own, so that the real one keeps its functions)
    loader = importlib.machinery.ExtensionFileLoader("luce_call", str(copy))
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("luce_call", loader))
    loader.exec_module(module)
    module.bind(*[ctypes.cast(w.wait_for_flag, ctypes.c_void_p).value] * 5)
    x, g = torch.zeros((2, 64), device="cuda"), torch.zeros(64, device="cuda")
    q, s = torch.zeros((2, 64), dtype=torch.int8, device="cuda"), torch.zeros(2, device="cuda")
    other = threading.Thread(target=lambda: (time.sleep(0.05), w.set_flag()))
    other.start()
    assert module.quantize_i8(x, q, s) == 0
    other.join()
    for status in (module.rmsnorm_i8(x, g, 1e-6, q, s), module.add_rmsnorm_i8(x, x, None, g, 1e-6, q, s),
                   module.linear_i8(q, s, q, s, None, x[:, :2]), module.logits_process(x, x, *[None] * 10)):
        assert status == 0  # (the flag stands)


# ----------------------------------------------------------------------------- rows without a token
@pytest.mark.parametrize("V", [333, 3001, 20000])
def test_greedy_head_says_which_rows_have_no_token(V):
    R, H = 6, 256
    head, w, gamma = make_head(R, V, H)
    x = torch.randn((R, H), generator=gen(2))
    x[1, 3], x[2, 5], x[4, 7] = math.nan, -math.inf, math.inf
    mask = torch.randint(-2**31, 2**31, (2, (V + 31) // 32), generator=gen(3)).to(torch.int32)
    mask[0] = 0  # allows nothing
    mask[1, 0] = -2  # (not token 0)
    kw = dict(mask=mask.cuda(), mask_rows=torch.tensor([-1, -1, -1, 0, 1, 0], dtype=torch.int32, device="cuda"))
    idx, val = head.run(x.cuda(), **kw)
    clean = GreedyHead(1, gamma.cuda(), 1e-6, head.head)
    idx0, val0 = clean.run(x[:1].cuda())
    assert torch.equal(idx[:1], idx0) and torch.equal(val[:1], val0)  # (the neighbours do not reach it)
    idx, val, logits = idx.cpu().long(), val.cpu(), head.logits.cpu()
    assert torch.all((idx >= 0) & (idx < V))
    assert torch.isnan(val[1]) and torch.isnan(val[2])
    assert idx[3] == 0 and val[3] == -math.inf and idx[5] == 0 and val[5] == -math.inf
    assert torch.isnan(val[4]) or val[4] == -math.inf
    at = logits[torch.arange(R), idx]
    assert torch.all((at == val) | (torch.isnan(at) & torch.isnan(val)))
    assert torch.all(torch.isnan(logits[1:3])) and torch.all(torch.isnan(logits[4]) | (logits[4] == -math.inf))


def test_as_many_rows_as_there_may_be():
    # 2^31 - 1 rows of one value: the count of blocks, the row numbers and the offsets at their ends
    T = 2**31 - 1
    x = torch.ones((T, 1), dtype=bf16, device="cuda")
    x[-3:, 0] = torch.tensor([-2.0, 0.0, 3.0], dtype=bf16)
    q, scale = torch.full((T + 40,), 55, dtype=torch.int8, device="cuda"), torch.full((T + 40,), 55.0, device="cuda")
    B.luce_quantize_i8(x, q[:T].view(T, 1), scale[:T])
    torch.cuda.synchronize()
    assert q[T - 3:T].tolist() == [-127, 0, 127] and torch.all(q[T:] == 55) and torch.all(scale[T:] == 55)
    same(scale[T - 3:T], torch.tensor([2.0, 0.0, 3.0]) / 127)
    for r in range(0, T - 3, 2**28):
        end = min(r + 2**28, T - 3)
        assert torch.all(q[r:end] == 127) and torch.all(scale[r:end] == scale[0])
    assert scale[0] == torch.tensor(1.0) / 127
