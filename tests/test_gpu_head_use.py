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
from test_gpu_head import (SCALE_TOL, _lib, _no_device_faults, bf16, check_rows, codes, f16, f32,  # noqa: F401
                           gen, logits_case, make_head, rows_input, same)  # (the fixtures hold for every test here)

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


# ----------------------------------------------------------------------------- the product's tiles
# Products by the kernels that they take, in one launch or two.  The choice is an estimate of time; each test below asks for it, so that none runs another kernel unseen.
TILES = [  # T, N, K, [(kernel, tokens of a tile, K split)]
    (10, 9788, 1056, [(1, 16, False)]), (10, 7521, 528, [(1, 16, True)]), (9, 8589, 16, [(1, 16, False)]),
    (1246, 131, 1040, [(1, 32, False)]), (18, 1418, 2704, [(1, 32, True)]), (17, 9732, 16, [(1, 32, False)]),
    (33, 10219, 1088, [(1, 48, False)]), (35, 1422, 2704, [(1, 48, True)]),
    (49, 10871, 1056, [(1, 64, False)]), (356, 129, 3904, [(1, 64, True)]), (49, 30303, 16, [(1, 64, False)]),
    (52, 9857, 3632, [(2, 64, False)]), (49, 6965, 5280, [(2, 64, True)]),
    (66, 9982, 1184, [(2, 96, False)]), (67, 3311, 2896, [(2, 96, True)]), (261, 23338, 16, [(2, 96, False)]),
    (98, 10483, 1152, [(2, 128, False)]), (98, 4909, 2224, [(2, 128, True)]), (202, 24999, 16, [(2, 128, False)]),
    (139, 14096, 2080, [(4, 160, False)]), (147, 5091, 3264, [(4, 160, True)]), (4879, 258, 3200, [(4, 160, False)]),
    (161, 13370, 2960, [(4, 192, False)]), (168, 5041, 3808, [(4, 192, True)]),
    (195, 12849, 2768, [(4, 224, False)]), (207, 4731, 4496, [(4, 224, True)]), (223, 7087, 15776, [(4, 224, True)]),
    (229, 13044, 3456, [(4, 256, False)]), (1242, 781, 5328, [(4, 256, True)]), (1968, 53319, 1040, [(4, 256, False)]),
    (9, 20278, 1632, [(1, 16, False), (0, 8, True)]), (10, 21035, 4656, [(1, 16, False), (1, 16, True)]),
    (51, 25907, 7584, [(1, 64, False), (2, 64, True)]), (69, 19595, 2272, [(2, 96, False), (0, 8, True)]),
    (189, 9915, 3008, [(2, 96, False), (1, 32, True)]), (65, 22772, 5056, [(2, 96, False), (2, 96, True)]),
    (149, 12937, 13296, [(2, 96, False), (4, 160, True)]), (139, 19469, 4944, [(4, 160, False), (0, 8, True)]),
    (173, 19772, 5104, [(4, 192, False), (1, 48, True)]), (130, 21998, 5184, [(4, 160, False), (2, 96, True)]),
    (134, 24353, 9024, [(4, 160, False), (4, 160, True)])]
SPLIT = {1: [t for t in TILES if t[3] == [(1, 64, True)]], 2: [t for t in TILES if t[3] == [(2, 96, True)]],
         4: [t for t in TILES if t[3] == [(4, 160, True)]]}


def assert_plan(T, N, K, dtype, want):
    plan = B.luce_linear_i8_plan(T, N, K, dtype)
    assert [(kernel, tokens, groups > 1) for kernel, tokens, groups, _ in plan] == want, (
        f"{T} x {N} x {K} takes {plan} now: another product is needed for {want}")
    assert sum(channels for *_, channels in plan) == N


def definition(xq, xs, wq, ws, b, dtype):
    """oracle/head.py's product on tensors of the GPU (64 bits there too), a slice of the channels at a time."""
    N, K = wq.shape
    out = torch.empty((xq.shape[0], N), dtype=dtype, device="cuda")
    step = max(1, min((1 << 28) // K, (1 << 25) // xq.shape[0]))
    for n in range(0, N, step):
        e = min(n + step, N)
        out[:, n:e] = O.linear_i8(xq, xs, wq[n:e], ws[n:e], None if b is None else b[n:e], dtype)
    return out


def product(T, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    xq, wq = (torch.randint(-128, 128, (r, K), generator=g, dtype=torch.int8, device="cuda") for r in (T, N))
    xs, ws = (torch.rand(r, generator=g, device="cuda") * 0.01 for r in (T, N))
    return xq, xs, wq, ws, torch.randn(N, generator=g, device="cuda")


def run_product(xq, xs, wq, ws, b, dtype, gap=0):
    T, N = xq.shape[0], wq.shape[0]
    wide = torch.full((T + 1, N + gap), 77.0, dtype=dtype, device="cuda")
    B.luce_linear_i8(xq, xs, wq, ws, b, wide[:T, :N])
    assert torch.all(wide[:, N:] == 77.0) and torch.all(wide[T:] == 77.0)
    return wide[:T, :N]


def equal(out, ref):
    bad = out != ref
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} differ, first at {tuple(bad.nonzero()[0].tolist())}"


def test_the_tiles_above_are_all_there_are():
    one = {p[0] for *_, p in TILES if len(p) == 1}
    widths = {1: (16, 32, 48, 64), 2: (64, 96, 128), 4: (160, 192, 224, 256)}
    assert one == {(k, w, split) for k in widths for w in widths[k] for split in (False, True)}
    first = {(p[0][0], p[1][0]) for *_, p in TILES if len(p) == 2}
    assert {a for a, _ in first} == {1, 2, 4} and {b for _, b in first} == {0, 1, 2, 4}


@pytest.mark.parametrize("T,N,K,plan", TILES)
def test_linear_every_kernel_and_tile(T, N, K, plan):
    dtype = [f32, bf16, f16][(T + N) % 3]
    assert_plan(T, N, K, dtype, plan)
    xq, xs, wq, ws, b = product(T, N, K, T + N)
    b = b if N % 2 else None
    equal(run_product(xq, xs, wq, ws, b, dtype, gap=T % 5), definition(xq, xs, wq, ws, b, dtype))


# unsplit, with chunks of 1024 values that are full, a little short and a little over
FULL = [(9, 9933, 1008, 1), (9, 9757, 1024, 1), (49, 10871, 1056, 1), (9, 9792, 2048, 1), (65, 9864, 1008, 2),
        (4968, 129, 1024, 2), (66, 9884, 1040, 2), (4961, 130, 2048, 2), (1968, 53319, 1040, 4), (131, 29948, 2048, 4),
        (130, 13109, 2064, 4), (4907, 266, 4096, 4)]


@pytest.mark.parametrize("T,N,K,kernel", FULL + [(*t[:3], k) for k in SPLIT for t in SPLIT[k]])
def test_linear_the_largest_sums_on_every_kernel(T, N, K, kernel):
    # chunks that add up to 2^24 (-128 x -128), and the largest sums of low bits
    p = B.luce_linear_i8_plan(T, N, K)
    assert len(p) == 1 and p[0][0] == kernel and (p[0][2] > 1) == ((T, N, K, kernel) not in FULL)
    xs, ws = torch.rand(T, device="cuda") * 0.01, torch.rand(N, device="cuda") * 0.01
    full = lambda r, v: torch.full((r, K), v, dtype=torch.int8, device="cuda")  # noqa: E731
    for x, w in ((-128, -128), (127, 127), (-128, 127)):
        out = run_product(full(T, x), xs, full(N, w), ws, None, f32)
        isum = torch.tensor(float(x * w * K), device="cuda")  # (below 2^31; rounded once)
        equal(out, isum * (xs[:, None] * ws[None, :]))
    x, w = full(T, 127), full(N, -128)
    x[:, ::2], w[:, 1::3] = -127, 125
    equal(run_product(x, xs, w, ws, None, f32), definition(x, xs, w, ws, None, f32))


CHAIN = [(49, 10871, 1056, [(1, 64, False)]), (66, 9982, 1184, [(2, 96, False)]), (139, 14096, 2080, [(4, 160, False)]),
         (35, 1422, 2704, [(1, 48, True)]), (98, 4909, 2224, [(2, 128, True)]), (147, 5091, 3264, [(4, 160, True)]),
         (10, 21035, 4656, [(1, 16, False), (1, 16, True)]), (130, 21998, 5184, [(4, 160, False), (2, 96, True)])]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("T,N,K,plan", CHAIN)
def test_chains_of_launches_that_start_early(T, N, K, plan, captured, pdl):
    # each reads what the one before wrote, and every buffer is written again in the next turn
    assert_plan(T, N, K, f32, plan)
    xs_in = [torch.randn((T, K), generator=gen(s)) for s in (1, 2)]
    wf = [torch.randn((N, K), generator=gen(s)).cuda() for s in (3, 4)]
    xd = [x.cuda() for x in xs_in]
    c = logits_case(T, N, hist=20)
    kw = {k: v.cuda() for k, v in c.items() if k != "logits"}
    q, s = torch.empty((T, K), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    wq, ws = torch.empty((N, K), dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    out, ls = torch.empty((T, N), device="cuda"), torch.zeros((4, T, N), device="cuda")
    torch.cuda.synchronize()

    def turns():
        for i in range(4):
            B.luce_quantize_i8(xd[i % 2], q, s)
            B.luce_quantize_i8(wf[i // 2], wq, ws)
            B.luce_linear_i8(q, s, wq, ws, None, out)
            B.luce_logits_process(out, ls[i], **kw)

    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            turns()
        for _ in range(3):
            g.replay()
    else:
        turns()
    torch.cuda.synchronize()
    for i in range(4):
        qr, sr, _ = O.rows_i8(xd[i % 2])
        wr, wsr, _ = O.rows_i8(wf[i // 2])
        ref = definition(qr, sr.to(f32), wr, wsr.to(f32), None, f32)
        if i == 3:
            equal(out, ref)
        same(ls[i], O.logits_process(ref.cpu(), **{k: v for k, v in c.items() if k != "logits"}))


def test_split_products_on_two_streams_at_once():
    # clusters that split K and wide ones, of two streams between one another
    cases = [(T, N, K) for k in SPLIT for T, N, K, _ in SPLIT[k]] + [(139, 14096, 2080), (130, 21998, 5184)]
    data = [product(*c, seed=i) for i, c in enumerate(cases)]
    refs = [definition(*d, f32) for d in data]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(r) for r in refs] for _ in streams]
    torch.cuda.synchronize()
    for turn in range(5):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                for i in range(len(cases)):
                    j = (i + k * 2 + turn) % len(cases)
                    B.luce_linear_i8(*data[j], outs[k][j])
    torch.cuda.synchronize()
    for o in outs:
        for a, r in zip(o, refs):
            equal(a, r)


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


@pytest.mark.parametrize("dtype", [bf16, f16])
@pytest.mark.parametrize("T,H", [(1024, 5120), (700, 10240), (310, 15360), (300, 20480), (100, 40960), (1000, 4099), (750, 6319),
                                 (300, 9211), (500, 9211), (160, 20481)])
def test_long_rows_of_sixteen_bits(T, H, dtype):
    # four and five chunks to a thread, on both sides of where a round of blocks ends
    x, gamma = rows_input(T, H, dtype, T + H), torch.randn(H, generator=gen(H))
    check_rows(x)
    check_rows(x, gamma, 1e-6)


# ----------------------------------------------------------------------------- the largest sizes
@pytest.mark.parametrize("T,H,shift", [(70001, 32768, 0), (70001, 32768, 1), (525000, 4099, 0), (36000, 65536, 0)])
def test_rows_beyond_2_31_elements(T, H, shift):
    # the last rows are those of a small call; the first are not written by them
    n = 5
    x = torch.zeros(T * H + shift, dtype=bf16, device="cuda")[shift:].view(T, H)
    ends = rows_input(2 * n, H, bf16, 3)
    ends[n - 1] = ends[0]
    x[:n], x[-n:] = ends[:n].cuda(), ends[n:].cuda()
    gamma = torch.rand(H, generator=gen(5)) + 0.5
    q, s = torch.full((T, H), 7, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    for norm in (False, True):
        if norm:
            B.luce_add_rmsnorm_i8(x, x, x, gamma.cuda(), 1e-6, q, s)  # (twice the rows, where they were)
            q_ref, s_ref, sum_ref = O.rows_i8(ends, gamma, 1e-6, ends)
            same(torch.cat([x[:n], x[-n:]]), sum_ref)
        else:
            B.luce_quantize_i8(x, q, s)
            q_ref, s_ref, _ = O.rows_i8(ends)
        same(torch.cat([q[:n], q[-n:]]), q_ref)
        got = torch.cat([s[:n], s[-n:]]).cpu().double()
        assert torch.all((got - s_ref).abs() <= SCALE_TOL * s_ref)
        assert not torch.any(s[n:-n]) and not torch.any(q[T // 2 - 9:T // 2 + 9])


@pytest.mark.parametrize("T,N,K", [(3, 16777215, 16), (300, 9000001, 16), (40001, 60001, 32), (300001, 9001, 16)])
def test_linear_outputs_of_the_largest_sizes(T, N, K):
    xq, xs, wq, ws, b = product(T, N, K, T)
    out = torch.empty((T, N), dtype=bf16, device="cuda")
    B.luce_linear_i8(xq, xs, wq, ws, b, out)
    for t in (slice(0, 3), slice(T // 2, T // 2 + 3), slice(T - 3, T)):
        equal(out[t], definition(xq[t].contiguous(), xs[t], wq, ws, b, bf16))


def test_logits_of_the_largest_vocabulary():
    V, L = 2**31 - 1, 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((1, V), dtype=bf16, device="cuda")
    x.normal_(generator=g)
    hist = torch.randint(0, V, (1, L), generator=g, dtype=torch.int64, device="cuda").to(torch.int32)
    hist[0, :6] = torch.tensor([V - 1, 0, V - 2, V - 1, -1, V - 33])
    bias_ids = torch.tensor([[V - 1, 5, V - 4, -1]], dtype=torch.int32, device="cuda")
    bias_vals = torch.tensor([[3.0, -2.0, 9.0, 1.0]], device="cuda")
    mask = torch.randint(-2**31, 2**31, (1, (V + 31) // 32), generator=g, dtype=torch.int64, device="cuda").to(torch.int32)
    row = lambda v, t=f32: torch.tensor([v], dtype=t, device="cuda")  # noqa: E731
    kw = dict(hist=hist, hist_len=row(L, torch.int32), prompt_len=row(2, torch.int32), repetition=row(1.3), frequency=row(0.25),
              presence=row(0.5), bias_ids=bias_ids, bias_vals=bias_vals)
    out = torch.empty((1, V), device="cuda")
    B.luce_logits_process(x, out, **kw, mask=mask)
    # the tokens that anything happens to, renumbered, by the definition; the rest are the logits or masked
    at = torch.unique(torch.cat([hist[0], bias_ids[0]]).long().clamp_(min=0))
    where = {int(t): i for i, t in enumerate(at.tolist())}
    small = {k: v.cpu() for k, v in kw.items()}
    for k in ("hist", "bias_ids"):
        small[k] = torch.tensor([[where[t] if t >= 0 else -1 for t in small[k][0].tolist()]], dtype=torch.int32)
    ref = O.logits_process(x[:, at].cpu(), **small)
    bit = lambda t: (mask[0, t // 32].long() >> (t % 32)) & 1  # noqa: E731
    ref[:, bit(at).cpu() == 0] = -math.inf
    same(out[:, at], ref)
    out[0, at] = 0.0
    step = 2**27
    for v in range(0, V, step):
        t = torch.arange(v, min(v + step, V), device="cuda")
        want = torch.where(bit(t) == 1, x[0, t[0]:t[-1] + 1].to(f32), -math.inf)
        want[at[(at >= t[0]) & (at <= t[-1])] - v] = 0.0
        assert torch.equal(out[0, t[0]:t[-1] + 1], want)


def test_logits_of_as_many_rows_as_there_may_be():
    R, V = 65535, 40
    c = logits_case(7, V, hist=9, bias=3, mask=True)
    n = R // 7 + 1
    many = {k: (v if k == "mask" else v.repeat((n,) + (1,) * (v.dim() - 1))[:R]).cuda() for k, v in c.items()}
    out = torch.empty((R, V), device="cuda")
    B.luce_logits_process(many.pop("logits"), out, **many)
    same(out, O.logits_process(**c).repeat((n, 1))[:R])
    with pytest.raises(B.LuceError):
        B.luce_logits_process(torch.zeros((R + 1, 2), device="cuda"), torch.zeros((R + 1, 2), device="cuda"))


@pytest.mark.parametrize("hist", [30, 40000])
def test_logits_ids_of_the_lowest_value_are_padding(hist):
    c = logits_case(2, 200000, hist=hist, bias=6, mask=True)
    c["hist"][:, 5:9] = torch.tensor([-2**31, -2**31 + 1, -200000, -2**30], dtype=torch.int32)
    c["bias_ids"][:, 3] = -2**31
    want = O.logits_process(**c)
    out = torch.empty((2, 200000), device="cuda")
    B.luce_logits_process(out=out, **{k: v.cuda() for k, v in c.items()})
    same(out, want)
