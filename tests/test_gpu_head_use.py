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
from test_gpu_head import _lib, _no_device_faults, codes, f32, gen, same  # noqa: F401  (fixtures of every test here)

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
