"""How the int8 decode head is called and built, where no GPU is needed: host
checks of its entry points, the bindings and the call module."""
import ctypes
import os
import sys

import pytest
import torch

from oracle import head as O
from quantized_moe_decode_luce_gb300 import binding as Bd
from quantized_moe_decode_luce_gb300 import build as B
from quantized_moe_decode_luce_gb300.layer import GreedyHead, LinearI8

vp, ci, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(B.build())


def test_mask_rows_without_masks(lib):
    f = lib.luce_logits_process
    f.argtypes = [vp, ci, ci, i64, i64, vp, i64, vp, vp, vp, vp, vp, vp, vp, ci, vp, ci, i64, vp, vp, i64, vp]

    def call(mask, n_masks, mask_rows):  # (no rows: nothing is launched)
        return f(None, 0, 0, 64, 64, None, 0, None, None, None, None, None, None, None, 0, mask, n_masks, 2, mask_rows,
                 None, 64, None)
    assert call(None, 0, 0x10000) == 0 and call(None, 0, None) == 0
    assert call(None, 2, 0x10000) == 1  # masks that are not there
    assert call(0x20000, 0, 0x10000) == 1 and call(0x20000, 2, 0x10000) == 0


def test_linear_plan_refusals(lib):
    f, plan = lib.luce_linear_i8_plan, (ci * 8)(*[9] * 8)
    f.argtypes = [ci, ci, ci, ci, vp]
    for T, N, K, dtype in ((-1, 8, 16, 0), (1 << 24, 8, 16, 0), (1, 0, 16, 0), (1, 1 << 24, 16, 0), (1, 8, 24, 0),
                           (1, 8, 0, 0), (1, 8, 65552, 0), (1, 8, 16, 3)):
        assert f(T, N, K, dtype, plan) == 1
    assert f(1, 8, 16, 0, None) == 1 and list(plan) == [9] * 8
    assert f(0, 8, 16, 0, plan) == 0 and list(plan) == [0] * 8
    for T, tokens in ((1, 1), (2, 2), (3, 4), (4, 4), (5, 8), (8, 8)):  # (a choice that asks no device)
        assert f(T, 100, 4096, 1, plan) == 0 and list(plan) == [0, tokens, 8 if tokens == 8 else 4, 100, 0, 0, 0, 0]


# ----------------------------------------------------------------------------- definitions
def test_a_row_of_zeros_has_scale_zero_without_an_epsilon():
    x = torch.zeros((2, 8))
    x[1, 3] = 4.0
    q, s, _ = O.rows_i8(x, torch.ones(8), 0.0)
    assert s[0] == 0 and torch.all(q[0] == 0) and q[1, 3] == 127
    assert abs(float(s[1]) * 127 - 8 ** 0.5) < 1e-6  # 4 / sqrt(16 / 8)
    q, s, _ = O.rows_i8(x, torch.zeros(8), 0.0)
    assert torch.all(s == 0) and torch.all(q == 0)


# ----------------------------------------------------------------------------- the call module
@pytest.fixture
def unloaded(monkeypatch, lib):
    monkeypatch.setattr(Bd, "_LIB", None)
    monkeypatch.setattr(Bd, "_fast", None)


def test_the_library_loads_with_its_call_module(unloaded):
    assert Bd.lib().luce_version() > 0 and Bd._fast is not None


@pytest.mark.parametrize("what", ["missing", "not a module", "another library"])
def test_the_library_loads_without_the_call_module(what, unloaded, monkeypatch, tmp_path):
    path = tmp_path / "luce_call.so"
    if what == "not a module":
        path.write_bytes(b"no shared object")
    monkeypatch.setattr(Bd, "call_path", lambda: B.LIB if what == "another library" else str(path))
    with pytest.warns(RuntimeWarning, match="call module"):
        L = Bd.lib()
    assert Bd._fast is None and L.luce_version() > 0 and Bd.status_string(1) == "invalid argument"
    x = torch.zeros((2, 64))
    with pytest.raises(TypeError):  # the bindings are there, and look at their arguments themselves
        Bd.luce_quantize_i8(x, x, x)
    with pytest.raises(TypeError):
        Bd.luce_logits_process(x, x)


def test_the_call_module_is_named_after_what_it_is_tied_to(monkeypatch):
    here = B.call_path()
    assert sys.implementation.cache_tag in here and os.path.dirname(here) == B.LIBDIR and os.path.exists(here)
    monkeypatch.setattr(torch, "__version__", "9.9.9+cu000")
    assert B.call_path() not in (here,) and not os.path.exists(B.call_path())


@pytest.mark.parametrize("what", ["compiler", "torch"])
def test_the_build_does_without_the_call_module(what, lib, monkeypatch, tmp_path):
    path = tmp_path / "luce_call.so"
    path.write_bytes(b"an older one")
    os.utime(path, (1, 1))

    def none(*a):
        raise ImportError("no torch")
    monkeypatch.setattr(B, "call_path", none if what == "torch" else lambda: str(path))
    monkeypatch.setattr(B, "call_command", lambda s, t: ["false"])
    with pytest.warns(RuntimeWarning, match="call module"):
        assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and path.exists() == (what == "torch")  # an older source's does not stay


def test_the_build_makes_the_call_module(lib, monkeypatch, tmp_path):
    path = tmp_path / "luce_call.so"
    monkeypatch.setattr(B, "call_path", lambda: str(path))
    monkeypatch.setattr(B, "call_command", lambda s, t: ["cp", s, t])
    B.build()
    assert path.exists() and os.listdir(tmp_path) == ["luce_call.so"]


# ----------------------------------------------------------------------------- GreedyHead
@pytest.fixture
def calls(monkeypatch, lib):
    """The library calls that a head makes, each with the device that is current, without a GPU."""
    made, current = [], [0]

    class Device:
        def __init__(self, i):
            self.i = i

        def __enter__(self):
            self.i, current[0] = current[0], self.i

        def __exit__(self, *a):
            current[0] = self.i

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    for name in ("luce_rmsnorm_i8", "luce_add_rmsnorm_i8", "luce_linear_i8", "luce_logits_process", "luce_argmax"):
        monkeypatch.setattr(Bd, name, lambda *a, name=name, **kw: made.append((name, current[0])))
    return made


def greedy_head():
    w = LinearI8(torch.zeros((100, 32), dtype=torch.int8), torch.zeros(100))
    return GreedyHead(2, torch.ones(32), 1e-6, w)


def test_a_head_runs_on_its_own_device(calls):
    head, x = greedy_head(), torch.zeros((2, 32))
    here = head.q.get_device()
    assert here != torch.cuda.current_device()
    head.run(x, x, hist=None)
    head.run(x)
    assert calls == [(n, here) for n in ("luce_add_rmsnorm_i8", "luce_linear_i8", "luce_logits_process", "luce_argmax",
                                         "luce_rmsnorm_i8", "luce_linear_i8", "luce_argmax")]
    assert torch.cuda.current_device() == 0


def test_a_head_without_a_residual_has_no_sum_to_store(calls):
    head, x = greedy_head(), torch.zeros((2, 32))
    with pytest.raises(ValueError):
        head.run(x, None, torch.zeros((2, 32)))
    assert calls == []  # nothing was launched
