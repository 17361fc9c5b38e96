"""LinearW4 looks at its activations before it calls the library (no GPU needed: nothing is launched)."""
import pytest
import torch

from quantized_moe_decode_luce_gb300 import binding as B
from quantized_moe_decode_luce_gb300.layer import LinearW4


# (rows of 112 codes pack into as many bytes and groups as rows of 128)
@pytest.mark.parametrize("K", [1, 64, 112, 144, 256])
def test_activations_of_another_width_are_refused(K, monkeypatch):
    calls = []
    monkeypatch.setattr(B, "luce_linear_w4", lambda *a: calls.append(a))
    w = LinearW4(torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 1)), 128, 128)
    with pytest.raises(ValueError, match="takes 128 values"):
        w.run(torch.zeros((2, K)), None, torch.zeros((2, 4)))
    assert not calls
    out = torch.zeros((2, 4))
    assert w.run(torch.zeros((2, 128)), None, out) is out and len(calls) == 1
