"""The error of the gate that the header states, over all gates whose value is
not 0: 2^-20 + 2^-23 max(-g, 0) relative, which the scale shows (a block of one
value has the scale |value| / 448, rounded once: 2^-24)."""
import pytest
import torch

from expert_util import E4M3
from tile_centric_comm_gb300 import tdg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("up", [2.0 ** 40, -3.0 * 2.0 ** 60])
def test_the_gates_error(up):
    symm = tdg.Symm(1, 1024, 16)
    every = torch.arange(0x10000, device="cuda").to(torch.int16).view(torch.bfloat16)
    gate = every[(every.float().abs() >= 2.0 ** -40) & (every.float() >= -87) & (every.float() <= 2.0 ** 40)]   # (false for NaN)
    x = torch.empty(gate.numel(), 32, dtype=torch.bfloat16, device="cuda")
    x[:, :16], x[:, 16:] = gate[:, None], up
    codes, scale = torch.empty(gate.numel(), 16, dtype=E4M3, device="cuda"), torch.empty(gate.numel(), 1, device="cuda")
    tdg.quantise_rows(symm, x, codes, scale, gated=True)
    g = gate.double()
    want = (g * torch.sigmoid(g) * up).abs() / 448
    assert float(want.min()) > 2.0 ** -99
    off = ((scale[:, 0].double() - want).abs() / want) / (2.0 ** -20 + 2.0 ** -23 * (-g).clamp(min=0) + 2.0 ** -24)
    assert float(off.max()) <= 1, (float(off.max()), float(g[off.argmax()]))
    # the largest of a block is 448 or, where the scale was rounded down, clamped to it
    assert bool((codes.double().abs() == 448).all())
