"""The gradient of the combine with dy in the place of y, for every number of
threads that a token gets: y is read before it is written over."""
import pytest
import torch

from test_gpu_moe_grad import Case

pytestmark = pytest.mark.gpu


# 32 threads, 64, 128 and 256; one choice, a whole group of eight, more than a group
@pytest.mark.parametrize("k", [1, 8, 11])
@pytest.mark.parametrize("W,T,H", [(1, 2500, 264), (1, 2601, 1032), (1, 1301, 2056), (2, 5, 2056), (1, 3, 7168)])
def test_dy_in_the_place_of_y(W, T, H, k):
    c = Case(W, T, H, 16, k, seed=k)
    y = c.y.clone()
    c.run()
    c.check()
    dgate = c.all(c.dgate)
    for r in range(W):
        c.dgate(r).fill_(-77.0)
    c.run(dy=c.y)
    assert c.symm.status()["code"] == 0
    assert torch.equal(c.y, c.dy) and torch.equal(c.all(c.dgate), dgate)
    c.check(y=y)
