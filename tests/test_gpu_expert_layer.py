"""The 8-bit expert layer as a program runs it: every call of the example's
path against the definition in 64 bits, given what the call before it left."""
import importlib.util
import os

import pytest
import torch

from expert_util import check_product, product, quantised
from tile_centric_comm_gb300 import tdg

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens", [1, 37, 300])
def test_every_call_of_a_step(example, tokens):
    layer = example.Layer(tokens, seed=tokens)
    W, H, I, E, k = example.W, example.HIDDEN, example.INNER, example.EXPERTS, example.TOP
    x = torch.randn(W, tokens, H, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").to(torch.bfloat16)
    for w, codes, scale in ((layer.w_in, layer.in8, layer.in_s), (layer.w_out, layer.out8, layer.out_s)):
        for e in (0, E - 1):
            want, s = quantised(w[e], rows=128)
            assert torch.equal(codes[e].view(torch.uint8), want) and torch.equal(scale[e], s)
    out = layer.forward(x)
    assert layer.heap.status()["code"] == 0
    gate = layer.all(layer.gate_off, (tokens, k), torch.float32)
    top = layer.all(layer.topk_off, (tokens, k), torch.int32)
    slot, base = layer.slot.view(W, tokens, k), layer.base.tolist()
    # rows by expert, a token's in each of its experts' ranges
    assert base[0] == 0 and base[-1] == layer.rows
    assert torch.equal(slot.flatten().sort().values, torch.arange(layer.rows, device="cuda"))
    assert bool(((slot >= layer.base[top.long()]) & (slot < layer.base[top.long() + 1])).all())
    codes, s = quantised(x.view(-1, H))
    tok = torch.empty(layer.rows, dtype=torch.int64, device="cuda")
    tok[layer.slot] = torch.arange(layer.rows, device="cuda") // k
    assert torch.equal(layer.x8.view(torch.uint8), codes[tok]) and torch.equal(layer.xs, s[tok])
    for e in range(E):
        lo, hi = base[e], base[e + 1]
        if hi > lo:
            want, mag = product(layer.x8[lo:hi], layer.xs[lo:hi], layer.in8[e], layer.in_s[e])
            check_product(layer.h[lo:hi], want, mag, H, f"first product, expert {e}")
            want, mag = product(layer.h8[lo:hi], layer.hs[lo:hi], layer.out8[e], layer.out_s[e])
            check_product(layer.y[lo:hi], want, mag, I, f"second product, expert {e}")
    g, u = layer.h.double().chunk(2, 1)
    v = g * torch.sigmoid(g) * u
    scale = layer.hs.double().repeat_interleave(128, 1)[:, :I]
    # half a step of the codes, and the gate's 2^-20 + 2^-23 |g| with |g| < 16 on value and scale
    q = v / scale
    assert bool(((layer.h8.double() - q).abs() <= torch.maximum(2.0 ** -4 * q.abs(), torch.full_like(q, 2.0 ** -10)) + 2.0 ** -17 * q.abs()).all())
    parts = gate[..., None].double() * layer.y[slot].double()
    tol = 2.0 ** -8 * parts.sum(2).abs() + 2.0 ** -23 * k * parts.abs().sum(2) + 1e-30
    assert bool(((out.double() - parts.sum(2)).abs() <= tol).all())


def test_the_layer_in_a_graph(example):
    """A whole step captured once and replayed on other tokens and routes."""
    layer = example.Layer(21)
    W, H = example.W, example.HIDDEN
    g = torch.Generator(device="cuda").manual_seed(3)

    def tokens():
        return torch.randn(W, 21, H, generator=g, device="cuda").to(torch.bfloat16)
    x = tokens()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        layer.forward(x)
        with torch.cuda.graph(graph, stream=side):
            out = layer.forward(x)
    torch.cuda.synchronize()
    for _ in range(3):
        x.copy_(tokens())
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, layer.forward(x))
    assert layer.heap.status()["code"] == 0


def test_the_example_runs(example):
    off, dx, dgate = example.run(tokens=40)
    assert all(v == v for v in (off, dx, dgate))
    # two chains of bf16 roundings (y, dy, drecv, the gradient itself): a few half steps of 2^-8
    assert dx <= 4 * 2.0 ** -8 and dgate <= 4 * 2.0 ** -8
