"""Gradients of the MoE dispatch and combine against their formulas in 64 bits,
against differences of the combine itself, and against autograd."""
import ctypes

import pytest
import torch

from expert_util import generator
from gpu_util import align
from tile_centric_comm_gb300 import tdg

pytestmark = pytest.mark.gpu
MARK = -77.0


class Case:
    """One routing, gates and gradients of the output in a heap; y and drecv in the receive layout."""

    def __init__(self, W, T, H, E, k, seed=0, scale=1.0):
        g = generator(seed + T)
        self.W, self.T, self.H, self.E, self.k = W, T, H, E, k
        self.gate_off = 4                        # off every grid but float32's
        self.dgate_off = align(self.gate_off + T * k * 4, 16) + 8
        self.dout_off = align(self.dgate_off + T * k * 4, 16)
        self.dx_off = self.dout_off + align(T * H * 2, 16)
        self.symm = tdg.Symm(W, self.dx_off + align(T * H * 2, 16) + 16, 16)
        self.rows = W * T * k
        topk = torch.rand(W, T, E, generator=g, device="cuda").topk(k, -1).indices
        self.slot = torch.empty(self.rows, dtype=torch.int64, device="cuda")
        self.slot[torch.sort(topk.flatten(), stable=True).indices] = torch.arange(self.rows, device="cuda")
        bf = torch.bfloat16
        for r in range(W):
            self.gate(r).copy_(torch.randn(T, k, generator=g, device="cuda").softmax(-1))
            self.dout(r).copy_((torch.randn(T, H, generator=g, device="cuda") * scale).to(bf))
            self.dx(r).fill_(MARK)
            self.dgate(r).fill_(MARK)
        self.y = torch.randn(self.rows, H, generator=g, device="cuda").to(bf)
        self.drecv = torch.randn(self.rows, H, generator=g, device="cuda").to(bf)
        self.dy = torch.full((self.rows, H), MARK, dtype=bf, device="cuda")

    def gate(self, r):
        return self.symm.view(r, self.gate_off, (self.T, self.k), torch.float32)

    def dgate(self, r):
        return self.symm.view(r, self.dgate_off, (self.T, self.k), torch.float32)

    def dout(self, r):
        return self.symm.view(r, self.dout_off, (self.T, self.H), torch.bfloat16)

    def dx(self, r):
        return self.symm.view(r, self.dx_off, (self.T, self.H), torch.bfloat16)

    def all(self, view):
        return torch.stack([view(r) for r in range(self.W)])

    def run(self, dy=None):
        tdg.moe_combine_grad(self.symm, self.T, self.H, self.k, self.gate_off, self.dout_off, self.dgate_off, self.slot, self.y,
                             self.dy if dy is None else dy)
        tdg.moe_dispatch_grad(self.symm, self.T, self.H, self.k, self.dx_off, self.slot, self.drecv)

    def check(self, y=None, refused=()):
        y = self.y if y is None else y
        T, H, k, W = self.T, self.H, self.k, self.W
        at = self.slot.view(W, T, k)
        ok = torch.ones(self.rows, dtype=torch.bool, device="cuda")
        ok[list(refused)] = False
        ok = ok.view(W, T, k)
        at = torch.where(ok, at, torch.zeros_like(at))
        dout, gate = self.all(self.dout).double(), self.all(self.gate).double()
        # dy: the float32 product of a float32 and a bf16 value, rounded to bf16
        want = (gate[..., None] * dout[:, :, None]).float().to(torch.bfloat16)
        assert torch.equal(self.dy[at[ok]], want[ok])
        # dgate: H float32 products and sums
        parts = y[at].double() * dout[:, :, None]
        tol = 2.0 ** -23 * (H + 8) * parts.abs().sum(-1) + 1e-40
        got = self.all(self.dgate).double()
        assert bool(((got - parts.sum(-1)).abs() <= tol)[ok].all()) and bool((got[~ok] == 0).all())
        # dx: at most k float32 additions, one rounding to bf16 (half a step: 2^-8)
        parts = self.drecv[at].double() * ok[..., None]
        sums = parts.sum(2)
        tol = 2.0 ** -8 * sums.abs() + 2.0 ** -23 * k * parts.abs().sum(2) + 1e-40
        assert bool(((self.all(self.dx).double() - sums).abs() <= tol).all())


# a token's threads: 32, 64 and 128 for many tokens, more for few
@pytest.mark.parametrize("W,T,H,E,k", [(1, 4999, 64, 8, 2), (2, 2501, 264, 8, 3), (1, 2601, 1032, 16, 2), (1, 1301, 2056, 8, 2), (3, 5, 512, 8, 8),
                                       (1, 1001, 1024, 40, 32), (8, 700, 8, 16, 9)])
def test_gradients_by_every_number_of_threads(W, T, H, E, k):
    c = Case(W, T, H, E, k)
    c.run()
    assert c.symm.status()["code"] == 0
    c.check()


@pytest.mark.parametrize("W,T,H,E,k", [(1, 1, 8, 1, 1), (1, 3, 16, 4, 2), (2, 257, 520, 8, 2), (8, 16, 7168, 64, 8), (4, 33, 2048, 16, 3), (3, 50, 2056, 48, 9),
                                       (2, 20, 264, 32, 32), (2, 700, 128, 64, 6)])
def test_gradients(W, T, H, E, k):
    c = Case(W, T, H, E, k)
    c.run()
    assert c.symm.status()["code"] == 0
    c.check()


def test_dy_in_the_place_of_y():
    c = Case(2, 65, 1032, 16, 4, seed=3)
    y = c.y.clone()
    c.run(dy=c.y)
    c.dy = c.y
    c.check(y=y)


def test_refused_choices_take_no_part():
    c = Case(2, 30, 264, 8, 3, seed=4)
    good = c.slot.clone()
    for bad, where in ((-1, None), (180, "slot"), (-3, "slot"), (2 ** 40, "slot"), (-2 ** 63, "slot")):
        c.slot.copy_(good)
        c.slot[100] = bad
        c.dy.fill_(MARK)
        c.run()
        st = c.symm.status()
        assert (st["code"], st["where"]) == ((0, 0) if where is None else (tdg.TDG_ERR_DEVICE, where))
        assert where is None or st["index"] == 100
        c.check(refused=[100])
        assert bool((c.dy[good[100]] == MARK).all())


def test_differences_of_the_combine():
    """out is linear in gates and rows: with small integers every sum is exact in bf16, and a difference of the
    combine's own outputs is the gradient."""
    W, T, H, E, k = 2, 25, 64, 8, 2
    c = Case(W, T, H, E, k, seed=5)
    g = generator(9)
    c.y.copy_(torch.randint(-4, 5, c.y.shape, generator=g, device="cuda"))
    for r in range(W):
        c.gate(r).copy_(torch.randint(1, 4, (T, k), generator=g, device="cuda"))
        c.dout(r).copy_(torch.randint(-2, 3, (T, H), generator=g, device="cuda"))
    heap = tdg.Symm(W, align(T * H * 2) * 2 + 2048, 16)
    topk_off, gate_off, out_off = align(T * H * 2), align(T * H * 2) + 512, align(T * H * 2) + 1024
    zeros = torch.empty(W * E, dtype=torch.int64, device="cuda"), torch.empty(E + 1, dtype=torch.int64, device="cuda")

    def loss(gates, y):
        for r in range(W):
            heap.view(r, gate_off, (T, k), torch.float32).copy_(gates[r])
        tdg.moe_dispatch_combine(heap, T, H, E, k, 0, topk_off, gate_off, out_off, y, *zeros, c.slot, torch.empty(8, dtype=torch.uint8, device="cuda"),
                                 y=y, phases=tdg.MOE_COMBINE)
        out = torch.stack([heap.view(r, out_off, (T, H), torch.bfloat16) for r in range(W)])
        return float((out.double() * c.all(c.dout).double()).sum())
    c.run()
    gates, dgate = c.all(c.gate), c.all(c.dgate)
    start = loss(gates, c.y)
    for r, t, kk in ((0, 0, 0), (1, 24, 1), (0, 11, 1), (1, 7, 0)):
        moved = gates.clone()
        moved[r, t, kk] += 1
        assert loss(moved, c.y) - start == float(dgate[r, t, kk])
        row = int(c.slot.view(W, T, k)[r, t, kk])
        for h in (0, 33, 63):
            y = c.y.clone()
            y[row, h] += 1
            assert loss(gates, y) - start == float(c.dy[row, h])


def test_a_layer_against_autograd():
    """Dispatch, a plain expert for every row, combine: gradients of the tokens and gates against autograd in 64 bits."""
    W, T, H, E, k = 2, 40, 128, 8, 3
    c = Case(W, T, H, E, k, seed=6)
    g = generator(12)
    x = torch.randn(W * T, H, generator=g, device="cuda").to(torch.bfloat16)
    weight = torch.randn(H, H, generator=g, device="cuda").double() / H ** 0.5
    tok = torch.empty(c.rows, dtype=torch.int64, device="cuda")
    tok[c.slot] = torch.arange(c.rows, device="cuda") // k
    c.y.copy_(torch.tanh(x[tok].double() @ weight).to(torch.bfloat16))
    tdg.moe_combine_grad(c.symm, T, H, k, c.gate_off, c.dout_off, c.dgate_off, c.slot, c.y, c.dy)
    c.drecv.copy_(((1 - c.y.double() ** 2) * c.dy.double()) @ weight.T)
    tdg.moe_dispatch_grad(c.symm, T, H, k, c.dx_off, c.slot, c.drecv)
    xd = x.double().requires_grad_()
    gd = c.all(c.gate).double().view(W * T, k).requires_grad_()
    y = torch.tanh(xd[tok] @ weight)
    out = (gd[..., None] * y[c.slot.view(W * T, k)]).sum(1)
    out.backward(c.all(c.dout).double().view(W * T, H))
    # y, dy and drecv are bf16 (2^-8 each) on the way: a part of a gradient is off by a few of these, and its sum by their root mean square at most
    for got, want in ((c.all(c.dx), xd.grad), (c.all(c.dgate), gd.grad)):
        got, want = got.double().flatten(), want.flatten()
        assert float((got - want).norm() / want.norm()) <= 4 * 2.0 ** -8


def test_far_rows():
    """Receive rows whose offsets pass 32 bits."""
    W, T, H, k = 2, 16000, 8192, 10
    c = Case(W, T, H, 16, k, seed=3)
    c.run()
    assert c.symm.status()["code"] == 0
    at = c.slot.view(W, T, k)
    for r, t in ((0, 0), (0, T - 1), (1, 777), (1, T - 1)):
        dout, gate, rows = c.dout(r)[t].double(), c.gate(r)[t].double(), at[r, t]
        assert torch.equal(c.dy[rows], (gate[:, None] * dout).float().to(torch.bfloat16))
        parts = c.y[rows].double() * dout
        assert bool(((c.dgate(r)[t].double() - parts.sum(-1)).abs() <= 2.0 ** -23 * (H + 8) * parts.abs().sum(-1)).all())
        parts = c.drecv[rows].double()
        tol = 2.0 ** -8 * parts.sum(0).abs() + 2.0 ** -23 * k * parts.abs().sum(0)
        assert bool(((c.dx(r)[t].double() - parts.sum(0)).abs() <= tol).all())


def test_replayed_with_other_data():
    c = Case(2, 31, 520, 8, 2, seed=7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        c.run()
        with torch.cuda.graph(graph, stream=side):
            c.run()
    torch.cuda.synchronize()
    other = Case(2, 31, 520, 8, 2, seed=8)
    c.slot.copy_(other.slot)
    c.y.copy_(other.y)
    c.drecv.copy_(other.drecv)
    for r in range(2):
        c.dout(r).copy_(other.dout(r))
    graph.replay()
    torch.cuda.synchronize()
    c.check()
    first = c.all(c.dgate)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.all(c.dgate), first)


def test_refusals():
    c = Case(2, 8, 64, 8, 2)
    for f, args in ((tdg.moe_combine_grad, (c.gate_off, c.dout_off, c.dgate_off, c.slot, c.y, c.dy)), (tdg.moe_dispatch_grad, (c.dx_off, c.slot, c.drecv))):
        for i, bad, kind in [(len(args) - 1, c.y[:31], ValueError), (len(args) - 1, c.y.float(), TypeError), (len(args) - 1, c.y.t(), ValueError),
                             (len(args) - 1, c.y.cpu(), ValueError)]:
            broken = list(args)
            broken[i] = bad
            with pytest.raises(kind):
                f(c.symm, 8, 64, 2, *broken)
        with pytest.raises(TypeError):
            f(c.symm, 8, 64, 2, *[a.int() if a is c.slot else a for a in args])

    def rc(name, cls, defaults, **kw):
        a = cls(**{**dict(world=2, k=2, T=8, H=64), **defaults, **kw})
        return getattr(tdg.lib(), name)(c.symm.h, ctypes.byref(a), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    region = c.symm.region_ptr(1)
    one = dict(gate_off=c.gate_off, dout_off=c.dout_off, dgate_off=c.dgate_off, slot=c.slot.data_ptr(), y=c.y.data_ptr(), dy=c.dy.data_ptr())
    two = dict(dx_off=c.dx_off, slot=c.slot.data_ptr(), drecv=c.drecv.data_ptr())
    for name, cls, d in (("tdg_moe_combine_grad", tdg.MoeCombineGradArgs, one), ("tdg_moe_dispatch_grad", tdg.MoeDispatchGradArgs, two)):
        assert rc(name, cls, d) == tdg.TDG_OK and rc(name, cls, d, T=0) == tdg.TDG_OK
        for kw in (dict(world=1), dict(k=0), dict(k=33), dict(T=-1), dict(T=1 << 30), dict(H=0), dict(H=60), dict(H=1 << 30), dict(slot=None),
                   dict(slot=c.slot.data_ptr() + 4)):
            assert rc(name, cls, d, **kw) == tdg.TDG_ERR_INVALID, (name, kw)
        assert rc(name, cls, d, T=1000, k=1) == tdg.TDG_ERR_NOMEM
    for kw in (dict(y=None), dict(dy=None), dict(y=c.y.data_ptr() + 8), dict(dy=c.dy.data_ptr() + 8), dict(gate_off=6), dict(dgate_off=6), dict(dout_off=8),
               dict(dy=c.slot.data_ptr()), dict(dy=c.y.data_ptr() + 16), dict(dy=region + align(c.dout_off, 16)), dict(dgate_off=c.gate_off),
               dict(dgate_off=c.dout_off), dict(y=region + align(c.dgate_off, 16) - 16)):
        assert rc("tdg_moe_combine_grad", tdg.MoeCombineGradArgs, one, **kw) == tdg.TDG_ERR_INVALID, kw
    for kw in (dict(gate_off=c.symm.region_bytes), dict(dgate_off=(1 << 64) - 4), dict(dout_off=c.symm.region_bytes - 16)):
        assert rc("tdg_moe_combine_grad", tdg.MoeCombineGradArgs, one, **kw) == tdg.TDG_ERR_NOMEM, kw
    for kw in (dict(drecv=None), dict(drecv=c.drecv.data_ptr() + 8), dict(dx_off=8), dict(drecv=region + align(c.dx_off, 16)), dict(slot=region + c.dx_off)):
        assert rc("tdg_moe_dispatch_grad", tdg.MoeDispatchGradArgs, two, **kw) == tdg.TDG_ERR_INVALID, kw
    assert rc("tdg_moe_dispatch_grad", tdg.MoeDispatchGradArgs, two, dx_off=c.symm.region_bytes - 16) == tdg.TDG_ERR_NOMEM
    torch.cuda.synchronize()
    assert c.symm.status()["code"] == 0
