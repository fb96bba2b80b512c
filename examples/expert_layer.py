"""A mixture-of-experts layer of a serving step in 8 bits, and the gradient of
its dispatch and combine, with the framework's own calls.

Every rank's tokens are routed to their top experts; the dispatch writes their
rows in 8 bits into the experts' rows; the experts' two products run over
ragged rows, silu(gate) * up quantised between them; the combine adds a token's
rows, weighted by its gates, where the token came from.

    python examples/expert_layer.py [--tokens N]

Weights and tokens are random.  What is shown: how far the layer's output is
from the same layer in float32, and, for experts that a program computes
itself (here one matrix for all, in plain torch), how far the gradients of
tokens and gates are from autograd's.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tile_centric_comm_gb300 import tdg  # noqa: E402

W, HIDDEN, INNER, EXPERTS, TOP = 4, 1024, 512, 32, 4


def align(x, a=1024):
    return (x + a - 1) // a * a


def blocks(n):
    return -(-n // 128)


class Layer:
    """Heap, weights and buffers of the layer for `tokens` tokens a rank."""

    def __init__(self, tokens, seed=0):
        self.T, T = tokens, tokens
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x_off = 0
        self.topk_off = align(T * HIDDEN * 2)
        self.gate_off = align(self.topk_off + T * TOP * 4)
        self.out_off = align(self.gate_off + T * TOP * 4)
        self.dx_off = align(self.out_off + T * HIDDEN * 2)       # the gradients' places
        self.dgate_off = align(self.dx_off + T * HIDDEN * 2)
        self.heap = tdg.Symm(W, align(self.dgate_off + T * TOP * 4), 16)
        self.rows = rows = W * T * TOP
        bf, f32, e4m3, i64 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int64

        def empty(*shape, dtype):
            return torch.empty(*shape, dtype=dtype, device="cuda")
        self.recv, self.y = empty(rows, HIDDEN, dtype=bf), empty(rows, HIDDEN, dtype=bf)
        self.counts, self.base, self.slot = empty(W * EXPERTS, dtype=i64), empty(EXPERTS + 1, dtype=i64), empty(rows, dtype=i64)
        self.workspace = empty(tdg.moe_workspace_bytes(W, T, EXPERTS), dtype=torch.uint8)
        self.x8, self.xs = empty(rows, HIDDEN, dtype=e4m3), empty(rows, blocks(HIDDEN), dtype=f32)
        self.h = empty(rows, 2 * INNER, dtype=bf)
        self.h8, self.hs = empty(rows, INNER, dtype=e4m3), empty(rows, blocks(INNER), dtype=f32)
        self.router = torch.randn(HIDDEN, EXPERTS, generator=g, device="cuda") / HIDDEN ** 0.5
        # the experts' weights: (experts, outputs, inputs), gate before up; laid out in 8 bits once
        self.w_in = (torch.randn(EXPERTS, 2 * INNER, HIDDEN, generator=g, device="cuda") / HIDDEN ** 0.5).to(bf)
        self.w_out = (torch.randn(EXPERTS, HIDDEN, INNER, generator=g, device="cuda") / INNER ** 0.5).to(bf)
        self.in8, self.in_s = self.quantised(self.w_in)
        self.out8, self.out_s = self.quantised(self.w_out)

    def quantised(self, w):
        codes = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device="cuda")
        scale = torch.empty(w.shape[0], blocks(w.shape[1]), blocks(w.shape[2]), device="cuda")
        tdg.quantise_blocks(self.heap, w, codes, scale)
        return codes, scale

    def moe(self, phases, y=None):
        tdg.moe_dispatch_combine(self.heap, self.T, HIDDEN, EXPERTS, TOP, self.x_off, self.topk_off, self.gate_off, self.out_off,
                                 self.recv, self.counts, self.base, self.slot, self.workspace, y=y, phases=phases)

    def all(self, off, shape, dtype):
        return torch.stack([self.heap.view(r, off, shape, dtype) for r in range(W)])

    def route(self, x):
        """Place the tokens x (W, T, HIDDEN), their experts and gates in the heap, and give every choice its row."""
        gate, top = (x.float() @ self.router).softmax(-1).topk(TOP, -1)
        gate = gate / gate.sum(-1, keepdim=True)
        for r in range(W):
            self.heap.view(r, self.x_off, x.shape[1:], torch.bfloat16).copy_(x[r])
            self.heap.view(r, self.topk_off, (self.T, TOP), torch.int32).copy_(top[r])
            self.heap.view(r, self.gate_off, (self.T, TOP), torch.float32).copy_(gate[r])
        self.moe(tdg.MOE_ROUTE)
        return gate, top

    def forward(self, x):
        """The layer of the tokens x (W, T, HIDDEN) bfloat16."""
        self.route(x)
        tdg.moe_dispatch_e4m3(self.heap, self.T, HIDDEN, TOP, self.x_off, self.slot, self.x8, self.xs)
        tdg.scaled_gemm(self.heap, self.x8, self.xs, self.in8, self.in_s, self.h, base=self.base)
        tdg.quantise_rows(self.heap, self.h, self.h8, self.hs, gated=True, count=self.base[EXPERTS:])
        tdg.scaled_gemm(self.heap, self.h8, self.hs, self.out8, self.out_s, self.y, base=self.base)
        self.moe(tdg.MOE_COMBINE, y=self.y)
        return self.all(self.out_off, (self.T, HIDDEN), torch.bfloat16)

    def plain(self, x, gate, top):
        """The layer in float32 from the weights themselves."""
        out = torch.zeros(x.shape, device="cuda")
        for e in range(EXPERTS):
            r, t, kk = (top == e).nonzero(as_tuple=True)
            g, u = (x[r, t].float() @ self.w_in[e].float().T).chunk(2, 1)
            out.index_put_((r, t), gate[r, t, kk, None] * ((torch.nn.functional.silu(g) * u) @ self.w_out[e].float().T), accumulate=True)
        return out

    def gradients(self, x, dout, weight):
        """Gradients of tokens and gates for experts y = tanh(x @ weight) that the program computes itself."""
        self.route(x)
        self.moe(tdg.MOE_DISPATCH)
        self.y.copy_(torch.tanh(self.recv.float() @ weight))
        for r in range(W):                                       # the gradient of the output, in the output's place
            self.heap.view(r, self.out_off, (self.T, HIDDEN), torch.bfloat16).copy_(dout[r])
        dy = torch.empty_like(self.y)
        tdg.moe_combine_grad(self.heap, self.T, HIDDEN, TOP, self.gate_off, self.out_off, self.dgate_off, self.slot, self.y, dy)
        drecv = (((1 - self.y.float() ** 2) * dy.float()) @ weight.T).to(torch.bfloat16)
        tdg.moe_dispatch_grad(self.heap, self.T, HIDDEN, TOP, self.dx_off, self.slot, drecv)
        return self.all(self.dx_off, (self.T, HIDDEN), torch.bfloat16), self.all(self.dgate_off, (self.T, TOP), torch.float32)


def apart(got, want):
    return ((got.double() - want.double()).norm() / want.double().norm()).item()


def run(tokens=50, seed=0):
    """Returns the relative differences of the output, of the tokens' gradient and of the gates'."""
    layer = Layer(tokens, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn(W, tokens, HIDDEN, generator=g, device="cuda").to(torch.bfloat16)
    out = layer.forward(x)
    gate, top = layer.route(x)
    off = apart(out, layer.plain(x, gate, top))

    weight = torch.randn(HIDDEN, HIDDEN, generator=g, device="cuda") / HIDDEN ** 0.5
    dout = torch.randn(W, tokens, HIDDEN, generator=g, device="cuda").to(torch.bfloat16)
    dx, dgate = layer.gradients(x, dout, weight)
    xr, gr = x.double().requires_grad_(), gate.double().requires_grad_()
    (gr[..., None] * torch.tanh(xr @ weight.double())[:, :, None]).sum(2).backward(dout.double())
    status = layer.heap.status()
    assert status["code"] == tdg.TDG_OK, status
    return off, apart(dx, xr.grad), apart(dgate, gr.grad)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=50, help="tokens of each rank")
    a = ap.parse_args()
    off, dx, dgate = run(a.tokens)
    print(f"{W} ranks x {a.tokens} tokens, {EXPERTS} experts, top {TOP}: output {off:.2%} off float32; "
          f"gradients of tokens {dx:.2%} and gates {dgate:.2%} off autograd")
