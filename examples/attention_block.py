"""One rank's attention block of a serving step, with the framework's own calls.

Prompts of different lengths go through the fused query-key-value projection
(AllGather + GEMM over the ranks' token shards), rotary positions and the cache
write, and attention over the whole prompts; then a few single tokens follow:
the same projection, rotary write and attention over the paged cache, whose
pages lie scattered over every rank's region of the symmetric heap.

    python examples/attention_block.py [--e4m3] [--steps N]

Weights and tokens are random.  What is checked: the single-token attention of
the cached tokens gives what the prompt attention gave for the same rows.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tile_centric_comm_gb300 import tdg  # noqa: E402

W, HIDDEN, HQ, HKV, D, PAGE = 8, 1024, 16, 2, 128, 64
COLS = (HQ + 2 * HKV) * D


def align(x, a=1024):
    return (x + a - 1) // a * a


class Block:
    """Heap, cache and weights of the block, for up to `rows` new rows a call."""

    def __init__(self, lengths, steps, e4m3=False, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        B = len(lengths)
        self.rows = align(max(sum(lengths), B), 8 * W)          # rows of a call, padded to whole shards
        need = [-(-(n + steps) // PAGE) for n in lengths]
        pages = -(-sum(need) // W)
        pool = tdg.paged_pool_bytes(pages, PAGE, HKV, D, e4m3)
        self.a_off = 0                                          # a rank's shard of the tokens
        self.g_off = align(self.rows // W * HIDDEN * 2)         # all of them, gathered
        k_off = align(self.g_off + self.rows * HIDDEN * 2)
        v_off = align(k_off + pool)
        self.part_off = align(v_off + pool)
        region = align(self.part_off + tdg.paged_decode_part_bytes(HQ, HKV, D))
        self.heap = tdg.Symm(W, region, 4096)
        scale = torch.full((HKV,), 0.02, device="cuda")
        self.cache = tdg.PagedCache(pages, PAGE, HKV, D, k_off, v_off, e4m3=e4m3,
                                    k_scale=scale if e4m3 else None, v_scale=scale if e4m3 else None)
        ids = torch.randperm(W * pages, generator=g, device="cuda").to(torch.int32)
        self.table = torch.zeros(B, max(need), dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.weight = (torch.randn(HIDDEN, COLS, generator=g, device="cuda") / HIDDEN ** 0.5).to(torch.bfloat16)
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        freq = 1e4 ** (-torch.arange(D // 2, device="cuda") / (D // 2))
        angle = torch.arange(max(lengths) + steps, device="cuda")[:, None] * freq
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1)
        self.side = torch.cuda.Stream()

    def project(self, x):
        """Rows of queries, keys and values of the tokens x, as views of one buffer."""
        n = x.shape[0]
        Ms = align(n, 8 * W) // W
        padded = torch.zeros(W * Ms, HIDDEN, dtype=torch.bfloat16, device="cuda")
        padded[:n] = x
        for r in range(W):                                      # the sequence-parallel shards
            self.heap.view(r, self.a_off, (Ms, HIDDEN), torch.bfloat16).copy_(padded[r * Ms:(r + 1) * Ms])
        qkv = torch.empty(W * Ms, COLS, dtype=torch.bfloat16, device="cuda")
        tdg.ag_gemm(self.heap, 0, Ms, HIDDEN, COLS, self.a_off, self.g_off, self.weight, qkv, mode="ce",
                    side_stream=self.side)
        heads = qkv[:n].view(n, HQ + 2 * HKV, D)
        return heads[:, :HQ], heads[:, HQ:HQ + HKV], heads[:, HQ + HKV:]

    def prompts(self, x, lengths):
        """Attention of whole prompts packed in the rows of x; fills the cache."""
        n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        cu = torch.nn.functional.pad(n.cumsum(0), (1, 0)).to(torch.int32)
        pos = torch.cat([torch.arange(m, dtype=torch.int32, device="cuda") for m in lengths])
        q, k, v = self.project(x)
        self.lens += n
        tdg.rope_append(self.heap, self.cache, q, k, v, q, self.cos_sin, pos, self.table, self.lens, cu=cu, k_out=k)
        out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        tdg.prompt_attention(self.heap, q, k, v, out, cu, cu)
        return q, out

    def token(self, x):
        """Attention of one new token per sequence, row b of x that of sequence b."""
        q, k, v = self.project(x)
        pos = self.lens.clone()
        self.lens += 1
        tdg.rope_append(self.heap, self.cache, q, k, v, q, self.cos_sin, pos, self.table, self.lens)
        return self.attend(q, self.lens)

    def attend(self, q, lens):
        out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        tdg.paged_decode(self.heap, self.cache, q, out, self.table, lens, self.part_off)
        return out


def run(lengths=(700, 33, 1, 258), steps=4, e4m3=False, seed=0):
    """Returns (largest difference between the two attentions of the same rows, largest value)."""
    block = Block(lengths, steps, e4m3, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)

    def tokens(n):
        return torch.randn(n, HIDDEN, generator=g, device="cuda").to(torch.bfloat16)
    q, out = block.prompts(tokens(sum(lengths)), lengths)
    # the prompts' last rows again, as single tokens over the cache
    last = torch.tensor(lengths, device="cuda").cumsum(0) - 1
    again = block.attend(q[last].contiguous(), block.lens)
    worst = (again.float() - out[last].float()).abs().max().item()
    most = out[last].float().abs().max().item()
    for _ in range(steps):
        out = block.token(tokens(len(lengths)))
    assert torch.isfinite(out.float()).all()
    assert block.lens.tolist() == [n + steps for n in lengths]
    status = block.heap.status()
    assert status["code"] == tdg.TDG_OK, status
    return worst, most


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--e4m3", action="store_true", help="an 8-bit cache")
    ap.add_argument("--steps", type=int, default=4, help="single tokens after the prompts")
    a = ap.parse_args()
    worst, most = run(steps=a.steps, e4m3=a.e4m3)
    print(f"prompts, then {a.steps} tokens a sequence: ok; the prompts' last rows over the cache differ by "
          f"{worst:.3g} of {most:.3g}")
