"""The example that runs projection, rotary cache write, prompt attention and
paged attention together: the attention of the prompts' last rows comes out the
same over whole prompts and over the cache."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("lengths", [(700, 33, 1, 258), (64,), (5, 129, 127, 128, 64, 63, 65, 2)])
def test_prompt_and_paged_attention_agree(example, lengths):
    # the same bf16 keys and values: both round the weights and the output once (2^-8 each, of the weighted values)
    worst, most = example.run(lengths, steps=3, seed=len(lengths))
    assert worst <= 4 * 2.0 ** -8 * max(most, 1.0)


def test_8_bit_cache(example):
    # keys and values off by 2^-4 of themselves move an output of unit-size values by no more than a few of that
    worst, most = example.run((300, 77), steps=2, e4m3=True, seed=9)
    assert worst <= 8 * 2.0 ** -4 * max(most, 1.0)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lengths,steps", [((700, 33, 1, 258), 4), ((63, 64, 65), 66)])
def test_every_call_against_64_bits(example, lengths, steps, e4m3):
    """Projection, rotation, every slot of the cache and every attention, of the prompts and of each step, from the
    bf16 rows that the calls were given; element by element, within the operators' own bounds."""
    import numpy as np
    import torch
    import oracle
    from attn_util import check_attention, to_bits
    from test_gpu_rope_append import _near, _near8
    H, K, D = example.HQ, example.HKV, example.D

    class Recorded(example.Block):
        def project(self, x):
            views = super().project(x)
            self.calls.append((x, [p.clone() for p in views], views))
            return views

    block = Recorded(lengths, steps, e4m3, seed=steps)
    block.calls = []
    g = torch.Generator(device="cuda").manual_seed(steps + 1)
    xs = [torch.randn(n, example.HIDDEN, generator=g, device="cuda").to(torch.bfloat16) for n in [sum(lengths)] + [len(lengths)] * steps]
    outs = [block.prompts(xs[0], lengths)[1]] + [block.token(x) for x in xs[1:]]
    torch.cuda.synchronize()
    assert block.heap.status()["code"] == 0 and block.lens.tolist() == [n + steps for n in lengths]

    cos_sin = block.cos_sin.cpu().numpy()
    ends = np.cumsum([0, *lengths])
    weight = block.weight.double()
    new = [([], [], []) for _ in lengths]           # of each sequence: turned keys, their error scale, values
    queries = []
    for i, (x, (q, k, v), views) in enumerate(block.calls):
        want = (x.double() @ weight).view(len(x), H + 2 * K, D)
        size = (x.double().abs() @ weight.abs()).view(len(x), H + 2 * K, D)
        off = (torch.cat([q, k, v], 1).double() - want).abs()
        assert (off <= 2.0 ** -8 * want.abs() + 2 * (example.HIDDEN + 1) * 2.0 ** -24 * size).all(), f"projection {i}"
        pos = np.concatenate([np.arange(n) for n in lengths]) if i == 0 else np.array(lengths) + i - 1
        pos = pos.astype(np.int32)[None]
        wq, mq = oracle.rope(to_bits(q), cos_sin, pos)
        wk, mk = oracle.rope(to_bits(k), cos_sin, pos)
        queries.append(to_bits(views[0]))
        _near(oracle.bf16_to_f64(queries[-1]), wq, mq, f"queries {i}")
        if i == 0:
            _near(oracle.bf16_to_f64(to_bits(views[1])), wk, mk, "keys")
        for b in range(len(lengths)):
            rows = slice(ends[b], ends[b + 1]) if i == 0 else slice(b, b + 1)
            for to, of in zip(new[b], (wk, mk, oracle.bf16_to_f64(to_bits(v)))):
                to.append(of[rows])

    pools = [np.concatenate([block.cache.pools(block.heap, r)[j].view(torch.uint8).cpu().numpy() for r in range(example.W)]) for j in range(2)]
    table = block.table.cpu().numpy()
    for b, n in enumerate(lengths):
        wk, mk, wv = (np.concatenate(x) for x in new[b])
        held = []
        for pool, want, mag, what in zip(pools, (wk, wv), (mk, 0 * wv), "kv"):
            rows = oracle.gather_pages(pool, table[b], n + steps)
            if e4m3:
                s = float(np.float32(0.02))
                _near8(oracle.e4m3_to_f64(rows), want / s, mag / s, f"cached {what} of sequence {b}")
                held.append(oracle.e4m3_to_f64(rows) * s)
            else:
                held.append(oracle.bf16_to_f64(np.ascontiguousarray(rows).view(np.uint16)))
                _near(held[-1], want, mag, f"cached {what} of sequence {b}")
        rows = slice(ends[b], ends[b + 1])                        # the prompt: over the rows themselves
        q, k, v = (oracle.bf16_to_f64(to_bits(p)[rows]) for p in block.calls[0][2])
        check_attention(to_bits(outs[0])[rows], oracle.attention(q, k, v), D, f"prompt {b}")
        for i in range(1, steps + 1):                             # each step: over the cache up to its token
            want = oracle.attention(oracle.bf16_to_f64(queries[i][b:b + 1]), held[0][:n + i], held[1][:n + i])
            check_attention(to_bits(outs[i])[b:b + 1], want, D, f"step {i} of sequence {b}")
