"""The attention operators of a serving step, as cases that can be run and timed.

Three operators stand behind the projection GEMMs of an attention block and in
front of its output projection:

- ``write``   rotary positions (one axis, or time / height / width) on the
              queries and keys of the new tokens, and the keys and values
              written into the pages of the symmetric heap's key-value cache;
- ``prompt``  causal attention over whole prompts packed one after another,
              with grouped heads and, for prompts fed in pieces, keys that
              reach further back than the queries;
- ``decode``  attention of one new token per sequence over the paged cache.

``own = False`` computes them in elementary torch operations in 32 bits,
rounded once at the end; ``own = True`` calls the framework.
"""
import itertools
import math
import random

import torch

own = False

DEV = "cuda"
AXES = {1: None, 3: (16, 24, 24)}   # rotary pairs of each axis, for 64 pairs


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one sequence generating: the write of its newest token (latency only)
        dict(name="write_one", op="write", W=8, B=1, Hq=64, Hkv=8, page=64, fp8=False, lo=1000, hi=1000, new=1, axes=1, mix=1),
        # a full batch generating into an 8-bit cache
        dict(name="write_step_256_fp8", op="write", W=8, B=256, Hq=64, Hkv=8, page=16, fp8=True, lo=1, hi=4096, new=1, axes=1, mix=2),
        # prompts with images entering a bf16 cache, three position axes, ragged lengths
        dict(name="write_prompts_axes", op="write", W=8, B=9, Hq=64, Hkv=8, page=64, fp8=False, lo=301, hi=4093, new=0, axes=3, mix=3),
        # one short question
        dict(name="prompt_short", op="prompt", B=1, Hq=64, Hkv=8, D=128, lo=119, hi=119, past=0, lse=False, mix=4),
        # a batch of ragged prompts read in place from the fused projection's rows; 5 query heads share a key head
        dict(name="prompt_ragged", op="prompt", B=12, Hq=40, Hkv=8, D=128, lo=17, hi=2311, past=0, lse=False, mix=5),
        # a piece of a long prompt: 1024 new tokens behind 7000 that came before
        dict(name="prompt_piece", op="prompt", B=2, Hq=64, Hkv=8, D=128, lo=1000, hi=1024, past=7000, lse=True, mix=6),
        # heads of 64, every query head with its own key head
        dict(name="prompt_d64", op="prompt", B=4, Hq=32, Hkv=32, D=64, lo=2048, hi=4096, past=0, lse=False, mix=7),
        # one long document
        dict(name="prompt_8k", op="prompt", B=1, Hq=64, Hkv=8, D=128, lo=8192, hi=8192, past=0, lse=False, mix=8),
        # one sequence generating at a usual length (latency)
        dict(name="decode_one", op="decode", W=8, B=1, Hq=64, Hkv=8, page=64, fp8=False, lo=1000, hi=1000, lse=False, mix=9),
        # a batch of very different lengths in small pages
        dict(name="decode_ragged", op="decode", W=8, B=64, Hq=64, Hkv=8, page=16, fp8=False, lo=1, hi=8192, lse=False, mix=10),
        # a large batch over an 8-bit cache
        dict(name="decode_128_fp8", op="decode", W=8, B=128, Hq=64, Hkv=8, page=64, fp8=True, lo=2048, hi=4096, lse=False, mix=11),
        # two very long contexts over every rank's pages
        dict(name="decode_long", op="decode", W=8, B=2, Hq=64, Hkv=8, page=128, fp8=False, lo=200000, hi=262144, lse=True, mix=12),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "prompt", "decode"])
    mix = rng.randrange(1, 1 << 20)
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "prompt":
        D = rng.choice([64, 128])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
        past = rng.choice([0, 0, 0, _spread(rng, 1, 8000)])
        hi = _spread(rng, 1, 4096)
        # as many prompts as stay below the long document's padded score matrix
        B = _spread(rng, 1, max(1, min(48, 40000 // (hi + past), 64 * 8192 * 8192 // (2 * Hq * hi * (hi + past)))))
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, lo=rng.randint(1, hi), hi=hi, past=past, lse=rng.random() < 0.3, mix=mix)
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8, 16])
    W, page, fp8 = rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128]), rng.random() < 0.4
    if op == "write":
        steps = rng.random() < 0.5
        hi = _spread(rng, 1, 4096)
        B = _spread(rng, 1, 300 if steps else max(1, min(48, 16000 // hi)))
        return dict(op=op, W=W, B=B, Hq=Hq, Hkv=Hkv, page=page, fp8=fp8, lo=rng.randint(1, hi), hi=hi, new=1 if steps else 0,
                    axes=rng.choice([1, 3]), mix=mix)
    hi = _spread(rng, 1, 200000)
    B = _spread(rng, 1, max(1, min(300, 250000 // hi)))
    return dict(op=op, W=W, B=B, Hq=Hq, Hkv=Hkv, page=page, fp8=fp8, lo=rng.randint(1, hi), hi=hi, lse=rng.random() < 0.3, mix=mix)


def _lengths(case):
    """The sequences' lengths: they belong to the case, the longest among them."""
    r = random.Random(case["mix"])
    n = [case["hi"]] + [r.randint(case["lo"], case["hi"]) for _ in range(case["B"] - 1)]
    r.shuffle(n)
    return n


def work(case):
    n, Hq, Hkv = _lengths(case), case["Hq"], case["Hkv"]
    if case["op"] == "prompt":
        D, past = case["D"], case["past"]
        pairs = sum(m * past + m * (m + 1) // 2 for m in n)
        T = sum(n)
        by = 2 * D * (2 * T * Hq + 2 * (T + past * len(n)) * Hkv) + (4 * T * Hq if case["lse"] else 0)
        return {"bytes": by, "flops": 4 * D * Hq * pairs}
    D, e = 128, 1 if case["fp8"] else 2
    if case["op"] == "write":
        T = case["B"] if case["new"] else sum(n)
        axes = case["axes"]
        return {"bytes": T * (2 * D * (2 * Hq + 2 * Hkv) + 2 * D * Hkv * e + 4 * axes + 4 * D), "flops": T * 3 * D * (Hq + Hkv)}
    by = 2 * D * Hkv * e * sum(n) + case["B"] * Hq * D * 4 + 4 * sum(-(-m // case["page"]) for m in n) + (4 * case["B"] * Hq if case["lse"] else 0)
    return {"bytes": by, "flops": 4 * D * Hq * sum(n)}


# --------------------------------------------------------------- the inputs
def _normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(torch.bfloat16)


def _keys_values(g, T, Hkv, D):
    """Keys and values as projections give them: channels of unlike size, values around a mean of their own."""
    size = torch.rand(Hkv, D, generator=g, device=DEV) + 0.5
    mean = 0.3 * torch.randn(Hkv, D, generator=g, device=DEV)
    k = torch.randn(T, Hkv, D, generator=g, device=DEV) * size
    v = torch.randn(T, Hkv, D, generator=g, device=DEV) + mean
    return k, v


def _heap(case, s, g, n):
    """The ranks' page pools in one buffer, and a page table that scatters every sequence over them."""
    W, Hkv, ps, D = case["W"], case["Hkv"], case["page"], 128
    need = [-(-m // ps) for m in n]
    pages = -(-sum(need) // W) + 1                       # of each rank
    kind = torch.float8_e4m3fn if case["fp8"] else torch.bfloat16
    pool = pages * Hkv * ps * D * (1 if case["fp8"] else 2)
    v_off = (pool + 1023) // 1024 * 1024
    part_off = 2 * v_off
    region = part_off + (32 << 20)                       # room for the split attention's partial results
    buf = torch.zeros(W * region + 16384, dtype=torch.uint8, device=DEV)
    first = -buf.data_ptr() % 1024
    rows = buf[first:first + W * region].view(W, region)
    s["k_pool"] = rows[:, :pool].view(kind).unflatten(1, (pages, Hkv, ps, D))
    s["v_pool"] = rows[:, v_off:v_off + pool].view(kind).unflatten(1, (pages, Hkv, ps, D))
    order = torch.randperm(W * pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(len(n), max(need), dtype=torch.int32, device=DEV)
    used = torch.arange(max(need), device=DEV)[None, :] < torch.tensor(need, device=DEV)[:, None]
    table[used] = order[:sum(need)]
    s |= dict(buf=buf, region=region, table=table, pages=pages, v_off=v_off, part_off=part_off,
              k_scale=torch.rand(Hkv, generator=g, device=DEV) * 0.01 + 0.02, v_scale=torch.rand(Hkv, generator=g, device=DEV) * 0.01 + 0.02,
              lens=torch.tensor(n, dtype=torch.int32, device=DEV))
    if own:  # the handle over the buffer, and the cache's description, that a program keeps
        from tile_centric_comm_gb300 import tdg
        s["symm"] = tdg.Symm(W, region, 64, buffer=buf)
        s["cache"] = tdg.PagedCache(pages, ps, Hkv, D, 0, v_off, e4m3=case["fp8"],
                                    k_scale=s["k_scale"] if case["fp8"] else None, v_scale=s["v_scale"] if case["fp8"] else None)


def _ends(n):
    return torch.tensor([0, *itertools.accumulate(n)], dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + case["mix"])
    n, B, Hq, Hkv = _lengths(case), case["B"], case["Hq"], case["Hkv"]
    s = dict(case=case)
    if case["op"] == "prompt":
        D, past = case["D"], case["past"]
        T, Tk = sum(n), sum(n) + past * B
        if past:
            s["q"] = _normal(g, T, Hq, D)
            k, v = _keys_values(g, Tk, Hkv, D)
            s["k"], s["v"] = k.to(torch.bfloat16), v.to(torch.bfloat16)
        else:  # the rows of the fused query-key-value projection, read in place
            rows = _normal(g, T, Hq + 2 * Hkv, D)
            k, v = _keys_values(g, T, Hkv, D)
            rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:] = k.to(torch.bfloat16), v.to(torch.bfloat16)
            s["q"], s["k"], s["v"] = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        s |= dict(out=torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV), cu_q=_ends(n), cu_k=_ends([m + past for m in n]),
                  lse=torch.empty(T, Hq, dtype=torch.float32, device=DEV) if case["lse"] else None, most_q=max(n), most_k=max(n) + past)
        if own:  # the handle that a program keeps
            from tile_centric_comm_gb300 import tdg
            s["symm"] = tdg.Symm(1, 1024, 64)
        return s
    D = 128
    _heap(case, s, g, n)
    if case["op"] == "write":
        T = B if case["new"] else sum(n)
        rows = torch.empty(T, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
        k, v = _keys_values(g, T, Hkv, D)
        rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:] = _normal(g, T, Hq, D), k.to(torch.bfloat16), v.to(torch.bfloat16)
        s["q"], s["k"], s["v"] = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        s["cu"] = None if case["new"] else _ends(n)
        at = s["lens"].long() - 1 if case["new"] else torch.arange(T, device=DEV) - torch.repeat_interleave(s["cu"][:-1].long(), s["lens"].long())
        if case["axes"] == 1:
            s["pos"] = at.to(torch.int32)[None]
        else:  # rows of an image 32 wide: all of it at one time, at a height and a width of its own
            s["pos"] = torch.stack([at // 1024, at // 32 % 32 + at // 1024, at % 32 + at // 1024]).to(torch.int32).contiguous()
        angle = torch.arange(max(n), device=DEV, dtype=torch.float64)[:, None] * 1e6 ** (-torch.arange(64, device=DEV, dtype=torch.float64) / 64)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["seq"] = torch.arange(B, device=DEV) if case["new"] else torch.repeat_interleave(torch.arange(B, device=DEV), s["lens"].long())
        s["at"] = at
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["k_out"] = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
        return s
    for r in range(case["W"]):  # every page holds keys and values, those behind the lengths what earlier sequences left there
        kv = _keys_values(g, s["pages"] * case["page"], Hkv, D)
        for x, name in zip(kv, ("k", "v")):
            x = x.view(s["pages"], case["page"], Hkv, D).transpose(1, 2)
            if case["fp8"]:
                x = (x / s[name + "_scale"][None, :, None, None]).clamp(-448, 448)
            s[name + "_pool"][r].copy_(x.to(s[name + "_pool"].dtype))
    s |= dict(q=_normal(g, B, Hq, D), out=torch.empty(B, Hq, D, dtype=torch.bfloat16, device=DEV),
              lse=torch.empty(B, Hq, dtype=torch.float32, device=DEV) if case["lse"] else None)
    return s


# ----------------------------------------------------- one pass, either way
def _rotate(x, cos, sin):
    a, b = x[..., :64].float(), x[..., 64:].float()
    c, s = cos[:, None], sin[:, None]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _plain_write(s):
    case = s["case"]
    pos = s["pos"].long()
    if case["axes"] == 1:
        row = s["cos_sin"][pos[0]]
        cos, sin = row[:, :64], row[:, 64:]
    else:
        pair = torch.arange(64, device=DEV)
        axis = (pair >= AXES[3][0]).long() + (pair >= AXES[3][0] + AXES[3][1]).long()
        p = pos[axis].T                                    # [T, 64]: the position that each pair goes by
        cos, sin = s["cos_sin"][p, pair], s["cos_sin"][p, pair + 64]
    q, k, v = _rotate(s["q"], cos, sin), _rotate(s["k"], cos, sin), s["v"].float()
    page = s["table"].long()[s["seq"], s["at"] // case["page"]]
    where = (page // s["pages"], page % s["pages"], slice(None), s["at"] % case["page"])
    kq, vq = k, v
    if case["fp8"]:
        kq = (k / s["k_scale"][None, :, None]).clamp(-448, 448)
        vq = (v / s["v_scale"][None, :, None]).clamp(-448, 448)
    s["k_pool"][where] = kq.to(s["k_pool"].dtype)
    s["v_pool"][where] = vq.to(s["v_pool"].dtype)
    return [q.to(torch.bfloat16), k.to(torch.bfloat16), s["k_pool"], s["v_pool"]]


def _softmax_rows(scores, keep):
    scores = torch.where(keep, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(scores.sub_(top))
    total = p.sum(-1, keepdim=True)
    return p, total, (top + torch.log(total)).squeeze(-1)


def _plain_prompt(s):
    case = s["case"]
    Hq, Hkv, D, B = case["Hq"], case["Hkv"], case["D"], case["B"]
    G, Lq, Lk = Hq // Hkv, s["most_q"], s["most_k"]
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    nq, nk = cq.diff(), ck.diff()
    i, j = torch.arange(Lq, device=DEV), torch.arange(Lk, device=DEV)
    q = s["q"][(cq[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)].float() * (1 / math.sqrt(D))
    k = s["k"][(ck[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)].float()
    v = s["v"][(ck[:-1, None] + j).clamp(max=s["v"].shape[0] - 1)].float()
    q = q.view(B, Lq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Lq, D)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, Hkv, G, Lq, Lk)
    keep = j[None, None] <= i[None, :, None] + (nk - nq)[:, None, None]       # the last query sees the last key
    p, total, lse = _softmax_rows(scores, keep[:, None, None])
    del scores
    o = torch.matmul(p.view(B, Hkv, G * Lq, Lk), v.transpose(1, 2)).view(B, Hkv, G, Lq, D) / total
    real = i[None] < nq[:, None]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, Lq, Hq, D)[real].to(torch.bfloat16)
    return [o, lse.permute(0, 3, 1, 2).reshape(B, Lq, Hq)[real]] if case["lse"] else [o]


def _plain_decode(s):
    case = s["case"]
    Hq, Hkv, B, D, ps = case["Hq"], case["Hkv"], case["B"], 128, case["page"]
    page = s["table"].long()
    L = page.shape[1] * ps
    where = (page // s["pages"], page % s["pages"])
    k = s["k_pool"][where].float().transpose(1, 2).reshape(B, Hkv, L, D)
    v = s["v_pool"][where].float().transpose(1, 2).reshape(B, Hkv, L, D)
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D) * (1 / math.sqrt(D))
    if case["fp8"]:
        q = q * s["k_scale"][:, None, None]
    keep = (torch.arange(L, device=DEV)[None] < s["lens"][:, None])[:, None, None]
    p, total, lse = _softmax_rows(torch.matmul(q, k.transpose(2, 3)), keep)
    o = torch.matmul(p, v) / total
    if case["fp8"]:
        o = o * s["v_scale"][:, None, None]
    o = o.reshape(B, Hq, D).to(torch.bfloat16)
    return [o, lse.reshape(B, Hq)] if case["lse"] else [o]


def run(state):
    s, case = state, state["case"]
    if not own:
        return {"write": _plain_write, "prompt": _plain_prompt, "decode": _plain_decode}[case["op"]](s)
    from tile_centric_comm_gb300 import tdg
    if case["op"] == "write":
        tdg.rope_append(s["symm"], s["cache"], s["q"], s["k"], s["v"], s["q_out"], s["cos_sin"], s["pos"], s["table"], s["lens"],
                        cu=s["cu"], k_out=s["k_out"], sections=AXES[case["axes"]])
        return [s["q_out"], s["k_out"], s["k_pool"], s["v_pool"]]
    if case["op"] == "prompt":
        tdg.prompt_attention(s["symm"], s["q"], s["k"], s["v"], s["out"], s["cu_q"], s["cu_k"], lse=s["lse"])
    else:
        tdg.paged_decode(s["symm"], s["cache"], s["q"], s["out"], s["table"], s["lens"], s["part_off"], lse=s["lse"])
    return [s["out"], s["lse"]] if case["lse"] else [s["out"]]


# -------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    if case["op"] != "write" and work(case)["flops"] > 3e12:
        return None
    s = prepare(case, seed)
    n, Hq, Hkv = _lengths(case), case["Hq"], case["Hkv"]
    G = Hq // Hkv
    if case["op"] == "write":
        kp, vp = s["k_pool"].double(), s["v_pool"].double()
        T = s["q"].shape[0]
        turn = s["cos_sin"].double()
        pos = s["pos"].long()
        sizes = AXES[case["axes"]] or (64,)
        z = []
        lo = 0
        for a, m in enumerate(sizes):
            z.append(torch.complex(turn[pos[a], lo:lo + m], turn[pos[a], 64 + lo:64 + lo + m]))
            lo += m
        z = torch.cat(z, 1)[:, None]
        got = []
        for x in (s["q"], s["k"]):
            y = torch.complex(x[..., :64].double(), x[..., 64:].double()) * z
            got.append(torch.cat([y.real, y.imag], -1))
        q, k, v = got[0], got[1], s["v"].double()
        ks = s["k_scale"].double()[None, :, None] if case["fp8"] else 1.0
        vs = s["v_scale"].double()[None, :, None] if case["fp8"] else 1.0
        most = 448.0 if case["fp8"] else math.inf
        table = s["table"].tolist()
        ids = []
        for b, m in enumerate(n):
            for t in ([m - 1] if case["new"] else range(m)):
                ids.append((table[b][t // case["page"]], t % case["page"]))
        page, slot = torch.tensor(ids, device=DEV).T
        assert len(ids) == T
        kp.view(-1, Hkv, case["page"], 128)[page, :, slot] = (k / ks).clamp(-most, most)
        vp.view(-1, Hkv, case["page"], 128)[page, :, slot] = (v / vs).clamp(-most, most)
        return [q, k, kp, vp]
    outs, lses = [], []
    if case["op"] == "prompt":
        D, past = case["D"], case["past"]
        tq = tk = 0
        for m in n:
            q, k, v = s["q"][tq:tq + m].double(), s["k"][tk:tk + m + past].double(), s["v"][tk:tk + m + past].double()
            tq, tk = tq + m, tk + m + past
            o = torch.empty(m, Hq, D, dtype=torch.float64, device=DEV)
            e = torch.empty(m, Hq, dtype=torch.float64, device=DEV)
            late = torch.arange(m + past, device=DEV)[None] > past + torch.arange(m, device=DEV)[:, None]
            for h in range(Hq):
                x = (q[:, h] @ k[:, h // G].T / math.sqrt(D)).masked_fill(late, -math.inf)
                e[:, h] = torch.logsumexp(x, 1)
                o[:, h] = torch.exp(x - e[:, h, None]) @ v[:, h // G]
            outs.append(o)
            lses.append(e)
        o, e = torch.cat(outs), torch.cat(lses)
    else:
        for b, m in enumerate(n):
            used = s["table"][b, :-(-m // case["page"])].long()
            k, v = (s[p][used // s["pages"], used % s["pages"]].double().transpose(0, 1).reshape(Hkv, -1, 128)[:, :m] for p in ("k_pool", "v_pool"))
            if case["fp8"]:
                k, v = k * s["k_scale"].double()[:, None, None], v * s["v_scale"].double()[:, None, None]
            q = s["q"][b].double().view(Hkv, G, 128)
            x = torch.einsum("hgd,htd->hgt", q, k) / math.sqrt(128)
            e = torch.logsumexp(x, 2)
            outs.append(torch.einsum("hgt,htd->hgd", torch.exp(x - e[..., None]), v).reshape(1, Hq, 128))
            lses.append(e.reshape(1, Hq))
        o, e = torch.cat(outs), torch.cat(lses)
    return [o, e] if case["lse"] else [o]
