"""The operators of a mixture-of-experts layer in 8-bit floating point, and the
gradient of its dispatch and combine, as cases that can be run and timed.

A tensor "in 8 bits" is e4m3 codes with a float32 scale for each block of 128
along the contraction: activations one scale for each row and block (1 x 128),
weights one for each 128 x 128.

- ``product``   out[m, n] = sum over blocks b of sa[m, b] sw[n / 128, b] times the
                block's product of codes: the projection of one layer;
- ``experts``   the same with weights of many experts and rows sorted by expert;
- ``quantise``  rows (plain, or silu(gate) * up of a fused gate-up projection)
                and weights into codes and scales;
- ``dispatch``  tokens of every rank into their experts' rows, in 8 bits;
- ``grad``      the gradients of dispatch and combine: of the experts' outputs,
                the gates and the tokens.

``own = False`` computes them in elementary torch operations in 32 bits,
rounded once at the end; ``own = True`` calls the framework.
"""
import functools
import math
import random

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
LEAST = 2.0 ** -100   # the smallest scale: that of a block of zeros


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one token through one rank's share of an up-projection (weights read once: latency and bandwidth)
        dict(name="product_one", op="product", M=1, N=3200, K=5120, f32=False, mix=1),
        # an odd batch of a serving step through the down-projection, float32 sums for a reduction between ranks
        dict(name="product_odd", op="product", M=333, N=5120, K=3200, f32=True, mix=2),
        # a long prompt through a fused gate-up projection
        dict(name="product_prompt", op="product", M=8192, N=7168, K=8192, f32=False, mix=3),
        # 128 tokens' top-8 rows through the gate-up products of 64 experts, some without a row
        dict(name="experts_step", op="experts", E=64, rows=1024, N=4096, K=7168, skew=1.2, spare=64, f32=False, mix=4),
        # a prompt's rows through the down products of 32 experts
        dict(name="experts_prompt", op="experts", E=32, rows=32768, N=7168, K=2048, skew=0.5, spare=0, f32=False, mix=5),
        # a serving step's activations into 8 bits (latency)
        dict(name="quantise_step", op="quantise", kind="rows", n=37, K=5120, E=1, mix=6),
        # a prompt's rows between the experts' two products
        dict(name="quantise_gated", op="quantise", kind="gated", n=32768, K=2048, E=1, mix=7),
        # a layer's weights, once after loading or after each step of a trainer
        dict(name="quantise_weights", op="quantise", kind="blocks", n=4096, K=7168, E=8, mix=8),
        # a serving step: 16 tokens of each of 8 ranks to 8 of 256 experts
        dict(name="dispatch_step", op="dispatch", W=8, T=16, H=7168, E=256, k=8, mix=9),
        # prompts on every rank
        dict(name="dispatch_prompt", op="dispatch", W=8, T=1024, H=7168, E=256, k=8, mix=10),
        # a small training step, odd number of tokens, rows no multiple of anything large
        dict(name="grad_small", op="grad", W=2, T=257, H=520, E=8, k=2, mix=11),
        # a training step of the layer
        dict(name="grad_large", op="grad", W=8, T=1024, H=7168, E=256, k=8, mix=12),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["product", "experts", "quantise", "dispatch", "grad"])
    mix = rng.randrange(1, 1 << 20)
    if op == "product":
        N, K = 8 * _spread(rng, 1, 2000), 16 * _spread(rng, 1, 800)
        return dict(op=op, M=_spread(rng, 1, min(16384, 4e11 / (N * K))), N=N, K=K, f32=rng.random() < 0.3, mix=mix)
    if op == "experts":
        E = _spread(rng, 1, 256)
        K = 16 * _spread(rng, 4, 500)
        N = 8 * _spread(rng, 8, min(1000, 1.8e9 / (8 * E * K)))
        return dict(op=op, E=E, rows=_spread(rng, 1, min(50000, 4e11 / (N * K))), N=N, K=K, skew=rng.choice([0.0, 0.5, 1.2]),
                    spare=rng.choice([0, 0, 1, 100]), f32=rng.random() < 0.3, mix=mix)
    if op == "quantise":
        kind = rng.choice(["rows", "gated", "blocks"])
        K = 16 * _spread(rng, 1, 800)
        E = _spread(rng, 1, 16) if kind == "blocks" else 1
        return dict(op=op, kind=kind, n=_spread(rng, 1, min(40000, 2e8 / (K * E))), K=K, E=E, mix=mix)
    W, E = rng.choice([1, 2, 4, 8]), rng.choice([8, 16, 64, 256])
    k = rng.choice([1, 2, 4, 6, 8])
    H = 16 * _spread(rng, 8, 512) if op == "dispatch" else 8 * _spread(rng, 8, 1024)
    return dict(op=op, W=W, T=_spread(rng, 1, min(4096, 4.5e8 / (W * k * H))), H=H, E=E, k=k, mix=mix)


@functools.lru_cache(maxsize=64)
def _shares(E, rows, skew, mix):
    """How many rows each expert has: they belong to the case."""
    r = random.Random(mix)
    liked = [(i + 1.0) ** -skew for i in range(E)]
    r.shuffle(liked)
    n = [0] * E
    for e in r.choices(range(E), liked, k=rows):
        n[e] += 1
    return n


def _experts_rows(case):
    return _shares(case["E"], case["rows"], case["skew"], case["mix"])


def _blocks(n):
    return -(-n // 128)


def work(case):
    op = case["op"]
    if op in ("product", "experts"):
        N, K, e = case["N"], case["K"], 4 if case["f32"] else 2
        n = [case["M"]] if op == "product" else _experts_rows(case)
        used, M = sum(1 for m in n if m), sum(n)
        index = 8 * (len(n) + 1) if op == "experts" else 0
        return {"bytes": used * (N * K + 4 * _blocks(N) * _blocks(K)) + M * (K + 4 * _blocks(K)) + M * N * e + index, "flops": 2 * M * N * K}
    if op == "quantise":
        n, K, E = case["n"], case["K"], case["E"]
        x = n * K * E
        scales = E * (_blocks(n) if case["kind"] == "blocks" else n) * _blocks(K)
        return {"bytes": x * (4 if case["kind"] == "gated" else 2) + x + 4 * scales, "flops": x * (8 if case["kind"] == "gated" else 3)}
    T, H, k = case["W"] * case["T"], case["H"], case["k"]
    if op == "dispatch":
        return {"bytes": T * H * 2 + 8 * T * k + T * k * (H + 4 * _blocks(H)), "flops": 3 * T * H}
    return {"bytes": 2 * (2 * T * H + 3 * T * k * H) + T * k * (8 + 4 + 4), "flops": 4 * T * k * H}


# --------------------------------------------------------------- the inputs
def _rows_of(g, *shape):
    """Activations: channels of unlike size, a few of them large."""
    size = torch.rand(shape[-1], generator=g, device=DEV) + 0.5
    size[torch.randint(0, shape[-1], (max(1, shape[-1] // 100),), generator=g, device=DEV)] *= 20
    return (torch.randn(*shape, generator=g, device=DEV) * size).to(torch.bfloat16)


def _scale_of(x):
    """Scales of values whose last axis holds one block."""
    return (x.abs().amax(-1) / 448).clamp(min=LEAST)


def _codes(x):
    return x.clamp(-448, 448).to(E4M3)


def _pad(x, n, axis):
    """x with its axis filled up with zeros to n."""
    lack = n - x.shape[axis]
    if lack == 0:
        return x
    shape = list(x.shape)
    shape[axis] = lack
    return torch.cat([x, x.new_zeros(shape)], axis)


def _by_rows(x):
    """(n, K) float32 into codes and scales (n, K / 128)."""
    n, K = x.shape
    x = _pad(x, 128 * _blocks(K), 1).view(n, -1, 128)
    s = _scale_of(x)
    return _codes(x / s[..., None]).reshape(n, -1)[:, :K], s


def _by_blocks(x):
    """(n, K) float32 into codes and scales (n / 128, K / 128)."""
    n, K = x.shape
    x = _pad(_pad(x, 128 * _blocks(K), 1), 128 * _blocks(n), 0)
    x = x.view(_blocks(n), 128, -1, 128).transpose(1, 2)
    s = _scale_of(x.flatten(2))
    y = _codes(x / s[..., None, None])
    return y.transpose(1, 2).reshape(_blocks(n) * 128, -1)[:n, :K], s


def _weights(g, E, N, K):
    codes = torch.empty(E, N, K, dtype=E4M3, device=DEV)
    scale = torch.empty(E, _blocks(N), _blocks(K), device=DEV)
    for e in range(E):
        codes[e], scale[e] = _by_blocks((torch.randn(N, K, generator=g, device=DEV) / K ** 0.5))
    return codes, scale


def _heap(s, W, sizes):
    """Views of every rank's region, one for each (name, shape, type)."""
    at, where = 0, []
    for name, shape, kind in sizes:
        where.append(at)
        at += -(-math.prod(shape) * kind.itemsize // 1024) * 1024
    region = at
    buf = torch.zeros(W * region + 16384, dtype=torch.uint8, device=DEV)
    first = -buf.data_ptr() % 1024
    ranks = buf[first:first + W * region].view(W, region)
    for (name, shape, kind), off in zip(sizes, where):
        s[name] = ranks[:, off:off + math.prod(shape) * kind.itemsize].view(kind).unflatten(1, shape)
        s[name + "_off"] = off
    s["buf"] = buf
    if own:  # the handle over the buffer that a program keeps
        from tile_centric_comm_gb300 import tdg
        s["symm"] = tdg.Symm(W, region, 16, buffer=buf)


def _route(g, W, T, E, k):
    """Distinct experts of every token, some liked more, and the rows that they get: by expert, then rank, token, choice."""
    liked = -0.6 * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    liked = liked[torch.randperm(E, generator=g, device=DEV)]
    pick = torch.randn(W, T, E, generator=g, device=DEV).add_(liked).topk(k, -1).indices
    order = torch.sort(pick.flatten(), stable=True).indices
    slot = torch.empty_like(order)
    slot[order] = torch.arange(order.numel(), device=DEV)
    return slot.view(W, T, k)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + case["mix"])
    op = case["op"]
    s = dict(case=case)
    if op in ("product", "experts"):
        n = [case["M"]] if op == "product" else _experts_rows(case)
        M, N, K = sum(n) + case.get("spare", 0), case["N"], case["K"]
        s["a"], s["a_scale"] = _by_rows(_rows_of(g, M, K).float())
        s["a"] = s["a"].contiguous()
        s["b"], s["b_scale"] = _weights(g, len(n), N, K)
        if op == "product":
            s["b"], s["b_scale"] = s["b"][0], s["b_scale"][0]
        ends = [0]
        for m in n:
            ends.append(ends[-1] + m)
        s["ends"] = ends
        s["base"] = torch.tensor(ends, dtype=torch.int64, device=DEV) if op == "experts" else None
        s["out"] = torch.zeros(M, N, dtype=torch.float32 if case["f32"] else torch.bfloat16, device=DEV)
        if own:
            from tile_centric_comm_gb300 import tdg
            s["symm"] = tdg.Symm(1, 1024, 16)
        return s
    if op == "quantise":
        n, K, E = case["n"], case["K"], case["E"]
        if case["kind"] == "blocks":
            s["x"] = (torch.randn(E, n, K, generator=g, device=DEV) / K ** 0.5).to(torch.bfloat16)
            s["scale"] = torch.empty(E, _blocks(n), _blocks(K), device=DEV)
        else:
            s["x"] = _rows_of(g, n, 2 * K if case["kind"] == "gated" else K)
            s["scale"] = torch.empty(n, _blocks(K), device=DEV)
        s["codes"] = torch.empty(*s["x"].shape[:-1], K, dtype=E4M3, device=DEV)
        if own:
            from tile_centric_comm_gb300 import tdg
            s["symm"] = tdg.Symm(1, 1024, 16)
        return s
    W, T, H, E, k = case["W"], case["T"], case["H"], case["E"], case["k"]
    s["slot"] = _route(g, W, T, E, k)
    rows = W * T * k
    if op == "dispatch":
        _heap(s, W, [("x", (T, H), torch.bfloat16)])
        s["x"].copy_(_rows_of(g, W, T, H))
        s["codes"] = torch.empty(rows, H, dtype=E4M3, device=DEV)
        s["scale"] = torch.empty(rows, _blocks(H), device=DEV)
        return s
    _heap(s, W, [("gate", (T, k), torch.float32), ("dout", (T, H), torch.bfloat16), ("dx", (T, H), torch.bfloat16), ("dgate", (T, k), torch.float32)])
    s["gate"].copy_(torch.randn(W, T, k, generator=g, device=DEV).softmax(-1))
    s["dout"].copy_((torch.randn(W, T, H, generator=g, device=DEV) * 0.01).to(torch.bfloat16))
    s["y"] = _rows_of(g, rows, H)
    s["drecv"] = (torch.randn(rows, H, generator=g, device=DEV) * 0.01).to(torch.bfloat16)
    s["dy"] = torch.empty(rows, H, dtype=torch.bfloat16, device=DEV)
    return s


# ----------------------------------------------------- one pass, either way
def _values(codes, scale):
    """Codes with a scale for each row (or 128 rows) and block of 128, as float32 values."""
    n, K = codes.shape
    if scale.shape[0] != n:
        scale = scale.repeat_interleave(128, 0)[:n]
    return codes.float() * scale.repeat_interleave(128, 1)[:, :K]


def _plain_product(s):
    out, ends = s["out"], s["ends"]
    weights = [(s["b"], s["b_scale"])] if s["base"] is None else list(zip(s["b"], s["b_scale"]))
    for (b, b_scale), lo, hi in zip(weights, ends, ends[1:]):
        if hi > lo:
            out[lo:hi] = torch.matmul(_values(s["a"][lo:hi], s["a_scale"][lo:hi]), _values(b, b_scale).T).to(out.dtype)
    return [out]


def _plain_quantise(s):
    case = s["case"]
    if case["kind"] == "blocks":
        for e in range(case["E"]):
            s["codes"][e], s["scale"][e] = _by_blocks(s["x"][e].float())
        return [s["codes"], s["scale"]]
    x = s["x"].float()
    if case["kind"] == "gated":
        gate, up = x.chunk(2, 1)
        x = gate / (1 + torch.exp(-gate)) * up
    s["codes"][:], s["scale"][:] = _by_rows(x)
    return [s["codes"], s["scale"]]


def _plain_dispatch(s):
    codes, scale = _by_rows(s["x"].flatten(0, 1).float())
    k = s["case"]["k"]
    at = s["slot"].flatten()
    s["codes"].view(torch.uint8)[at] = codes.view(torch.uint8).repeat_interleave(k, 0)
    s["scale"][at] = scale.repeat_interleave(k, 0)
    return [s["codes"], s["scale"]]


def _plain_grad(s):
    W, T, H, k = (s["case"][c] for c in ("W", "T", "H", "k"))
    for r in range(W):
        at = s["slot"][r].flatten()
        dout = s["dout"][r].float()
        s["dy"][at] = (s["gate"][r][..., None] * dout[:, None]).to(torch.bfloat16).view(T * k, H)
        s["dgate"][r] = (s["y"][at].float().view(T, k, H) * dout[:, None]).sum(-1)
        s["dx"][r] = s["drecv"][at].float().view(T, k, H).sum(1).to(torch.bfloat16)
    return [s["dy"], s["dgate"], s["dx"]]


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"product": _plain_product, "experts": _plain_product, "quantise": _plain_quantise,
                "dispatch": _plain_dispatch, "grad": _plain_grad}[op](s)
    from tile_centric_comm_gb300 import tdg
    if op in ("product", "experts"):
        tdg.scaled_gemm(s["symm"], s["a"], s["a_scale"], s["b"], s["b_scale"], s["out"], base=s["base"])
        return [s["out"]]
    if op == "quantise":
        if case["kind"] == "blocks":
            tdg.quantise_blocks(s["symm"], s["x"], s["codes"], s["scale"])
        else:
            tdg.quantise_rows(s["symm"], s["x"], s["codes"], s["scale"], gated=case["kind"] == "gated")
        return [s["codes"], s["scale"]]
    if op == "dispatch":
        tdg.moe_dispatch_e4m3(s["symm"], case["T"], case["H"], case["k"], s["x_off"], s["slot"], s["codes"], s["scale"])
        return [s["codes"], s["scale"]]
    # the experts' own backward pass stands between the two and gives drecv
    T, H, k = case["T"], case["H"], case["k"]
    tdg.moe_combine_grad(s["symm"], T, H, k, s["gate_off"], s["dout_off"], s["dgate_off"], s["slot"], s["y"], s["dy"])
    tdg.moe_dispatch_grad(s["symm"], T, H, k, s["dx_off"], s["slot"], s["drecv"])
    return [s["dy"], s["dgate"], s["dx"]]


# -------------------------------------------------- the definition, 64 bits
def _exact_rows(x):
    """Quotients and scales of float64 rows, block by block."""
    codes, scales = torch.empty_like(x), []
    for lo in range(0, x.shape[1], 128):
        part = x[:, lo:lo + 128]
        sc = torch.maximum(part.max(1).values, -part.min(1).values) / 448
        sc = torch.where(sc < LEAST, torch.full_like(sc, LEAST), sc)
        codes[:, lo:lo + 128] = part / sc[:, None]
        scales.append(sc)
    return codes, torch.stack(scales, 1)


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op in ("product", "experts"):
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        for e, (lo, hi) in enumerate(zip(s["ends"], s["ends"][1:])):
            if lo == hi:
                continue
            b, sb = (s["b"], s["b_scale"]) if op == "product" else (s["b"][e], s["b_scale"][e])
            of = torch.arange(case["N"], device=DEV) // 128
            for j in range(_blocks(case["K"])):
                cut = slice(128 * j, 128 * j + 128)
                part = s["a"][lo:hi, cut].double() @ b[:, cut].double().T
                out[lo:hi] += part * s["a_scale"][lo:hi, j].double()[:, None] * sb[of, j].double()[None]
        return [out]
    if op == "quantise":
        x = s["x"].double()
        K, n = case["K"], case["n"]
        if case["kind"] == "gated":
            x = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
        if case["kind"] != "blocks":
            return list(_exact_rows(x))
        scale = torch.empty(s["scale"].shape, dtype=torch.float64, device=DEV)
        for i in range(_blocks(n)):
            for j in range(_blocks(K)):
                cut = (slice(None), slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128))
                part = x[cut]
                sc = part.abs().flatten(1).max(1).values / 448
                scale[:, i, j] = torch.where(sc < LEAST, torch.full_like(sc, LEAST), sc)
                x[cut] = part / scale[:, i, j, None, None]
        return [x, scale]
    W, T, H, k = (case[c] for c in ("W", "T", "H", "k"))
    if op == "dispatch":
        codes, scale = _exact_rows(s["x"].reshape(W * T, H).double())
        came_from = torch.empty(W * T * k, dtype=torch.int64, device=DEV)
        came_from[s["slot"].flatten()] = torch.arange(W * T * k, device=DEV) // k
        return [codes[came_from], scale[came_from]]
    dy = torch.empty(W * T * k, H, dtype=torch.float64, device=DEV)
    dgate = torch.empty(W, T, k, dtype=torch.float64, device=DEV)
    dx = torch.zeros(W, T, H, dtype=torch.float64, device=DEV)
    for j in range(k):
        at = s["slot"][..., j]
        dout = s["dout"].double()
        dy[at] = s["gate"][..., j, None].double() * dout
        dgate[..., j] = torch.einsum("wth,wth->wt", dout, s["y"][at].double())
        dx += s["drecv"][at].double()
    return [dy, dgate, dx]
