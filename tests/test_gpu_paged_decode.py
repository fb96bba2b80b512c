"""GPU parity of the attention of single tokens over the paged cache against
the oracle: every slot that no sequence owns, and every slot behind a length,
holds NaN."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from tile_centric_comm_gb300 import tdg
from attn_util import Cache, bits, check_attention, check_lse, strided_rows, to_bits

pytestmark = pytest.mark.gpu


def run_case(c, Hq, seed=0, scale=0.0, stream=None, root=0, q_mul=1.0):
    g = np.random.default_rng(seed + 7)
    B, D = len(c.lens), c.D
    q = bits(g.standard_normal((B, Hq, D)) * q_mul)
    _, (qd, out) = strided_rows([q, np.full_like(q, 0x7FC1)])
    lse = torch.full((B, Hq), float("nan"), device="cuda")
    tdg.paged_decode(c.symm, c.cache, qd, out, c.table_d, c.lens_d, c.part_off, root=root, lse=lse, scale=scale,
                     stream=stream)
    torch.cuda.synchronize()
    assert c.symm.status()["code"] == 0
    return q, to_bits(out), lse.cpu().numpy()


def check_case(c, Hq, got, some=None, scale=0.0):
    q, out, lse = got
    for b in range(len(c.lens)) if some is None else some:
        k, v = c.sequence(b)
        want = oracle.attention(oracle.bf16_to_f64(q[b:b + 1]), k, v, True, scale or None)
        check_attention(out[b:b + 1], want, c.D, f"sequence {b} of {c.lens[b]}")
        check_lse(lse[b:b + 1], want, c.D, f"lse of sequence {b}")




@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("W,page,Hq,Hkv", [
    (1, 16, 8, 1),
    (2, 32, 5, 5),      # one query head per key head
    (3, 64, 14, 2),     # 7
    (4, 128, 32, 2),    # 16
    (2, 256, 40, 2),    # 20: more than one group of 16 heads
    (8, 16, 64, 8),
])
def test_lengths(D, e4m3, W, page, Hq, Hkv):
    # none, one, around the pages' and the tiles' ends
    lens = [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 200, 0, 257, 500]
    c = Cache(W, lens, Hkv, D, page, e4m3, seed=Hq + D, extra_entries=1)
    got = run_case(c, Hq, seed=Hq, root=W - 1)
    check_case(c, Hq, got)
    again = run_case(c, Hq, seed=Hq, root=W - 1)
    assert all(np.array_equal(a, b) for a, b in zip(got, again))     # the same bits every time


@pytest.mark.parametrize("lens", [[1], [5000], [70000], [9000, 1, 0, 30000], [64] * 700, [3] * 1500])
def test_splits(lens):
    c = Cache(4, lens, 2, 64, 16, seed=len(lens))
    got = run_case(c, 16, seed=1)
    check_case(c, 16, got, some=range(0, len(lens), max(1, len(lens) // 40)))


def test_all_empty_and_no_sequences():
    c = Cache(2, [0, 0, 0], 2, 128, 16)
    check_case(c, 4, run_case(c, 4))
    q = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    tdg.paged_decode(c.symm, c.cache, q, q.clone(), c.table_d[:0], c.lens_d[:0], c.part_off)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("q_mul", [1e-30, 1e-3, 30.0])
def test_query_sizes(e4m3, q_mul):
    # tiny queries give nearly even weights, large ones nearly a single one
    c = Cache(2, [700, 33, 129], 2, 128, 32, e4m3, seed=3)
    check_case(c, 16, run_case(c, 16, seed=4, q_mul=q_mul))


def test_scale_stream_and_graph():
    c = Cache(2, [90, 300, 1000], 2, 128, 16, seed=8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    check_case(c, 8, run_case(c, 8, seed=2, scale=0.25, stream=s), scale=0.25)
    # captured once, replayed on longer sequences
    g = np.random.default_rng(9)
    q = bits(g.standard_normal((3, 8, 128)))
    _, (qd,) = strided_rows([q])
    out, lse = torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((3, 8), device="cuda")
    lens = torch.ones_like(c.lens_d)
    graph = torch.cuda.CUDAGraph()
    tdg.paged_decode(c.symm, c.cache, qd, out, c.table_d, lens, c.part_off, lse=lse)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        tdg.paged_decode(c.symm, c.cache, qd, out, c.table_d, lens, c.part_off, lse=lse)
    for n in ([90, 300, 1000], [0, 65, 64]):
        lens.copy_(torch.tensor(n))
        graph.replay()
        torch.cuda.synchronize()
        for b in range(3):
            k, v = c.sequence(b, n[b])
            want = oracle.attention(oracle.bf16_to_f64(q[b:b + 1]), k, v)
            check_attention(to_bits(out)[b:b + 1], want, 128)
            check_lse(lse.cpu().numpy()[b:b + 1], want, 128)


@pytest.mark.slow
def test_pools_past_32_bits():
    # 4.6 GB per pool and region: byte offsets and element indices of the last pages pass 2^32
    W, Hkv, D, page = 2, 8, 128, 128
    pages = 17600
    pool = tdg.paged_pool_bytes(pages, page, Hkv, D)
    assert pool > 1 << 32
    v_off = -(-pool // 1024) * 1024
    part_off = 2 * v_off
    symm = tdg.Symm(W, part_off + tdg.paged_decode_part_bytes(64, Hkv, D), 64)
    cache = tdg.PagedCache(pages, page, Hkv, D, 0, v_off)
    g = np.random.default_rng(1)
    ids = [2 * pages - 1, 0, pages - 1, pages, 2 * pages - 2]
    n = 4 * page + 77
    k, v = bits(g.standard_normal((5, Hkv, page, D))), bits(g.standard_normal((5, Hkv, page, D)))
    for i, p in enumerate(ids):
        for src, dst in zip((k, v), cache.pools(symm, p // pages)):
            dst[p % pages].copy_(torch.from_numpy(src[i].view(np.int16)).view(torch.bfloat16))
    q = bits(g.standard_normal((1, 64, D)))
    qd = torch.from_numpy(q.view(np.int16)).view(torch.bfloat16).cuda()
    out = torch.empty_like(qd)
    tdg.paged_decode(symm, cache, qd, out, torch.tensor([ids], dtype=torch.int32, device="cuda"),
                     torch.tensor([n], dtype=torch.int32, device="cuda"), part_off)
    torch.cuda.synchronize()
    assert symm.status()["code"] == 0
    row = np.arange(5)
    want = oracle.attention(oracle.bf16_to_f64(q), oracle.bf16_to_f64(oracle.gather_pages(k, row, n)),
                            oracle.bf16_to_f64(oracle.gather_pages(v, row, n)))
    check_attention(to_bits(out), want, D)


@pytest.mark.parametrize("what", ["negative", "long", "page"])
def test_bad_indices_are_reported(what):
    c = Cache(2, [90, 300], 2, 128, 16, seed=8)
    if what == "negative":
        c.lens_d[0] = -5
    elif what == "long":
        c.lens_d[0] = 16 * c.table.shape[1] + 1
    else:
        c.table_d[0, 2] = 2 * c.pages
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    tdg.paged_decode(c.symm, c.cache, q, out, c.table_d, c.lens_d, c.part_off)
    torch.cuda.synchronize()
    st = c.symm.status()
    assert st["code"] == tdg.TDG_ERR_DEVICE and st["where"] == "page" and st["index"] == 0
    k, v = c.sequence(1)                       # the other sequence is untouched by it
    check_attention(to_bits(out)[1:], oracle.attention(np.zeros((1, 8, 128)), k, v), 128)


def test_refusals():
    c = Cache(2, [90, 300], 2, 128, 16, seed=8)
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)

    def rc(desc=(), **kw):
        n = c.table.shape[1]
        a = tdg.PagedDecodeArgs(world=2, root=0, cache=c.cache.desc, B=2, Hq=8, q=q.data_ptr(), q_stride=1024,
                                out=out.data_ptr(), out_stride=1024, table=c.table_d.data_ptr(), table_entries=n,
                                table_stride=n, lens=c.lens_d.data_ptr(), part_off=c.part_off)
        for key, v in kw.items():
            setattr(a, key, v)
        for key, v in desc:
            setattr(a.cache, key, v)
        return tdg.lib().tdg_paged_decode(c.symm.h, ctypes.byref(a), None)

    bad, nomem = tdg.TDG_ERR_INVALID, tdg.TDG_ERR_NOMEM
    assert rc() == tdg.TDG_OK
    assert rc(world=3) == bad and rc(root=2) == bad and rc(root=-1) == bad
    assert rc(B=-1) == bad and rc(B=65536) == bad
    assert rc(Hq=9) == bad and rc(Hq=0) == bad and rc(Hq=2 * 129, q_stride=1 << 16, out_stride=1 << 16) == bad
    assert rc(q=None) == bad and rc(q=q.data_ptr() + 8) == bad and rc(q_stride=1016) == bad and rc(out_stride=1028) == bad
    assert rc(table=None) == bad and rc(lens=None) == bad and rc(table_entries=-1) == bad
    assert rc(table_stride=1) == bad
    assert rc(scale=-1.0) == bad and rc(scale=float("nan")) == bad and rc(scale=float("inf")) == bad
    assert rc(part_off=8) == bad and rc(part_off=0) == bad             # over the keys
    assert rc(part_off=c.symm.region_bytes) == nomem
    assert rc(desc=[("D", 96)]) == bad and rc(desc=[("Hkv", 3)]) == bad and rc(desc=[("page_size", 0)]) == bad
    assert rc(desc=[("k_scale", q.data_ptr())]) == bad and rc(desc=[("pages", 0)]) == bad
    assert rc(desc=[("pages", 1 << 30)]) == bad                        # page ids past 2^31
    with pytest.raises(ValueError, match="table"):
        tdg.paged_decode(c.symm, c.cache, q, out, c.table_d[:1], c.lens_d, c.part_off)
    with pytest.raises(TypeError, match="int32"):
        tdg.paged_decode(c.symm, c.cache, q, out, c.table_d.long(), c.lens_d, c.part_off)
    with pytest.raises(TypeError, match="bfloat16"):
        tdg.paged_decode(c.symm, c.cache, q.half(), out, c.table_d, c.lens_d, c.part_off)
    torch.cuda.synchronize()
    assert c.symm.status()["code"] == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page,Hq,Hkv", [(16, 8, 1), (64, 14, 2), (256, 40, 2), (32, 24, 24)])
def test_lengths_in_a_wide_table(D, e4m3, page, Hq, Hkv):
    # a table for far longer sequences: no cluster takes a pair, equal runs of the line are taken
    lens = [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 200, 0, 257, 500, 900, 3, 64, 0]
    c = Cache(2, lens, Hkv, D, page, e4m3, seed=Hq + D, extra_entries=16384 // page)
    got = run_case(c, Hq, seed=Hq)
    check_case(c, Hq, got)
    again = run_case(c, Hq, seed=Hq)
    assert all(np.array_equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("Hkv,lens", [
    (1, [1]), (1, [65]), (1, [128]), (1, [129]), (1, [500]), (2, [511, 64]), (3, [1000, 0, 1, 777]),
    (8, [100] * 9 + [0, 128]), (19, [130, 64]), (37, [300, 0]), (150, [70, 129]),
])
def test_clusters(e4m3, Hkv, lens):
    # from 8 CTAs a pair to one, with more CTAs than tiles, and with empty sequences
    c = Cache(1, lens, Hkv, 128, 16, e4m3, seed=Hkv)
    got = run_case(c, 4 * Hkv, seed=Hkv)
    check_case(c, 4 * Hkv, got)


@pytest.mark.parametrize("what", ["negative", "long", "page"])
def test_bad_indices_in_a_wide_table(what):
    c = Cache(2, [90, 300], 2, 128, 16, seed=8, extra_entries=1024)
    if what == "negative":
        c.lens_d[0] = -5
    elif what == "long":
        c.lens_d[0] = 16 * c.table.shape[1] + 1
    else:
        c.table_d[0, 2] = 2 * c.pages
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    tdg.paged_decode(c.symm, c.cache, q, out, c.table_d, c.lens_d, c.part_off)
    torch.cuda.synchronize()
    st = c.symm.status()
    assert st["code"] == tdg.TDG_ERR_DEVICE and st["where"] == "page" and st["index"] == 0
    k, v = c.sequence(1)
    check_attention(to_bits(out)[1:], oracle.attention(np.zeros((1, 8, 128)), k, v), 128)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_queries_of_many_short_pairs(e4m3, D):
    # a dozen pairs a CTA, each of one tile: the queries' two buffers are refilled all the time, and every
    # pair's queries have a size of their own, so that another pair's would show
    B, Hq, Hkv = 900, 32, 4
    lens = [1 + 5 * i % 7 for i in range(B)]
    c = Cache(2, lens, Hkv, D, 16, e4m3, seed=D)
    g = np.random.default_rng(D + 1)
    q = bits(g.standard_normal((B, Hq, D)) * np.exp2(g.integers(-3, 3, (B, Hkv, 1, 1)).repeat(Hq // Hkv, 2).reshape(B, Hq, 1)))
    _, (qd, out) = strided_rows([q, np.full_like(q, 0x7FC1)])
    first = None
    for _ in range(5):
        lse = torch.full((B, Hq), float("nan"), device="cuda")
        tdg.paged_decode(c.symm, c.cache, qd, out, c.table_d, c.lens_d, c.part_off, lse=lse)
        torch.cuda.synchronize()
        got = q, to_bits(out), lse.cpu().numpy()
        if first is None:
            first = got
            check_case(c, Hq, got, some=range(0, B, 9))
        assert np.array_equal(got[1], first[1]) and np.array_equal(got[2], first[2])
    assert c.symm.status()["code"] == 0


def test_overlapping_calls_on_two_streams():
    # each with partial results of its own: two places of one region, then two regions
    lens = [5000, 0, 1, 300, 77, 9000]
    c = Cache(2, lens, 2, 128, 16, seed=21, extra_entries=2048)      # a wide table: both launches, with partial results
    part = tdg.paged_decode_part_bytes(16, 2, 128)
    symm = tdg.Symm(2, c.part_off + 2 * part, 64)
    for r in range(2):
        for to, of in zip(c.cache.pools(symm, r), c.cache.pools(c.symm, r)):
            to.copy_(of)
    g = np.random.default_rng(22)
    q = [bits(g.standard_normal((B, 16, 128))) for B in (6, 4)]
    qd = [torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).cuda() for x in q]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for offs, roots in (((c.part_off, c.part_off + part), (0, 0)), ((c.part_off, c.part_off), (0, 1))):
        outs = [[torch.empty_like(x) for _ in range(20)] for x in qd]
        torch.cuda.synchronize()
        for i in range(20):
            for j, n in enumerate((6, 4)):
                tdg.paged_decode(symm, c.cache, qd[j], outs[j][i], c.table_d[:n], c.lens_d[:n], offs[j], root=roots[j],
                                 stream=streams[j])
        torch.cuda.synchronize()
        assert symm.status()["code"] == 0
        for j, n in enumerate((6, 4)):
            for b in range(n):
                k, v = c.sequence(b)
                want = oracle.attention(oracle.bf16_to_f64(q[j][b:b + 1]), k, v)
                check_attention(to_bits(outs[j][0])[b:b + 1], want, 128, f"call {j}, sequence {b}")
            assert all(torch.equal(o.view(torch.int16), outs[j][0].view(torch.int16)) for o in outs[j])


@pytest.mark.parametrize("extra", [0, 1024])
def test_refuses_what_would_overwrite_its_inputs(extra):
    # both paths; nothing is launched: the heap, tables and outputs keep their bytes
    c = Cache(2, [90, 300], 2, 128, 16, True, seed=8, extra_entries=extra)
    n = c.table.shape[1]
    row = 8 * 128 * 2                                           # bytes of an output row
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((2, 8), 7.0, device="cuda")
    scale = torch.full((4096,), 0.5, device="cuda")             # the key scales lie in a buffer with room behind them
    region, base, part = c.symm.region_bytes, c.symm.base, c.part_off

    def rc(desc=(), **kw):
        a = tdg.PagedDecodeArgs(world=2, root=0, cache=c.cache.desc, B=2, Hq=8, q=q.data_ptr(), q_stride=1024,
                                out=out.data_ptr(), out_stride=1024, lse=lse.data_ptr(), table=c.table_d.data_ptr(),
                                table_entries=n, table_stride=n, lens=c.lens_d.data_ptr(), part_off=part)
        a.cache.k_scale = scale.data_ptr()
        for key, v in kw.items():
            setattr(a, key, v)
        return tdg.lib().tdg_paged_decode(c.symm.h, ctypes.byref(a), None)

    bad = tdg.TDG_ERR_INVALID
    free = c.symm.base_off + region + part                      # rank 1's room for partial results is not used
    c.symm.buf[free:free + 16 * row] = 0xFF
    before = c.symm.buf.clone()
    part_bytes = tdg.paged_decode_part_bytes(8, 2, 128)
    for r in range(2):                                          # over the pools of any rank
        for off in (0, c.v_off):
            assert rc(out=base + r * region + off) == bad and rc(lse=base + r * region + off + 4) == bad
    assert rc(out=base + part) == bad and rc(out=base + part + part_bytes - 16) == bad   # over the partial results
    assert rc(lse=base + part) == bad and rc(q=base + part) == bad
    assert rc(q=base + part + part_bytes - 16) == bad
    assert rc(lse=out.data_ptr() + row) == bad and rc(lse=q.data_ptr() + 2 * row - 4) == bad
    assert rc(lse=c.lens_d.data_ptr()) == bad and rc(lse=c.table_d.data_ptr() + 4) == bad
    assert rc(lse=scale.data_ptr() + 4) == bad and rc(out=scale.data_ptr()) == bad
    assert rc(lens=base + part) == bad and rc(table=base + part + 64) == bad
    assert rc(lens=out.data_ptr()) == bad and rc(table=out.data_ptr() + 16) == bad
    torch.cuda.synchronize()
    assert torch.equal(c.symm.buf, before) and (out == 7).all() and (lse == 7).all()
    # next to one another is no overlap
    assert rc(out=base + region + part, lse=base + region + part + 2 * row, q=base + region + part + 2 * row + 64) == 0
    assert rc(lse=scale.data_ptr() + 8) == 0 and rc() == 0
    torch.cuda.synchronize()
    assert c.symm.status()["code"] == 0 and not torch.equal(c.symm.buf[free:free + 2 * row], before[free:free + 2 * row])


@pytest.mark.parametrize("extra", [0, 1024])
@pytest.mark.parametrize("unseen", [False, True])
@pytest.mark.parametrize("size", [2.0 ** 8, 2.0 ** 14, 2.0 ** 18])
def test_outlier_channel_over_an_8_bit_cache(size, unseen, extra):
    # one channel of every query far above the others; the keys use it, or hold 0 there, so that the small elements,
    # of which f16 drops the end below 2^-25 of the largest, decide
    c = Cache(2, [700, 33, 129], 2, 128, 32, True, seed=31, extra_entries=extra)
    if unseen:
        c.k[..., 5] = 0
        c.upload()
    g = np.random.default_rng(32)
    x = g.standard_normal((3, 16, 128))
    x[..., 5] = size * (1 + g.random((3, 16)))
    q = bits(x)
    qd = torch.from_numpy(q.view(np.int16)).view(torch.bfloat16).cuda()
    out, lse = torch.empty_like(qd), torch.empty((3, 16), device="cuda")
    tdg.paged_decode(c.symm, c.cache, qd, out, c.table_d, c.lens_d, c.part_off, lse=lse)
    torch.cuda.synchronize()
    assert c.symm.status()["code"] == 0
    out, lse, qv = to_bits(out), lse.cpu().numpy().astype(np.float64), oracle.bf16_to_f64(q)
    for b in range(3):
        k, v = c.sequence(b)
        want = oracle.attention(qv[b:b + 1], k, v)
        # a query element is off by 2^-25 of the largest, a score by that times the key's, which moves a weight by as
        # much and the sum of weights too; beside what any attention's scores are off by
        top = np.abs(qv[b:b + 1]).max(-1)
        off = 2.0 ** -25 * top * np.abs(k).sum(-1).max(0).repeat(8) / np.sqrt(128)
        tol = ((2 * 2.0 ** -8 + 128 * 2.0 ** -23 * want["smag"] + 2 * np.expm1(2 * off))[..., None]) * want["mag"] + 1e-30
        assert np.all(np.abs(oracle.bf16_to_f64(out[b:b + 1]) - want["out"]) <= tol), f"sequence {b}"
        tol = 128 * 2.0 ** -23 * want["smag"] + 2.0 ** -20 * (np.abs(want["lse"]) + 1) + off
        assert np.all(np.abs(lse[b] - want["lse"]) <= tol), f"lse of sequence {b}"
