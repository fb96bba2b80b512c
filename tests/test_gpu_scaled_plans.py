"""Products of 8-bit matrices by the kernel that each size goes to: what a call
launches is read from a capture of it, so that a size which a later choice
sends elsewhere fails here instead of leaving a kernel untested."""
import pytest
import torch

from expert_util import check_product, generator, product
from launch_util import launches
from test_gpu_scaled_gemm import E4M3, MARK, Case, blocks
from tile_centric_comm_gb300 import tdg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def symm():
    return tdg.Symm(1, 1024, 16)


def plan(symm, case, base=None):
    """(kernel, CTAs, CTAs of a cluster) of each launch of the case's call."""
    def short(name):
        kinds = [k for k, part in (("wide", "scaled_wide_kernel"), ("narrow 64", "NarrowShapeILi64E"), ("narrow 128", "NarrowShapeILi128E")) if part in name]
        assert len(kinds) == 1, name
        return kinds[0]
    return [(short(name), ctas, cluster) for name, ctas, cluster in launches(lambda s: case.run(symm, base, stream=s))]


def wide_tiles(M, N):
    return -(-M // 256) * -(-N // 256)


def pairs():
    return torch.cuda.get_device_properties(0).multi_processor_count // 2


@pytest.mark.parametrize("M,N,K,kernel,cluster", [(1, 3200, 5120, "narrow 64", 4), (17, 264, 400, "narrow 64", 2), (300, 256, 272, "narrow 64", 1),
                                                  (100, 7160, 8208, "narrow 128", 2), (333, 5112, 3216, "narrow 128", 1),
                                                  (250, 5112, 2576, "wide", 4), (2000, 7160, 528, "wide", 2)])
def test_every_kernel_is_reached(symm, M, N, K, kernel, cluster):
    c = Case(M, N, K)
    assert [(k, n) for k, _, n in plan(symm, c)] == [(kernel, cluster)]
    c.run(symm)
    c.check(symm)


# one and two whole rounds of the grid, then what is behind them by two pairs a tile; 41 blocks of K: odd halves
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("lead", [0, 1])
@pytest.mark.parametrize("M,N", [(1000, 6136), (1500, 6872)])
def test_whole_rounds_then_halves_of_k(symm, M, N, lead, f32):
    c = Case(M, N, 5136, f32=f32, lead=lead)
    rest = wide_tiles(M, N) % pairs()
    assert plan(symm, c) == [("wide", 2 * pairs(), 2), ("wide", 4 * rest, 4)]
    c.run(symm)
    c.check(symm)
    before = c.out.clone()
    c.run(symm)
    assert torch.equal(c.out, before)


def test_two_launches_in_a_graph_and_on_streams_at_once(symm):
    cases = [Case(m, n, 5136, seed=i) for i, (m, n) in enumerate(((1000, 6136), (1500, 6872), (1000, 6136)))]
    for c in cases:
        assert len(plan(symm, c)) == 2
    streams = [torch.cuda.Stream() for _ in cases]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=streams[0]):
        for c in cases:
            c.run(symm)
    for _ in range(3):
        for c, s in zip(cases, streams):
            c.run(symm, stream=s)
    torch.cuda.synchronize()
    first = [c.out.clone() for c in cases]
    for c in cases:
        c.check(symm)
        c.out.fill_(MARK)
    graph.replay()
    torch.cuda.synchronize()
    for c, f in zip(cases, first):
        assert torch.equal(c.out, f)


# a pair walks several tiles: of 5, 10, 6 and 3 blocks, so that accumulators, scale chunks (of 4 blocks) and
# staging buffers carry over from a tile to the next in every phase
SEVERAL = [(2000, 7160, 528), (5000, 1032, 1168), (2500, 2072, 656), (3000, 5120, 272)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("lead", [0, 1])
@pytest.mark.parametrize("M,N,K", SEVERAL)
def test_several_wide_tiles_a_pair(symm, M, N, K, lead, f32):
    c = Case(M, N, K, f32=f32, lead=lead)
    assert plan(symm, c) == [("wide", 2 * pairs(), 2)] and wide_tiles(M, N) > pairs()
    c.run(symm)
    c.check(symm)


SHARES = {
    "ragged": ([700, 0, 513, 257, 1, 900, 29], 2312, 1168), "some empty": ([0, 1000, 0, 0, 611, 384, 0, 300], 2304, 656),
    "all to one": ([0, 2400, 0, 0], 2312, 1168), "whole tiles": ([256, 512, 768, 256, 512], 2568, 528),
}


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("first,spare", [(0, 0), (5, 70)])
@pytest.mark.parametrize("name", SHARES)
def test_experts_by_wide_tiles(symm, name, first, spare, f32):
    rows, N, K = SHARES[name]
    ends = [first]
    for n in rows:
        ends.append(ends[-1] + n)
    c = Case(ends[-1] + spare, N, K, E=len(rows), f32=f32)
    base = torch.tensor(ends, dtype=torch.int64, device="cuda")
    assert [(k, n) for k, _, n in plan(symm, c, base)] == [("wide", 2)]
    c.run(symm, base=base)
    c.check(symm, ends)


def test_wide_offsets_are_read_at_each_replay(symm):
    c = Case(2400, 2312, 1168, E=6)
    ends = torch.tensor([0, 400, 400, 900, 1500, 1501, 2400], device="cuda")
    assert [k for k, _, _ in plan(symm, c, ends)] == ["wide"]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        c.run(symm, ends)
    for new in ([0, 400, 400, 900, 1500, 1501, 2400], [3, 3, 2000, 2000, 2001, 2300, 2399], [9, 12, 20, 20, 21, 21, 33]):
        ends.copy_(torch.tensor(new))
        c.out.fill_(MARK)
        graph.replay()
        torch.cuda.synchronize()
        c.check(symm, new)


def test_integers_are_exact_in_wide_tiles(symm):
    g = generator(1)
    c = Case(2500, 2072, 656, f32=True)
    c.a.copy_(torch.randint(-8, 9, c.a.shape, generator=g, device="cuda").float().to(E4M3))
    c.b.copy_(torch.randint(-8, 9, c.b.shape, generator=g, device="cuda").float().to(E4M3))
    c.a_scale.copy_(torch.exp2(torch.randint(-1, 2, c.a_scale.shape, generator=g, device="cuda").float()))
    c.b_scale.copy_(torch.exp2(torch.randint(-1, 2, c.b_scale.shape, generator=g, device="cuda").float()))
    assert [k for k, _, _ in plan(symm, c)] == ["wide"]
    c.run(symm)
    want, _ = product(c.a, c.a_scale, c.b, c.b_scale)
    assert torch.equal(c.out.double(), want)


def test_a_row_that_is_not_finite_stays_alone_in_wide_tiles(symm):
    M, N, K = 2500, 2072, 656
    c = Case(M, N, K)
    assert [k for k, _, _ in plan(symm, c)] == ["wide"]
    clean = c.run(symm).clone()
    c.a.view(torch.uint8)[7, 3] = 0x7F           # NaN
    c.a_scale[1300, 0] = float("inf")
    c.a_scale[M - 1, blocks(K) - 1] = float("nan")
    c.run(symm)
    good = torch.ones(M, dtype=torch.bool, device="cuda")
    good[[7, 1300, M - 1]] = False
    assert torch.equal(c.out[good], clean[good])
    assert bool(c.out[7].isnan().all()) and not bool(c.out[1300].isfinite().any()) and bool(c.out[M - 1].isnan().all())
    c = Case(M, N, K)
    c.b.view(torch.uint8)[1030, 1] = 0xFF        # and a row of weights one column
    c.run(symm)
    good = torch.arange(N, device="cuda") != 1030
    assert torch.equal(c.out[:, good], clean[:, good]) and bool(c.out[:, 1030].isnan().all())


def test_rows_behind_an_expert_never_reach_it_in_wide_tiles(symm):
    """What a tile reads past an expert's last row is another expert's, or NaN; it is neither used nor written."""
    ends = [0, 600, 600, 1300, 1900, 2250]
    c = Case(2400, 2312, 1168, E=5)
    c.a.view(torch.uint8)[2250:] = 0x7F
    c.a_scale[2250:] = float("nan")
    base = torch.tensor(ends, device="cuda")
    assert [k for k, _, _ in plan(symm, c, base)] == ["wide"]
    c.run(symm, base=base)
    c.check(symm, ends)


@pytest.mark.parametrize("M,N,K,kernel", [(40, 136, 144, "narrow 64"), (2400, 2312, 1168, "wide")])
@pytest.mark.parametrize("ends,bad", [([-1, .25, .5, 1], {0}), ([0, .25, .125, 1], {1}), ([0, .25, .5, 1.025], {2}), ([0, 2.0 ** 20, .5, .75], {0, 1}),
                                      ([-2.0 ** 40, 2.0 ** 40, -3, .5], {0, 1, 2})])
def test_the_expert_whose_offsets_are_bad_is_named_and_left_out(symm, M, N, K, kernel, ends, bad):
    """ends in parts of M (-1 and -3 as they are): the status names one of the bad experts, and the others' rows are right."""
    ends = [int(v) if v in (-1, -3) else round(v * M) for v in ends]
    assert {e for e in range(3) if not 0 <= ends[e] <= ends[e + 1] <= M} == bad
    c = Case(M, N, K, E=3)
    base = torch.tensor(ends, dtype=torch.int64, device="cuda")
    assert [k for k, _, _ in plan(symm, c, base)] == [kernel]
    c.run(symm, base=base)
    torch.cuda.synchronize()
    st = symm.status()
    assert st["code"] == tdg.TDG_ERR_DEVICE and st["where"] == "cu" and st["index"] in bad
    covered = torch.zeros(M, dtype=torch.int64, device="cuda")
    for e in set(range(3)) - bad:
        covered[ends[e]:ends[e + 1]] += 1
    for e in set(range(3)) - bad:
        rows = torch.arange(ends[e], ends[e + 1], device="cuda")
        rows = rows[covered[rows] == 1]          # (a row of two experts is undefined)
        want, mag = product(c.a[rows], c.a_scale[rows], c.b[e], c.b_scale[e])
        check_product(c.out[rows], want, mag, K, f"expert {e}")
    assert bool((c.out[covered == 0] == MARK).all())


@pytest.mark.parametrize("M,N,K,kernel", [(4000, 512, 256, "narrow 64"), (40000, 512, 1040, "wide")])
def test_bad_offsets_take_no_longer_than_good_ones(symm, M, N, K, kernel):
    """Every other expert with all M rows, 128 times as many as there are: what the call computes stays bounded by M and E."""
    E = 256
    c = Case(M, N, K, E=E)
    good = torch.arange(E + 1, device="cuda") * M // E
    bad = torch.tensor([0, M] * (E // 2) + [0], device="cuda")
    assert [k for k, _, _ in plan(symm, c, good)] == [kernel]

    def time(base):
        times = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            c.run(symm, base)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)
    usual, ms = time(good), time(bad)
    assert symm.status()["where"] == "cu"
    assert ms < 4 * usual + 0.05                 # (128 times the products without the bound)
