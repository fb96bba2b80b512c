"""Products of 8-bit matrices by the kernel that each size goes to: what a call
launches is read from a capture of it, so that a size which a later choice
sends elsewhere fails here instead of leaving a kernel untested."""
import pytest
import torch

from launch_util import launches
from test_gpu_scaled_gemm import MARK, Case
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
