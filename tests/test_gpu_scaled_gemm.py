"""Products of 8-bit matrices with a scale for each block of 128, of one matrix
and of many experts', against the definition in 64 bits."""
import ctypes

import pytest
import torch

from expert_util import E4M3, blocks, check_product, generator, product, random_codes, random_scales
from tile_centric_comm_gb300 import tdg

pytestmark = pytest.mark.gpu
MARK = -77.0


@pytest.fixture(scope="module")
def symm():
    return tdg.Symm(1, 1024, 16)


class Case:
    def __init__(self, M, N, K, E=None, f32=False, lead=0, seed=0):
        g = generator(seed + 7 * M + N + K)
        self.M, self.N, self.K, self.E = M, N, K, E
        pad = 16 * lead
        self.a = random_codes(g, M, K + pad)[:, pad:]
        self.a_scale = random_scales(g, M, blocks(K) + lead)[:, lead:]
        lead_e = () if E is None else (E,)
        self.b = random_codes(g, *lead_e, N, K)
        self.b_scale = random_scales(g, *lead_e, blocks(N), blocks(K))
        self.wide = torch.full((M + 2, N + 2 * pad), MARK, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        self.out = self.wide[1:-1, pad:N + pad]
        self.pad = pad

    def run(self, symm, base=None, stream=None):
        tdg.scaled_gemm(symm, self.a, self.a_scale, self.b, self.b_scale, self.out, base=base, stream=stream)
        return self.out

    def check(self, symm, ends=None):
        """ends: the experts' row offsets; rows outside them keep their mark."""
        assert symm.status()["code"] == 0
        covered = torch.zeros(self.M, dtype=torch.bool, device="cuda")
        for e, (lo, hi) in enumerate(zip(ends, ends[1:]) if ends else [(0, self.M)]):
            if hi > lo:
                b, sb = (self.b, self.b_scale) if self.E is None else (self.b[e], self.b_scale[e])
                want, mag = product(self.a[lo:hi], self.a_scale[lo:hi], b, sb)
                check_product(self.out[lo:hi], want, mag, self.K, f"expert {e}")
                covered[lo:hi] = True
        assert bool((self.out[~covered] == MARK).all())
        assert bool((self.wide[0] == MARK).all()) and bool((self.wide[-1] == MARK).all())
        assert bool((self.wide[:, :self.pad] == MARK).all()) and bool((self.wide[:, self.N + self.pad:] == MARK).all())


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K", [
    (1, 8, 16), (1, 128, 128), (2, 136, 144), (1, 3200, 5120), (15, 264, 1040), (16, 120, 2048), (17, 1000, 272), (33, 128, 4096), (64, 520, 640),
    (63, 2048, 16), (48, 20000, 128), (65, 256, 256), (66, 8, 528), (127, 392, 1024), (128, 256, 128), (129, 24, 144), (255, 512, 384), (256, 264, 512),
    (257, 128, 1280), (300, 5120, 112), (511, 640, 2064), (700, 1400, 400), (1500, 2056, 96)])
def test_one_matrix(symm, M, N, K, f32):
    c = Case(M, N, K, f32=f32)
    c.run(symm)
    c.check(symm)


@pytest.mark.parametrize("tiles", [36, 37, 46, 47, 76, 77])
@pytest.mark.parametrize("K", [512, 1040])
def test_weight_tiles_around_the_clusters_that_run_at_once(symm, tiles, K):
    c = Case(19, 128 * tiles - 8, K)
    c.run(symm)
    c.check(symm)


@pytest.mark.parametrize("M,N,K", [(5, 72, 144), (40, 256, 2048), (300, 264, 272)])
@pytest.mark.parametrize("f32", [False, True])
def test_strided_rows(symm, M, N, K, f32):
    c = Case(M, N, K, f32=f32, lead=1)
    c.run(symm)
    c.check(symm)


SHARES = {
    "one row": [0, 0, 1, 0], "none": [0, 0, 0], "all to one": [0, 300, 0, 0, 0], "few each": [3, 1, 0, 17, 2, 0, 0, 16], "ragged": [0, 65, 1, 129, 257, 16, 0, 300, 64],
    "wide": [256, 255, 257, 512, 1], "many": [i % 7 for i in range(256)], "narrow tiles": [64, 65, 63, 128, 1, 0, 20],
}


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("name", SHARES)
@pytest.mark.parametrize("N,K,first,spare", [(264, 272, 0, 0), (128, 1152, 5, 70)])
def test_experts(symm, name, N, K, first, spare, f32):
    ends = [first]
    for n in SHARES[name]:
        ends.append(ends[-1] + n)
    c = Case(ends[-1] + spare, N, K, E=len(ends) - 1, f32=f32)
    c.run(symm, base=torch.tensor(ends, dtype=torch.int64, device="cuda"))
    c.check(symm, ends)


# shapes of narrow tiles with more than 64 rows
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K,lead", [(100, 7160, 8208, 0), (65, 7168, 8192, 1), (128, 7176, 8064, 0), (333, 5112, 3216, 1)])
def test_tiles_of_more_than_64_rows(symm, M, N, K, lead, f32):
    c = Case(M, N, K, f32=f32, lead=lead)
    c.run(symm)
    c.check(symm)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rows", [[100, 128, 65, 0, 200, 129, 64, 114], [1, 17, 33, 49, 80, 81, 112, 427], [800, 0, 0, 0, 0, 0, 0, 0], [96] * 8])
def test_experts_with_tiles_of_more_than_64_rows(symm, rows, f32):
    ends = [0]
    for n in rows:
        ends.append(ends[-1] + n)
    c = Case(800, 2056, 4112, E=8, f32=f32)
    c.run(symm, base=torch.tensor(ends, dtype=torch.int64, device="cuda"))
    c.check(symm, ends)


# shapes that two pairs of CTAs share a tile of: 21 blocks of K, rows and columns that end inside a tile
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,lead", [(250, 5112, 0), (100, 8072, 1), (500, 4392, 1), (129, 9216, 0)])
def test_tiles_with_halves_of_k(symm, M, N, lead, f32):
    c = Case(M, N, 2576, f32=f32, lead=lead)
    c.run(symm)
    c.check(symm)
    before = c.out.clone()
    c.run(symm)
    assert torch.equal(c.out, before)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N", [(600, 7160), (300, 10008)])
def test_whole_rounds_and_halves_of_k(symm, M, N, f32):
    c = Case(M, N, 4112, f32=f32, lead=1)
    c.run(symm)
    c.check(symm)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rows", [[200, 0, 256], [0, 456, 0], [455, 0, 1], [70, 130, 256], [0, 0, 7]])
def test_experts_with_halves_of_k(symm, rows, f32):
    ends = [0]
    for n in rows:
        ends.append(ends[-1] + n)
    c = Case(456, 2304, 2576, E=3, f32=f32)
    c.run(symm, base=torch.tensor(ends, dtype=torch.int64, device="cuda"))
    c.check(symm, ends)


def test_offsets_that_go_back_with_halves_of_k(symm):
    """More tiles than the rows can have: reported, the call ends, and the next one is right."""
    c = Case(1000, 768, 5136, E=8)
    c.run(symm, base=torch.tensor([0, 1000] * 4 + [0], dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
    assert symm.status()["code"] != 0
    ends = [0, 100, 300, 400, 500, 600, 800, 801, 1000]
    c.run(symm, base=torch.tensor(ends, dtype=torch.int64, device="cuda"))
    c.check(symm, ends)


def test_most_experts(symm):
    ends = [0]
    for e in range(4096):
        ends.append(ends[-1] + (e % 5 == 0))
    c = Case(ends[-1], 8, 16, E=4096)
    c.run(symm, base=torch.tensor(ends, device="cuda"))
    c.check(symm, ends)


@pytest.mark.parametrize("M", [20, 300])
def test_integers_are_exact(symm, M):
    """Small integers and powers of two: every sum is exact, and so is the float32 output."""
    g = generator(M)
    c = Case(M, 264, 1168, f32=True)
    c.a.copy_(torch.randint(-8, 9, c.a.shape, generator=g, device="cuda").float().to(E4M3))
    c.b.copy_(torch.randint(-8, 9, c.b.shape, generator=g, device="cuda").float().to(E4M3))
    c.a_scale.copy_(torch.exp2(torch.randint(-1, 2, c.a_scale.shape, generator=g, device="cuda").float()))
    c.b_scale.copy_(torch.exp2(torch.randint(-1, 2, c.b_scale.shape, generator=g, device="cuda").float()))
    c.run(symm)
    want, _ = product(c.a, c.a_scale, c.b, c.b_scale)
    assert torch.equal(c.out.double(), want)


@pytest.mark.parametrize("M,K", [(30, 2048), (300, 272)])
def test_a_row_that_is_not_finite_stays_alone(symm, M, K):
    c = Case(M, 256, K)
    c.run(symm)
    clean = c.out.clone()
    c.a.view(torch.uint8)[7, 3] = 0x7F           # NaN
    c.a_scale[11, 0] = float("inf")
    c.a_scale[M - 1, blocks(K) - 1] = float("nan")
    c.run(symm)
    good = [m for m in range(M) if m not in (7, 11, M - 1)]
    assert torch.equal(c.out[good], clean[good])
    assert bool(c.out[7].isnan().all()) and not bool(c.out[11].isfinite().any()) and bool(c.out[M - 1].isnan().all())
    # and a row of weights one column
    c = Case(M, 256, K)
    c.b.view(torch.uint8)[130, 1] = 0xFF
    c.run(symm)
    good = [n for n in range(256) if n != 130]
    assert torch.equal(c.out[:, good], clean[:, good]) and bool(c.out[:, 130].isnan().all())


def test_rows_behind_an_expert_never_reach_it(symm):
    """The tiles read past an expert's last row; what lies there is another expert's, or NaN."""
    ends = [0, 20, 20, 90]
    c = Case(100, 264, 400, E=3)
    c.a.view(torch.uint8)[90:] = 0x7F
    c.a_scale[90:] = float("nan")
    c.run(symm, base=torch.tensor(ends, device="cuda"))
    c.check(symm, ends)


@pytest.mark.parametrize("bad,index", [([0, 10, 5, 40], 1), ([-1, 10, 20, 40], 0), ([0, 10, 20, 41], 2), ([0, 2 ** 40, 20, 30], 0), ([0, 5, 2 ** 62, 7], 1),
                                       ([-2 ** 63, 2 ** 63 - 1, -5, 40], 0)])
def test_offsets_out_of_order_or_range_are_reported(symm, bad, index):
    c = Case(40, 136, 144, E=3)
    c.run(symm, base=torch.tensor(bad, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
    st = symm.status()
    assert st["code"] == tdg.TDG_ERR_DEVICE and st["where"] == "cu"
    assert st["index"] in (index, index + 1, 2)
    # an expert whose own offsets are good and whose rows no other has is computed
    if bad[1] == 10 and bad[0] == -1:
        want, mag = product(c.a[20:40], c.a_scale[20:40], c.b[2], c.b_scale[2])
        check_product(c.out[20:40], want, mag, 144)
        assert bool((c.out[:10] == MARK).all())


def test_same_bits_again_and_in_a_graph(symm):
    for M, E in ((1, None), (50, None), (400, None), (60, 4)):
        c = Case(M, 392, 2048, E=E, f32=True)
        ends = None if E is None else torch.tensor([0, 3, 3, 40, 60], device="cuda")
        first = c.run(symm, ends).clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            c.run(symm, ends)
            with torch.cuda.graph(graph, stream=side):
                c.run(symm, ends)
                c.run(symm, ends)
        torch.cuda.synchronize()
        c.out.fill_(MARK)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, first)
        if E is not None:                        # the offsets are read at each replay
            ends.copy_(torch.tensor([0, 0, 25, 25, 50]))
            c.out.fill_(MARK)
            graph.replay()
            c.check(symm, [0, 0, 25, 25, 50])
        else:
            new = Case(M, 392, 2048, f32=True, seed=1)
            c.a.copy_(new.a)
            graph.replay()
            c.check(symm)


def test_halves_of_k_in_a_graph_and_on_streams_at_once(symm):
    cases = [Case(m, n, 4112, seed=i) for i, (m, n) in enumerate(((250, 5112), (600, 7160), (1, 4096), (500, 4096)))]
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


def test_two_streams_at_once(symm):
    cases = [Case(m, 520, 1024, seed=s) for s, m in enumerate((3, 200, 40, 600))]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cases, streams):
            c.run(symm, stream=s)
    torch.cuda.synchronize()
    for c in cases:
        c.check(symm)


def test_far_offsets(symm):
    """Weights and rows whose offsets pass 32 bits."""
    g = generator(1)
    E, N, K = 5, 1024, 1 << 20                   # 5 GiB of codes
    c = Case(0, 8, 16)
    c.M, c.N, c.K, c.E, c.pad = 40, N, K, E, 0
    c.a, c.a_scale = random_codes(g, 40, K), random_scales(g, 40, blocks(K))
    c.b = torch.empty(E, N, K, dtype=E4M3, device="cuda")
    c.b.view(torch.uint8).random_(0, 0x70, generator=g)
    c.b_scale = random_scales(g, E, blocks(N), blocks(K))
    c.wide = torch.full((42, N), MARK, dtype=torch.bfloat16, device="cuda")
    c.out = c.wide[1:-1]
    ends = [0, 1, 1, 2, 20, 40]
    c.run(symm, base=torch.tensor(ends, device="cuda"))
    assert symm.status()["code"] == 0
    for lo, hi, e in ((0, 1, 0), (2, 4, 3), (38, 40, 4)):
        for n in (0, N - 16):
            want, mag = product(c.a[lo:hi], c.a_scale[lo:hi], c.b[e, n:n + 16], c.b_scale[e, n // 128:n // 128 + 1])
            check_product(c.out[lo:hi, n:n + 16], want, mag, K)


@pytest.mark.parametrize("M,N,K", [(600000, 4096, 256), (3, 1 << 20, 48)])
def test_far_rows_and_columns(symm, M, N, K):
    """Outputs (and rows of a) whose offsets pass 32 bits; very many columns."""
    g = generator(2)
    a = torch.empty(M, K, dtype=E4M3, device="cuda")
    a.view(torch.uint8).random_(0, 0x70, generator=g)
    b, sa, sb = random_codes(g, N, K), random_scales(g, M, blocks(K)), random_scales(g, blocks(N), blocks(K))
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")     # (of 2 G finite outputs some are MARK)
    tdg.scaled_gemm(symm, a, sa, b, sb, out)
    assert symm.status()["code"] == 0
    for lo in (0, M // 2, max(0, M - 40)):
        for n in (0, N // 2 // 128 * 128, N - 128):
            want, mag = product(a[lo:lo + 40], sa[lo:lo + 40], b[n:n + 128], sb[n // 128:n // 128 + 1])
            check_product(out[lo:lo + 40, n:n + 128], want, mag, K)
    assert not bool(out[:, ::1031].isnan().any())


def test_refusals(symm):
    c = Case(24, 136, 256, f32=False)
    a, sa, b, sb, out = c.a, c.a_scale, c.b, c.b_scale, c.out.contiguous()
    base = torch.tensor([0, 24], device="cuda")
    for args, match in [((a.float(), sa, b, sb, out), "float8"), ((a, sa.double(), b, sb, out), "float32"), ((a, sa, b.view(torch.uint8), sb, out), "float8"),
                        ((a, sa, b, sb, out.half()), "bfloat16"), ((a[:23], sa, b, sb, out), "fit"), ((a, sa[:, :1], b, sb, out), "fit"),
                        ((a, sa, b[:128], sb, out), "fit"), ((a, sa, b, sb[:1], out), "fit"), ((a, sa, b[None], sb[None], out), "fit"),
                        ((a, sa, b, sb, out.t()), "contiguous"), ((a, sa, b, sb, out.cpu()), "heap"), ((a, sa, b.cpu(), sb, out), "CUDA")]:
        with pytest.raises((TypeError, ValueError), match=match):
            tdg.scaled_gemm(symm, *args)
    with pytest.raises(ValueError, match="fit"):
        tdg.scaled_gemm(symm, a, sa, b, sb, out, base=base)
    for bad, kind in ((base.int(), TypeError), (base[:1], ValueError), (base.cpu(), ValueError)):
        with pytest.raises(kind):
            tdg.scaled_gemm(symm, a, sa, b[None], sb[None], out, base=bad)

    def rc(**kw):
        args = tdg.ScaledGemmArgs(M=24, N=136, K=256, E=1, a=a.data_ptr(), a_stride=256, a_scale=sa.data_ptr(), a_scale_stride=2, b=b.data_ptr(),
                                  b_scale=sb.data_ptr(), out=out.data_ptr(), out_stride=136)
        for key, v in kw.items():
            setattr(args, key, v)
        return tdg.lib().tdg_scaled_gemm(symm.h, ctypes.byref(args), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc() == tdg.TDG_OK and rc(M=0, a=None) == tdg.TDG_OK
    for kw in (dict(M=-1), dict(M=1 << 31), dict(N=0), dict(N=132), dict(N=1 << 24), dict(K=0), dict(K=8), dict(K=250), dict(K=1 << 24), dict(E=0), dict(E=2),
               dict(E=4097, base=base.data_ptr()), dict(a=None), dict(b=None), dict(out=None), dict(a_scale=None), dict(b_scale=None),
               dict(a=a.data_ptr() + 8), dict(b=b.data_ptr() + 8), dict(out=out.data_ptr() + 8), dict(a_scale=sa.data_ptr() + 2), dict(b_scale=sb.data_ptr() + 1),
               dict(base=base.data_ptr() + 4), dict(a_stride=240), dict(a_stride=264), dict(a_scale_stride=1), dict(out_stride=128), dict(out_stride=140),
               dict(out_f32=2), dict(out=a.data_ptr()), dict(out=b.data_ptr() + 256), dict(a_scale=out.data_ptr()), dict(b_scale=out.data_ptr() + 16),
               dict(base=out.data_ptr()), dict(N=8388608, E=4096, base=base.data_ptr())):
        assert rc(**kw) == tdg.TDG_ERR_INVALID, kw
    torch.cuda.synchronize()
    assert symm.status()["code"] == 0
