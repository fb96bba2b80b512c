"""Conversions into 8 bits with a scale for each block, and the 8-bit dispatch,
against the definition in 64 bits."""
import ctypes

import pytest
import torch

from expert_util import E4M3, LEAST, blocks, generator, quantised, values
from tile_centric_comm_gb300 import tdg

pytestmark = pytest.mark.gpu
POISON = 0x5A


@pytest.fixture(scope="module")
def symm():
    return tdg.Symm(1, 1024, 16)


def _rows(g, n, width, lead=0):
    """Rows of a buffer `lead` columns wider, channels of unlike size."""
    size = torch.exp2(torch.randint(-6, 7, (width + lead,), generator=g, device="cuda").float())
    return (torch.randn(n, width + lead, generator=g, device="cuda") * size).to(torch.bfloat16)[:, lead:]


def _outputs(n, K, lead=0):
    codes = torch.full((n, K + lead), POISON, dtype=torch.uint8, device="cuda").view(E4M3)
    scale = torch.full((n, blocks(K) + lead // 16), -1.0, device="cuda")
    return codes, scale


@pytest.mark.parametrize("n,K,lead", [(1, 16, 0), (1, 128, 16), (3, 144, 0), (7, 112, 32), (37, 5120, 0), (129, 272, 16), (513, 2048, 0),
                                      (2500, 1040, 0), (20000, 128, 0)])
def test_rows(symm, n, K, lead):
    x = _rows(generator(n + K), n, K, lead)
    codes, scale = _outputs(n, K, lead)
    tdg.quantise_rows(symm, x, codes[:, lead:], scale[:, :blocks(K)])
    want, s = quantised(x)
    assert torch.equal(scale[:, :blocks(K)], s)
    assert torch.equal(codes.view(torch.uint8)[:, lead:], want)
    # nothing beside the rows is written
    assert bool((codes.view(torch.uint8)[:, :lead] == POISON).all()) and bool((scale[:, blocks(K):] == -1).all())
    assert symm.status()["code"] == 0


def test_rows_values_where_it_can_go_wrong(symm):
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(12, 128, dtype=torch.bfloat16, device="cuda")
    x[1] = -0.0
    x[2, 5] = 2.0 ** -133                        # a subnormal, alone
    x[3] = torch.arange(128, device="cuda") * 1e-38
    x[4] = (torch.arange(128, device="cuda") - 64).float() * 5e36   # near the largest
    x[5, ::3], x[5, 1] = nan, 3.0
    x[6] = nan
    x[7, 9], x[7, 10], x[7, 11] = inf, 2.0, nan
    x[8, :], x[8, 0] = 1.0, 448.0
    # ties: scale 1, quotients halfway between two codes, both ways
    x[9, :] = torch.arange(128, device="cuda") * 0.0625
    x[9, 0] = 448
    x[10, :] = 2.0 ** -10 * torch.arange(128, device="cuda")        # halfway below the smallest codes
    x[10, 0] = -448
    x[11, :] = -torch.arange(128, device="cuda").float()
    codes, scale = _outputs(12, 128)
    tdg.quantise_rows(symm, x, codes, scale)
    want, s = quantised(x)
    assert torch.equal(scale, s) and scale[0, 0] == LEAST and scale[7, 0] == inf
    nans = values(codes, torch.ones_like(scale)).isnan()
    assert torch.equal(nans, want.view(E4M3).double().isnan())
    assert torch.equal(codes.view(torch.uint8)[~nans], want[~nans])
    assert nans[5].sum() == 43 and nans[6].all() and nans[7].sum() == 2


def test_every_bf16_value_against_many_scales(symm):
    """Quotients of all finite bf16 values up to the block's largest: bit for bit."""
    pos = torch.arange(0, 0x7F80, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    g = generator(3)
    for e in (-120, -100, -30, -3, 0, 5, 60, 119):
        top = ((1 + torch.rand(256, generator=g, device="cuda")) * 2.0 ** e).to(torch.bfloat16)
        near = pos[(pos.float() <= 2.0 ** e) & (pos.float() > 2.0 ** max(e - 24, -133))]
        x = near[torch.randint(0, near.numel(), (256, 128), generator=g, device="cuda")]
        x[:, 7] = top
        codes, scale = _outputs(256, 128)
        tdg.quantise_rows(symm, x, codes, scale)
        want, s = quantised(x)
        assert torch.equal(scale, s), e
        assert torch.equal(codes.view(torch.uint8), want), e


@pytest.mark.parametrize("n,K,lead", [(1, 16, 0), (5, 240, 16), (40, 2048, 0), (700, 176, 0), (9000, 256, 0)])
def test_gated(symm, n, K, lead):
    g = generator(n)
    x = (_rows(g, n, 2 * K, lead).float() * 0.1).to(torch.bfloat16)
    wide = torch.zeros(n, 2 * K + lead, dtype=torch.bfloat16, device="cuda")
    wide[:, lead:] = x
    x = wide[:, lead:]
    codes, scale = _outputs(n, K)
    tdg.quantise_rows(symm, x, codes, scale, gated=True)
    gate, up = x.double()[:, :K], x.double()[:, K:]
    v = gate * torch.sigmoid(gate) * up
    _, s = quantised(v)
    off = 2.0 ** -20 + 2.0 ** -23 * (-gate).clamp(min=0)        # relative, of each value
    _, most = quantised(v.abs() * off)                          # so much a block's largest value moves at most
    assert bool(((scale.double() - s.double()).abs() <= most.double() + 2.0 ** -24 * s.double()).all())
    q = v / s.double().repeat_interleave(128, 1)[:, :K]
    moved = off + (most.double() / s.double()).repeat_interleave(128, 1)[:, :K] + 2.0 ** -23
    err = (codes.double() - q).abs()
    assert bool((err <= torch.maximum(2.0 ** -4 * q.abs(), torch.full_like(q, 2.0 ** -10)) + moved * q.abs()).all())


def test_gated_far_gates(symm):
    x = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    x[0, :16], x[0, 16:] = -1e4, 1.0            # closed: no infinity on the way
    x[1, :16], x[1, 16:] = 300.0, -2.0
    x[2, :16] = torch.arange(-104, -88, device="cuda")
    x[2, 16:] = 1e30
    x[3, 0] = float("nan")
    codes, scale = _outputs(4, 16)
    tdg.quantise_rows(symm, x, codes, scale, gated=True)
    assert bool((codes[0].double() == 0).all()) and scale[0, 0] == LEAST
    assert bool((codes[1].double() == -448).all())
    assert bool(scale[2].isfinite().all()) and bool(codes[2].float().isfinite().all())
    assert codes[3].double().isnan().sum() == 1


@pytest.mark.parametrize("E,N,K", [(None, 1, 16), (None, 128, 128), (1, 130, 272), (3, 257, 144), (2, 96, 1040), (5, 384, 640)])
def test_blocks(symm, E, N, K):
    g = generator(N)
    shape = (N, K) if E is None else (E, N, K)
    x = (torch.randn(*shape, generator=g, device="cuda") * torch.exp2(torch.randint(-6, 7, (K,), generator=g, device="cuda").float())).to(torch.bfloat16)
    codes = torch.full(shape, POISON, dtype=torch.uint8, device="cuda").view(E4M3)
    scale = torch.empty(*shape[:-2], blocks(N), blocks(K), device="cuda")
    tdg.quantise_blocks(symm, x, codes, scale)
    for e in range(E or 1):
        want, s = quantised(x if E is None else x[e], rows=128)
        assert torch.equal(scale if E is None else scale[e], s)
        assert torch.equal((codes if E is None else codes[e]).view(torch.uint8), want)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("n", [0, 1, 77, 200])
def test_count_leaves_the_other_rows_alone(symm, n, gated):
    x = _rows(generator(n), 200, 512)
    codes, scale = _outputs(200, 256 if gated else 512)
    count = torch.tensor([9, n, 9], dtype=torch.int64, device="cuda")[1:]
    tdg.quantise_rows(symm, x, codes, scale, gated=gated, count=count)
    full, fscale = _outputs(200, codes.shape[1])
    tdg.quantise_rows(symm, x, full, fscale, gated=gated)
    assert torch.equal(codes[:n].view(torch.uint8), full[:n].view(torch.uint8)) and torch.equal(scale[:n], fscale[:n])
    assert bool((codes[n:].view(torch.uint8) == POISON).all()) and bool((scale[n:] == -1).all())
    assert symm.status()["code"] == 0


@pytest.mark.parametrize("n,used", [(-1, 0), (-2 ** 62, 0), (201, 200), (2 ** 62, 200)])
def test_a_count_out_of_range_is_reported(symm, n, used):
    x = _rows(generator(5), 200, 128)
    codes, scale = _outputs(200, 128)
    tdg.quantise_rows(symm, x, codes, scale, count=torch.tensor([n], dtype=torch.int64, device="cuda"))
    st = symm.status()
    assert st["code"] == tdg.TDG_ERR_DEVICE and st["where"] == "cu"
    assert bool((scale[used:] == -1).all()) and bool((scale[:used] > 0).all())


def test_far_rows(symm):
    """Offsets past 32 bits: rows of 5 GB."""
    n, K = 300001, 8192
    x = torch.empty(n, K, dtype=torch.bfloat16, device="cuda").normal_(generator=generator(4))
    codes, scale = torch.empty(n, K, dtype=E4M3, device="cuda"), torch.empty(n, blocks(K), device="cuda")
    tdg.quantise_rows(symm, x, codes, scale)
    for lo in (0, 131071, 262143, n - 50):
        want, s = quantised(x[lo:lo + 50])
        assert torch.equal(scale[lo:lo + 50], s) and torch.equal(codes[lo:lo + 50].view(torch.uint8), want)
    tdg.quantise_blocks(symm, x[None], codes[None], scale[None, :blocks(n)].contiguous())
    want, _ = quantised(x[262144:262272], rows=128)
    assert torch.equal(codes[262144:262272].view(torch.uint8), want)


def test_captured_and_replayed_on_another_stream(symm):
    x = _rows(generator(6), 64, 256)
    codes, scale = _outputs(64, 256)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        tdg.quantise_rows(symm, x, codes, scale)
        with torch.cuda.graph(graph, stream=side):
            tdg.quantise_rows(symm, x, codes, scale)
    for seed in (7, 8):
        x.copy_(_rows(generator(seed), 64, 256))
        graph.replay()
        want, s = quantised(x)
        assert torch.equal(codes.view(torch.uint8), want) and torch.equal(scale, s)


def test_refusals(symm):
    bf, f32 = torch.bfloat16, torch.float32
    x = torch.zeros(8, 256, dtype=bf, device="cuda")
    codes, scale = _outputs(8, 256)
    for bad, match in [((x.float(), codes, scale), "bfloat16"), ((x, codes.view(torch.uint8), scale), "float8"), ((x[:7], codes, scale), "fit"),
                       ((x, codes[:, :128], scale), "fit"), ((x, codes, scale[:, :1]), "fit"), ((x.t(), codes, scale), "contiguous"),
                       ((x.cpu(), codes, scale), "heap"), ((x, codes, scale.half()), "float32"), ((x[0], codes, scale), "rows, columns")]:
        with pytest.raises((TypeError, ValueError), match=match):
            tdg.quantise_rows(symm, *bad)
    with pytest.raises(ValueError, match="fit"):
        tdg.quantise_rows(symm, x, codes, scale, gated=True)
    with pytest.raises(TypeError, match="int64"):
        tdg.quantise_rows(symm, x, codes, scale, count=torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="fit"):
        tdg.quantise_blocks(symm, x, codes, scale)
    with pytest.raises(ValueError, match="expected"):
        tdg.quantise_blocks(symm, x[0], codes, scale)

    def rc(**kw):
        a = tdg.QuantiseArgs(kind=0, rows=8, K=256, E=1, x=x.data_ptr(), x_stride=256, codes=codes.data_ptr(), codes_stride=256,
                             scale=scale.data_ptr(), scale_stride=2)
        for key, v in kw.items():
            setattr(a, key, v)
        return tdg.lib().tdg_quantise(symm.h, ctypes.byref(a), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc() == tdg.TDG_OK and rc(rows=0) == tdg.TDG_OK and rc(kind=2, E=0) == tdg.TDG_OK
    for kw in (dict(kind=3), dict(kind=-1), dict(rows=-1), dict(K=0), dict(K=8), dict(K=248), dict(K=1 << 30), dict(E=2), dict(x=None), dict(codes=None),
               dict(scale=None), dict(x=x.data_ptr() + 8), dict(codes=codes.data_ptr() + 8), dict(scale=scale.data_ptr() + 2), dict(x_stride=255),
               dict(x_stride=252 + 8), dict(x_stride=248), dict(codes_stride=264), dict(codes_stride=240), dict(scale_stride=1), dict(kind=1),
               dict(kind=2, scale_stride=3), dict(kind=2, count=scale.data_ptr()), dict(count=scale.data_ptr() + 4), dict(codes=x.data_ptr()),
               dict(scale=x.data_ptr() + 16), dict(scale=codes.data_ptr() + 2040), dict(count=codes.data_ptr()), dict(rows=1 << 31), dict(kind=2, rows=1 << 20, E=1 << 20)):
        assert rc(**kw) == tdg.TDG_ERR_INVALID, kw
    torch.cuda.synchronize()
    assert symm.status()["code"] == 0


# ------------------------------------------------------- the 8-bit dispatch
def _dispatch(W, T, H, E, k, seed):
    g = generator(seed)
    symm = tdg.Symm(W, T * H * 2 + 1024, 16)
    for r in range(W):
        symm.view(r, 1024, (T, H), torch.bfloat16).copy_(_rows(g, T, H))
    topk = torch.rand(W, T, E, generator=g, device="cuda").topk(k, -1).indices
    slot = torch.empty(W * T * k, dtype=torch.int64, device="cuda")
    slot[torch.sort(topk.flatten(), stable=True).indices] = torch.arange(W * T * k, device="cuda")
    return symm, slot


@pytest.mark.parametrize("W,T,H,E,k", [(1, 1, 16, 4, 1), (2, 3, 144, 8, 8), (8, 16, 7168, 64, 8), (4, 129, 272, 32, 32), (3, 1000, 1024, 16, 2)])
def test_dispatch(W, T, H, E, k):
    symm, slot = _dispatch(W, T, H, E, k, seed=T)
    codes, scale = _outputs(W * T * k, H)
    tdg.moe_dispatch_e4m3(symm, T, H, k, 1024, slot, codes, scale)
    assert symm.status()["code"] == 0
    tok = torch.empty(W * T * k, dtype=torch.int64, device="cuda")
    tok[slot] = torch.arange(W * T * k, device="cuda") // k
    x = torch.cat([symm.view(r, 1024, (T, H), torch.bfloat16) for r in range(W)])
    want, s = quantised(x)
    assert torch.equal(scale, s[tok]) and torch.equal(codes.view(torch.uint8), want[tok])


def test_dispatch_of_refused_choices():
    symm, slot = _dispatch(2, 40, 128, 8, 4, seed=1)
    good = slot.clone()
    slot[13] = -1                                # as the routing writes for a bad expert id
    codes, scale = _outputs(320, 128)
    tdg.moe_dispatch_e4m3(symm, 40, 128, 4, 1024, slot, codes, scale)
    assert symm.status()["code"] == 0
    assert bool((scale[good[13]] == -1).all()) and int((scale == -1).sum()) == 1
    for bad in (320, -2, 2 ** 40, -2 ** 63):
        slot[13] = bad
        codes, scale = _outputs(320, 128)
        tdg.moe_dispatch_e4m3(symm, 40, 128, 4, 1024, slot, codes, scale)
        st = symm.status()
        assert st["code"] == tdg.TDG_ERR_DEVICE and st["where"] == "slot" and st["index"] == 13
        assert bool((scale[good[13]] == -1).all()) and int((scale == -1).sum()) == 1


def test_dispatch_refusals():
    symm, slot = _dispatch(2, 8, 128, 8, 2, seed=2)
    codes, scale = _outputs(32, 128)
    with pytest.raises(ValueError, match="needs"):
        tdg.moe_dispatch_e4m3(symm, 8, 128, 2, 1024, slot[:31], codes, scale)
    with pytest.raises(ValueError, match="needs"):
        tdg.moe_dispatch_e4m3(symm, 8, 128, 2, 1024, slot, codes[:31], scale)
    with pytest.raises(TypeError, match="int64"):
        tdg.moe_dispatch_e4m3(symm, 8, 128, 2, 1024, slot.int(), codes, scale)

    def rc(**kw):
        a = tdg.MoeDispatchE4m3Args(world=2, k=2, T=8, H=128, x_off=1024, slot=slot.data_ptr(), codes=codes.data_ptr(), scale=scale.data_ptr())
        for key, v in kw.items():
            setattr(a, key, v)
        return tdg.lib().tdg_moe_dispatch_e4m3(symm.h, ctypes.byref(a), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    region = symm.region_ptr(1)
    assert rc() == tdg.TDG_OK and rc(T=0) == tdg.TDG_OK
    for kw in (dict(world=1), dict(k=0), dict(k=33), dict(T=-1), dict(H=0), dict(H=120), dict(slot=None), dict(codes=None), dict(scale=None),
               dict(slot=slot.data_ptr() + 4), dict(codes=codes.data_ptr() + 8), dict(scale=scale.data_ptr() + 1), dict(x_off=1032),
               dict(codes=region + 1024), dict(scale=region + 1024), dict(codes=slot.data_ptr()), dict(scale=codes.data_ptr()), dict(T=1 << 30)):
        assert rc(**kw) == tdg.TDG_ERR_INVALID, kw
    for kw in (dict(x_off=2048), dict(x_off=(1 << 64) - 16), dict(T=64, k=1)):
        assert rc(**kw) == tdg.TDG_ERR_NOMEM, kw
    torch.cuda.synchronize()
    assert symm.status()["code"] == 0
