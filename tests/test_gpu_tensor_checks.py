"""The binding's native tensor checks give what the Python ones give, value or error."""
import pytest
import torch

from tile_centric_comm_gb300 import tdg

pytestmark = pytest.mark.gpu


def _both(native, checked, *args):
    def outcome(f):
        try:
            return f(*args)
        except (TypeError, ValueError) as e:
            return type(e), str(e)
    got, want = outcome(native), outcome(checked)
    assert got == want
    return got


def test_same_outcomes():
    tdg._attn()
    dev = tdg.Symm(1, 1024, 16).device
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    x = torch.zeros(6, 12, 64, dtype=bf, device="cuda")
    wide = torch.zeros(6, 12 * 64 + 8, dtype=bf, device="cuda")[:, :768].unflatten(1, (12, 64))
    good = [x, wide, wide[:1], wide[:0], x[:, 2:5], x[:, :1], x[::2], x[1:], torch.nn.Parameter(x),
            torch.zeros(0, 12, 64, dtype=bf, device="cuda"), torch.zeros(6, 0, 64, dtype=bf, device="cuda"),
            x.expand(6, 12, 64), x[:1].expand(6, 12, 64)]
    bad = [x.float(), x.cpu(), x[0], x.transpose(0, 1), x[:, ::2], x[:, :, ::2], x[:, :, :1], None, 3, x.unsqueeze(0), [1.0]]
    for t in good:
        assert isinstance(_both(tdg._rows, tdg._checked_rows, t, "x", dev)[0], int)
    for t in bad:
        assert isinstance(_both(tdg._rows, tdg._checked_rows, t, "x", dev)[0], type)

    m = torch.zeros(5, 9, dtype=i32, device="cuda")
    for t in [m, m[:, :4], m[:1], m[:, :1], m[:0], m[::2], m[:1, 3:]]:
        assert isinstance(_both(tdg._table, tdg._checked_table, t, "m", dev)[0], int)
    for t in [m.long(), m.cpu(), m[0], m.t(), m[:, ::2], None]:
        assert isinstance(_both(tdg._table, tdg._checked_table, t, "m", dev)[0], type)

    for t, kind, n in [(m, i32, 45), (m[0], i32, 9), (m[1:3], i32, 0), (m[:0], i32, 0), (x.float(), f32, 1)]:
        assert isinstance(_both(tdg._flat, tdg._checked_flat, t, "t", kind, n, dev), int)
    for t, kind, n in [(m, i32, 46), (m, f32, 1), (m[:, :4], i32, 1), (m.cpu(), i32, 1), (None, i32, 0), ("m", i32, 0)]:
        assert isinstance(_both(tdg._flat, tdg._checked_flat, t, "t", kind, n, dev), tuple)


def test_scales_off_the_4_byte_grid_are_refused():
    import ctypes
    from attn_util import Cache
    c = Cache(1, [20], 2, 128, 16, True, seed=1)
    x = torch.zeros(1, 4, 128, dtype=torch.bfloat16, device="cuda")
    out, n = torch.empty_like(x), c.table.shape[1]
    scale = torch.full((8,), 0.5, device="cuda")

    def both(k_scale, v_scale):
        cache = tdg.PagedCacheDesc.from_buffer_copy(c.cache.desc)
        cache.k_scale, cache.v_scale = k_scale, v_scale
        where = dict(table=c.table_d.data_ptr(), table_entries=n, table_stride=n, lens=c.lens_d.data_ptr())
        rope = tdg.RopeAppendArgs(world=1, cache=cache, T=1, B=1, Hq=0, k=x.data_ptr(), v=x.data_ptr(), k_stride=512, v_stride=512, **where)
        decode = tdg.PagedDecodeArgs(world=1, cache=cache, B=1, Hq=4, q=x.data_ptr(), q_stride=512, out=out.data_ptr(), out_stride=512,
                                     part_off=c.part_off, **where)
        return (tdg.lib().tdg_rope_append(c.symm.h, ctypes.byref(rope), None), tdg.lib().tdg_paged_decode(c.symm.h, ctypes.byref(decode), None))

    p = scale.data_ptr()
    assert both(p + 4, p + 8) == (0, 0)
    for off in (1, 2, 3):
        assert both(p + off, p) == both(p, p + off) == (tdg.TDG_ERR_INVALID, tdg.TDG_ERR_INVALID)
    torch.cuda.synchronize()
    assert c.symm.status()["code"] == 0


def test_scales_on_another_device_are_refused():
    # the heap's handle says that it is on a second GPU; nothing is launched there
    from types import SimpleNamespace
    scale = torch.full((2,), 0.5, device="cuda")
    cache = tdg.PagedCache(4, 16, 2, 128, 0, 1 << 16, e4m3=True, k_scale=scale, v_scale=scale)
    heap = SimpleNamespace(device=torch.device("cuda", 1), world=1, h=None)
    x = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda")
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="v_scale: on cuda:0, the heap is on cuda:1"):
        tdg.rope_append(heap, cache, None, x, x, None, None, None, table, lens)
    with pytest.raises(ValueError, match="v_scale: on cuda:0, the heap is on cuda:1"):
        tdg.paged_decode(heap, cache, x, x.clone(), table, lens, 0)
    with pytest.raises(ValueError, match="v_scale"):
        tdg.PagedCache(4, 16, 2, 128, 0, 1 << 16, e4m3=True, k_scale=scale, v_scale=scale.cpu())
    with pytest.raises(TypeError, match="torch.Tensor"):
        tdg.PagedCache(4, 16, 2, 128, 0, 1 << 16, e4m3=True, k_scale=[0.5, 0.5], v_scale=scale)
    # a cache without scales is of no device
    with pytest.raises(ValueError, match="k: on cuda:0, the heap is on cuda:1"):
        tdg.rope_append(heap, tdg.PagedCache(4, 16, 2, 128, 0, 1 << 16), None, x, x, None, None, None, table, lens)
