"""GPU parity of the rotary cache write against the oracle: turned queries and
keys, the pages written, and everything that must stay as it was."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from tile_centric_comm_gb300 import tdg
from attn_util import U, Cache, bits, bf16_f64, strided_rows, to_bits, to_dev_bf16

pytestmark = pytest.mark.gpu


def _table(g, P, rot):
    ang = g.uniform(0, 6.28, (P, rot // 2))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _near(got, want, mag, what):
    tol = U * np.abs(want) + 2.0 ** -22 * mag + 1e-38
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} outside the bound, first at {np.argwhere(bad)[0].tolist()}"


def _near8(got, want, mag, what):
    tol = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 + 2.0 ** -21 * mag
    want = np.clip(want, -448, 448)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} outside the bound, first at {np.argwhere(bad)[0].tolist()}"


class Case:
    def __init__(self, W, lens, new, Hq, Hkv, D, page, e4m3=False, rot=None, axes=1, inter=False, seed=0,
                 one=False, tail=0):
        self.c = Cache(W, lens, Hkv, D, page, e4m3, seed=seed, extra_entries=2)
        g = self.g = np.random.default_rng(seed + 100)
        self.new, self.one = list(new), one
        T = self.T = len(lens) if one else sum(new) + tail      # `tail` rows of no sequence
        self.rot = D if rot is None else rot
        self.q, self.k, self.v = (bits(g.standard_normal((T, n, D)) * 3) for n in (Hq, Hkv, Hkv))
        self.cos_sin = _table(g, 37, self.rot) if self.rot else None
        self.pos = g.integers(0, 37, (axes, T)).astype(np.int32)
        half = self.rot // 2
        self.sections = None if axes == 1 else [half - half // 3, half // 3] if axes == 2 else [3, half - 7, 4]
        self.inter = inter
        self.cu = None if one else np.concatenate([[0], np.cumsum(new)]).astype(np.int32)

    def run(self, in_place=False, k_out=True, stream=None):
        c = self.c
        buf, (q, k, v) = strided_rows([self.q, self.k, self.v])
        q_out = q if in_place else torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        ko = (k if in_place else torch.full(k.shape, float("nan"), dtype=torch.bfloat16, device="cuda")) if k_out else None
        tdg.rope_append(c.symm, c.cache, q, k, v, q_out,
                        torch.from_numpy(self.cos_sin).cuda() if self.rot else None,
                        torch.from_numpy(self.pos).cuda(), c.table_d, c.lens_d,
                        cu=None if self.one else torch.from_numpy(self.cu).cuda(), k_out=ko,
                        sections=self.sections, interleaved=self.inter, stream=stream)
        torch.cuda.synchronize()
        assert c.symm.status()["code"] == 0
        assert np.all(to_bits(buf[:, -1]) == 0x7FC1)              # the column beside them
        return bf16_f64(to_bits(q_out)), bf16_f64(to_bits(ko)) if k_out else None

    def check(self, q, k):
        c = self.c
        if self.rot:
            wq, mq = oracle.rope(self.q, self.cos_sin, self.pos, self.sections, self.inter)
            wk, mk = oracle.rope(self.k, self.cos_sin, self.pos, self.sections, self.inter)
        else:
            wq, wk = bf16_f64(self.q), bf16_f64(self.k)
            mq, mk = 0 * wq, 0 * wk
        _near(q, wq, mq, "q")
        if k is not None:
            _near(k, wk, mk, "k")
        got = c.download()
        rows = oracle.cache_rows(c.table, c.lens, c.page, self.cu)
        wv = bf16_f64(self.v)
        for i, (codes, before, want, mag) in enumerate(((got[0], c.k, wk, mk), (got[1], c.v, wv, 0 * wv))):
            now = np.stack([codes[p, :, s] for p, s in rows]) if rows else np.zeros((0, *codes.shape[1:2], codes.shape[3]))
            n = len(rows)
            if c.e4m3:
                s = (c.k_scale, c.v_scale)[i].astype(np.float64)[None, :, None]
                _near8(oracle.e4m3_to_f64(now), want[:n] / s, mag[:n] / s, "kv"[i] + " cache")
            elif n:
                _near(bf16_f64(now), want[:n], mag[:n], "kv"[i] + " cache")
            rest = codes.copy()
            for p, s in rows:
                rest[p, :, s] = before[p, :, s]
            assert np.array_equal(rest, before), "kv"[i] + ": a slot that belongs to no new row changed"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("axes,inter", [(1, False), (3, False), (2, True), (1, True)])
def test_prompts(D, e4m3, axes, inter):
    # rows of sequences that had tokens before, an empty one, one of a single row, rows of nobody at the end
    c = Case(3, [40, 7, 0, 65, 16], [33, 0, 0, 65, 1], 6, 2, D, 16, e4m3, axes=axes, inter=inter, seed=D + axes, tail=2)
    c.check(*c.run())


@pytest.mark.parametrize("Hq,Hkv,page,e4m3", [(1, 1, 16, False), (64, 8, 64, False), (40, 8, 16, True), (7, 7, 256, False),
                                              (33, 3, 32, True)])
def test_one_token_each(Hq, Hkv, page, e4m3):
    c = Case(2, [1, 16, 17, 300, 256], None or [1] * 5, Hq, Hkv, 128, page, e4m3, seed=Hq, one=True)
    c.check(*c.run())


@pytest.mark.parametrize("rot", [0, 16, 96])
def test_partial_rotation_in_place(rot):
    c = Case(2, [30, 5], [30, 2], 4, 2, 128, 16, rot=rot, seed=rot)
    c.check(*c.run(in_place=True))


def test_many_short_sequences_on_another_stream():
    g = np.random.default_rng(5)
    lens = g.integers(0, 9, 600).tolist()
    new = [int(g.integers(0, n + 1)) for n in lens]
    c = Case(4, lens, new, 2, 1, 64, 16, seed=5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.check(*c.run(k_out=False, stream=s))


def test_no_queries_and_no_cache():
    c = Case(2, [30, 5], [30, 2], 4, 2, 128, 16, seed=9)
    k = to_dev_bf16(c.k)
    tdg.rope_append(c.c.symm, c.c.cache, None, k, None, None, torch.from_numpy(c.cos_sin).cuda(),
                    torch.from_numpy(c.pos[0]).cuda(), None, None, k_out=k)
    torch.cuda.synchronize()
    want, mag = oracle.rope(c.k, c.cos_sin, c.pos)
    _near(bf16_f64(to_bits(k)), want, mag, "k")
    assert all(np.array_equal(a, b) for a, b in zip(c.c.download(), (c.c.k, c.c.v)))
    z = k[:0]
    tdg.rope_append(c.c.symm, c.c.cache, None, z, None, None, None, None, None, None, k_out=z)   # no rows


@pytest.mark.parametrize("what", ["pos", "page", "short", "long", "cu"])
def test_bad_indices_are_reported_and_skipped(what):
    c = Case(2, [20, 5], [4, 2], 4, 2, 64, 16, seed=11)
    code = "pos" if what == "pos" else "page"
    if what == "pos":
        c.pos[0, 2] = 37
    elif what == "page":
        c.c.table_d[0, 1] = 2 * c.c.pages
    elif what == "short":
        c.c.lens_d[1] = 1                 # two new rows in a sequence of one
    elif what == "long":
        c.c.lens_d[1] = 16 * c.c.table.shape[1] + 1
    else:
        c.cu[1] = 5                       # rows 5 .. 6 go backwards: the second sequence begins in the first
        c.cu[2] = 4
    k = to_dev_bf16(c.k)
    out = torch.full(k.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    tdg.rope_append(c.c.symm, c.c.cache, None, k, to_dev_bf16(c.v), None, torch.from_numpy(c.cos_sin).cuda(),
                    torch.from_numpy(c.pos).cuda(), c.c.table_d, c.c.lens_d, cu=torch.from_numpy(c.cu).cuda(), k_out=out)
    torch.cuda.synchronize()
    st = c.c.symm.status()
    if what != "cu":                      # offsets out of order: no access out of bounds is all that is promised
        assert st["code"] == tdg.TDG_ERR_DEVICE and st["where"] == code
    if what == "pos":
        got = to_bits(out)
        assert np.all(got[2] == to_bits(torch.full((1,), float("nan"), dtype=torch.bfloat16))[0]) and not np.any(np.isnan(bf16_f64(got[[0, 1, 3]])))
    assert c.c.symm.status()["code"] == 0


def test_refusals():
    c = Case(2, [30, 5], [30, 2], 4, 2, 128, 16, seed=13)
    k = to_dev_bf16(c.k)
    q = to_dev_bf16(c.q)
    out = torch.empty_like(q)
    cs, pos = torch.from_numpy(c.cos_sin).cuda(), torch.from_numpy(c.pos).cuda()
    cu = torch.from_numpy(c.cu).cuda()

    def rc(desc=(), **kw):
        a = tdg.RopeAppendArgs(world=2, cache=c.c.cache.desc, T=c.T, B=2, Hq=4, q=q.data_ptr(), k=k.data_ptr(),
                               v=k.data_ptr(), q_stride=512, k_stride=256, v_stride=256, q_out=out.data_ptr(),
                               q_out_stride=512, cos_sin=cs.data_ptr(), max_pos=37, rot_dim=128, axes=1,
                               pos=pos.data_ptr(), pos_stride=c.T, cu=cu.data_ptr(), table=c.c.table_d.data_ptr(),
                               table_entries=c.c.table.shape[1], table_stride=c.c.table.shape[1],
                               lens=c.c.lens_d.data_ptr())
        for key, v in kw.items():
            setattr(a, key, v)
        for key, v in desc:
            setattr(a.cache, key, v)
        return tdg.lib().tdg_rope_append(c.c.symm.h, ctypes.byref(a), None)

    assert rc() == tdg.TDG_OK
    bad, nomem = tdg.TDG_ERR_INVALID, tdg.TDG_ERR_NOMEM
    assert rc(world=1) == bad
    assert rc(T=-1) == bad
    assert rc(rot_dim=24) == bad and rc(rot_dim=144) == bad and rc(rot_dim=-16) == bad
    assert rc(axes=0) == bad and rc(axes=4) == bad
    assert rc(axes=2, sections=(ctypes.c_int * 3)(30, 33, 0)) == bad
    assert rc(axes=2, sections=(ctypes.c_int * 3)(-1, 65, 0)) == bad
    assert rc(max_pos=0) == bad and rc(cos_sin=None) == bad and rc(pos=None) == bad
    assert rc(q_stride=504) == bad and rc(k_stride=260) == bad
    assert rc(q=q.data_ptr() + 2) == bad and rc(k=None) == bad
    assert rc(q=None) == bad and rc(q_out=None) == bad and rc(Hq=0) == bad
    assert rc(q_out=k.data_ptr()) == bad                               # an output over another input
    assert rc(q_out=q.data_ptr() + 64) == bad                          # nearly in place
    assert rc(cu=None) == bad                                          # then T == B
    assert rc(lens=None) == bad and rc(v=None) == bad
    assert rc(table_stride=c.c.table.shape[1] - 1) == bad and rc(table_entries=1 << 28, table_stride=1 << 28) == bad
    assert rc(interleaved=2) == bad
    assert rc(desc=[("page_size", 48)]) == bad and rc(desc=[("D", 96)]) == bad and rc(desc=[("kv_type", 2)]) == bad
    assert rc(desc=[("k_off", 512)]) == bad and rc(desc=[("v_off", 0)]) == bad
    assert rc(desc=[("kv_type", 1)]) == bad                            # 8 bits without scales
    assert rc(desc=[("pages", 1 << 20)]) == nomem
    assert rc(desc=[("v_off", 1 << 30)]) == nomem
    with pytest.raises(TypeError, match="bfloat16"):
        tdg.rope_append(c.c.symm, c.c.cache, None, k.float(), None, None, None, None, None, None)
    with pytest.raises(ValueError, match="contiguous"):
        t = k.transpose(0, 1).contiguous().transpose(0, 1)
        tdg.rope_append(c.c.symm, c.c.cache, None, t, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="heads"):
        tdg.rope_append(c.c.symm, c.c.cache, None, k[:, :1], None, None, None, None, None, None)
    with pytest.raises(ValueError, match="scale"):
        tdg.PagedCache(1, 16, 1, 64, 0, 1024, e4m3=True)
    torch.cuda.synchronize()
    assert c.c.symm.status()["code"] == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_refuses_what_would_overwrite_its_inputs(e4m3):
    # nothing is launched: heap and outputs keep their bytes
    c = Case(2, [30, 5], [30, 2], 4, 2, 128, 16, e4m3, axes=2, seed=13)
    m = c.c.table.shape[1]
    q, k, v = to_dev_bf16(c.q), to_dev_bf16(c.k), to_dev_bf16(c.v)
    q_out, k_out = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    cs, pos, cu = (torch.from_numpy(x).cuda() for x in (c.cos_sin, c.pos, c.cu))
    base, region = c.c.symm.base, c.c.symm.region_bytes

    def rc(desc=(), **kw):
        a = tdg.RopeAppendArgs(world=2, cache=c.c.cache.desc, T=c.T, B=2, Hq=4, q=q.data_ptr(), k=k.data_ptr(),
                               v=v.data_ptr(), q_stride=512, k_stride=256, v_stride=256, q_out=q_out.data_ptr(),
                               k_out=k_out.data_ptr(), q_out_stride=512, k_out_stride=256, cos_sin=cs.data_ptr(),
                               max_pos=37, rot_dim=128, axes=2, sections=(ctypes.c_int * 3)(30, 34, 0),
                               pos=pos.data_ptr(), pos_stride=c.T, cu=cu.data_ptr(), table=c.c.table_d.data_ptr(),
                               table_entries=m, table_stride=m, lens=c.c.lens_d.data_ptr())
        for key, x in kw.items():
            setattr(a, key, x)
        for key, x in desc:
            setattr(a.cache, key, x)
        return tdg.lib().tdg_rope_append(c.c.symm.h, ctypes.byref(a), None)

    bad = tdg.TDG_ERR_INVALID
    before = c.c.symm.buf.clone()
    for out in (q_out, k_out):                                   # indices and tables under an output
        at = out.data_ptr()
        for name in ("cos_sin", "pos", "cu", "table", "lens"):
            assert rc(**{name: at}) == bad and rc(**{name: at + 4096}) == bad, name
        assert rc(pos=at - 4 * c.T - 4, pos_stride=c.T) == bad   # the second axis' positions
        if e4m3:
            assert rc(desc=[("k_scale", at)]) == bad and rc(desc=[("v_scale", at + 64)]) == bad
    for r in range(2):                                           # and in a pool of any rank
        for off in (0, c.c.v_off):
            at = base + r * region + off
            for name in ("cos_sin", "pos", "cu", "table", "lens", "q", "k", "v", "q_out", "k_out"):
                assert rc(**{name: at}) == bad, name
            if e4m3:
                assert rc(desc=[("v_scale", at)]) == bad
    torch.cuda.synchronize()
    assert torch.equal(c.c.symm.buf, before) and (q_out == 7).all() and (k_out == 7).all()
    # what is not read may lie anywhere
    assert rc(table=None, lens=k_out.data_ptr(), cu=q_out.data_ptr()) == 0
    assert rc(rot_dim=0, pos=q_out.data_ptr(), cos_sin=k_out.data_ptr()) == 0
    torch.cuda.synchronize()
    assert c.c.symm.status()["code"] == 0


@pytest.mark.parametrize("D", [64, 128])
def test_8_bit_codes_are_those_of_the_quotient(D):
    # every bf16 value over scales with ties, ordinary ones, and one whose reciprocal passes float32; values, and
    # keys that are not turned, are exact inputs, so the codes are determined
    scales = np.array([7 / 256, 0.03, 0.017, 1.0, 3.0, 2.0 ** -7, 2.5e-39, 1e30], np.float32)
    T, Hkv = 65536 // D, len(scales)
    c = Cache(1, [T], Hkv, D, 64, True, seed=1, fill=False)
    for s in c.scales:
        s.copy_(torch.from_numpy(scales))
    x = np.repeat(np.arange(65536, dtype=np.uint16).reshape(T, 1, D), Hkv, 1)
    xd = to_dev_bf16(x)
    tdg.rope_append(c.symm, c.cache, None, xd, xd.clone(), None, None, None, c.table_d, c.lens_d,
                    cu=torch.tensor([0, T], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert c.symm.status()["code"] == 0
    with np.errstate(all="ignore"):
        quotient = bf16_f64(x).astype(np.float32) / scales[None, :, None]
    want = oracle.f64_to_e4m3(quotient)
    nan = np.isnan(quotient)
    for pool, what in zip(c.download(), "kv"):
        got = oracle.gather_pages(pool, c.table[0], T)
        assert np.all((got[nan] & 0x7F) == 0x7F), what
        wrong = (got != want) & ~nan
        assert not wrong.any(), f"{what}: {wrong.sum(axis=(0, 2))} codes by scale, first {quotient[wrong][0]}: {got[wrong][0]:#x} for {want[wrong][0]:#x}"


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("cu", [[0, 5, 4], [0, -3, 6], [0, 100, 6], [6, 0, 6], [0, 2 ** 31 - 1, 6], [-2 ** 31, 2, 6], [3, 3, 2], [9, 9, 9]])
def test_offsets_out_of_order_write_into_listed_sequences_only(cu, e4m3):
    c = Case(2, [20, 9], [4, 2], 4, 2, 64, 16, e4m3, seed=12)
    q, k = to_dev_bf16(c.q), to_dev_bf16(c.k)
    q_out, k_out = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    tdg.rope_append(c.c.symm, c.c.cache, q, k, to_dev_bf16(c.v), q_out, torch.from_numpy(c.cos_sin).cuda(),
                    torch.from_numpy(c.pos).cuda(), c.c.table_d, c.c.lens_d, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), k_out=k_out)
    torch.cuda.synchronize()
    st = c.c.symm.status()
    assert st["code"] == 0 or (st["code"] == tdg.TDG_ERR_DEVICE and st["where"] == "page")     # a length below the new rows
    for got, x, what in ((q_out, c.q, "q"), (k_out, c.k, "k")):                                # the rows are turned all the same
        want, mag = oracle.rope(x, c.cos_sin, c.pos)
        _near(bf16_f64(to_bits(got)), want, mag, what)
    # where row t goes: the first sequence that ends behind it, counted back from that one's length
    stored = {}
    for t in range(c.T):
        b = sum(int(e) <= t for e in cu[1:])
        if b < 2 and cu[b] <= t < cu[b + 1] and c.c.lens[b] >= cu[b + 1] - cu[b]:
            j = c.c.lens[b] - (cu[b + 1] - t)
            assert 0 <= j < c.c.lens[b]
            stored[int(c.c.table[b, j // 16]), j % 16] = t
    for codes, before, x, scale in zip(c.c.download(), (c.c.k, c.c.v), (c.k, c.v), (c.c.k_scale, c.c.v_scale)):
        rest = codes.copy()
        for (page, slot), t in stored.items():
            want, mag = oracle.rope(x, c.cos_sin, c.pos) if x is c.k else (bf16_f64(x), 0 * bf16_f64(x))
            if e4m3:
                s = scale.astype(np.float64)[:, None]
                _near8(oracle.e4m3_to_f64(codes[page, :, slot]), want[t] / s, mag[t] / s, f"row {t}")
            else:
                _near(bf16_f64(codes[page, :, slot]), want[t], mag[t], f"row {t}")
            rest[page, :, slot] = before[page, :, slot]
        assert np.array_equal(rest, before)                                                    # and nowhere else
