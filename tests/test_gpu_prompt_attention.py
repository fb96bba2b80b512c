"""GPU parity of the attention over packed prompts against the oracle."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from tile_centric_comm_gb300 import tdg
from attn_util import bits, check_attention, check_lse, strided_rows, to_bits, to_dev_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def symm():
    return tdg.Symm(1, 1024, 16)


def _ends(n, gap=0):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32) + gap


class Case:
    def __init__(self, nq, nk, Hq, Hkv, D, seed=0, tail=0, q_mul=1.0):
        g = np.random.default_rng(seed)
        self.nq, self.nk, self.Hq, self.Hkv, self.D = list(nq), list(nk), Hq, Hkv, D
        self.cu_q, self.cu_k = _ends(nq), _ends(nk)
        Tq, Tk = sum(nq) + tail, sum(nk) + tail
        self.q = bits(g.standard_normal((Tq, Hq, D)) * q_mul)
        self.k, self.v = bits(g.standard_normal((Tk, Hkv, D))), bits(g.standard_normal((Tk, Hkv, D)) + 0.25)

    def run(self, symm, causal=True, scale=0.0, lse=True, stream=None):
        Tq = len(self.q)
        _, (q, out) = strided_rows([self.q, np.full_like(self.q, 0x7FC1)])
        _, (k, v) = strided_rows([self.k, self.v])
        e = torch.full((Tq, self.Hq), float("nan"), device="cuda") if lse else None
        cu_q, cu_k = (torch.from_numpy(c).cuda() for c in (self.cu_q, self.cu_k))
        torch.cuda.synchronize()
        tdg.prompt_attention(symm, q, k, v, out, cu_q, cu_k, lse=e, causal=causal, scale=scale, stream=stream)
        torch.cuda.synchronize()
        assert symm.status()["code"] == 0
        return to_bits(out), e.cpu().numpy() if lse else None

    def check(self, got, causal=True, scale=0.0, some=None, rows=None):
        out, lse = got
        for b in range(len(self.nq)) if some is None else some:
            qs, ks = slice(self.cu_q[b], self.cu_q[b + 1]), slice(self.cu_k[b], self.cu_k[b + 1])
            q, k, v = (oracle.bf16_to_f64(x) for x in (self.q[qs], self.k[ks], self.v[ks]))
            o, e = out[qs], None if lse is None else lse[qs]
            if rows is not None and len(q) > rows and causal:     # the last rows of a long one
                q, o, e = q[-rows:], o[-rows:], None if e is None else e[-rows:]
            want = oracle.attention(q, k, v, causal, scale or None)
            check_attention(o, want, self.D, f"sequence {b} ({self.nq[b]} x {self.nk[b]})")
            if e is not None:
                check_lse(e, want, self.D, f"lse of sequence {b}")
        assert np.all(out[self.cu_q[-1]:] == 0x7FC1)              # rows of no sequence


LENS = [1, 2, 0, 127, 128, 129, 31, 255, 256, 257, 16, 300]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (5, 1), (14, 2), (8, 1), (16, 1), (6, 2)])
def test_packed_causal(symm, D, Hq, Hkv):
    c = Case(LENS, LENS, Hq, Hkv, D, seed=Hq * D, tail=3)
    got = c.run(symm)
    c.check(got)
    again = c.run(symm)
    assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1], equal_nan=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (3, 3), (128, 1), (33, 1)])
def test_unlike_lengths(symm, D, causal, Hq, Hkv):
    # pieces behind cached keys, more queries than keys (rows that see nothing), no keys, no queries
    nq = [1, 64, 100, 40, 7, 0, 5, 130]
    nk = [300, 64, 513, 13, 0, 50, 128, 129]
    c = Case(nq, nk, Hq, Hkv, D, seed=Hq, tail=1)
    c.check(c.run(symm, causal), causal)


def test_no_lse_scale_and_stream(symm):
    c = Case([70, 200], [70, 200], 4, 2, 128, seed=3)
    s = torch.cuda.Stream()
    c.check(c.run(symm, scale=0.2, lse=False, stream=s), scale=0.2)


@pytest.mark.parametrize("q_mul", [1e-30, 20.0])
def test_query_sizes(symm, q_mul):
    c = Case([300, 257], [300, 600], 8, 2, 128, seed=4, q_mul=q_mul)
    c.check(c.run(symm))


def test_growing_scores(symm):
    # every later key scores higher than all before it, by far more than the exponent's comfortable range
    c = Case([640], [640], 2, 1, 128, seed=6)
    k = np.zeros((640, 1, 128), np.float32)
    k[:, 0, 0] = np.arange(640) * 0.5
    q = np.zeros((640, 2, 128), np.float32)
    q[..., 0] = 8.0
    q[:, 1, 0] = -8.0                                    # and falling for the other head
    c.q, c.k = bits(q), bits(k)
    c.check(c.run(symm))


@pytest.mark.parametrize("D", [64, 128])
def test_what_others_hold_does_not_matter(symm, D):
    # the neighbours of sequence 1 hold NaN and infinity in queries, keys and values, its own later keys too
    c = Case([70, 130, 90], [70, 130, 90], 4, 2, D, seed=5, tail=2)
    good = slice(70, 200)
    for x in (c.q, c.k, c.v):
        keep = x[good].copy()
        x[:] = np.where(np.arange(x.size).reshape(x.shape) % 2, 0x7FC1, 0x7F80).astype(np.uint16)
        x[good] = keep
    got = c.run(symm)
    c.check(got, some=[1])
    # a key that a row does not see may hold anything: all rows but the last stay as they were
    c.k[199] = 0x7FC1
    bad = c.run(symm)
    assert np.array_equal(bad[0][70:199], got[0][70:199]) and np.array_equal(bad[1][70:199], got[1][70:199])


def test_many_sequences(symm):
    g = np.random.default_rng(7)
    n = g.integers(0, 40, 500).tolist()
    c = Case(n, n, 4, 1, 64, seed=7)
    c.check(c.run(symm))


def test_nothing_to_do(symm):
    q = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((0, 2, 128), dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    tdg.prompt_attention(symm, q, k, k, q, cu, cu)
    # queries without a single key
    c = Case([5], [0], 4, 2, 128)
    out, lse = c.run(symm)
    assert np.all(out == 0) and np.all(np.isneginf(lse))


@pytest.mark.slow
@pytest.mark.parametrize("Hq,Hkv,D,n", [(64, 8, 128, 8192), (40, 8, 128, 5001), (8, 8, 64, 12345)])
def test_long(symm, Hq, Hkv, D, n):
    c = Case([n], [n], Hq, Hkv, D, seed=n)
    c.check(c.run(symm), rows=3)
    # and rows at the beginning and in the middle
    out, lse = c.run(symm)
    for i in (0, 1, 127, 128, n // 2):
        q, k, v = (oracle.bf16_to_f64(x) for x in (c.q[i:i + 1], c.k[:i + 1], c.v[:i + 1]))
        want = oracle.attention(q, k, v)
        check_attention(out[i:i + 1], want, D, f"row {i}")
        check_lse(lse[i:i + 1], want, D, f"row {i}")


@pytest.mark.parametrize("cu_q,cu_k", [([0, 50, 40, 90], [0, 50, 60, 90]), ([0, 30, 60, 91], [0, 30, 60, 90]),
                                       ([-1, 30, 60, 90], [0, 30, 60, 90]), ([0, 30, 60, 90], [0, 30, 60, 95])])
def test_bad_offsets_are_reported(symm, cu_q, cu_k):
    c = Case([30, 30, 30], [30, 30, 30], 4, 2, 64)
    q, k, v = (to_dev_bf16(x) for x in (c.q, c.k, c.v))
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    tdg.prompt_attention(symm, q, k, v, out, torch.tensor(cu_q, dtype=torch.int32, device="cuda"),
                         torch.tensor(cu_k, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    st = symm.status()
    assert st["code"] == tdg.TDG_ERR_DEVICE and st["where"] == "cu"


def test_refusals(symm):
    c = Case([30], [30], 4, 2, 128)
    q, k, v = (to_dev_bf16(x) for x in (c.q, c.k, c.v))
    out = torch.empty_like(q)
    cu = torch.from_numpy(c.cu_q).cuda()

    def rc(**kw):
        a = tdg.PromptAttentionArgs(Tq=30, Tk=30, B=1, Hq=4, Hkv=2, D=128, q=q.data_ptr(), k=k.data_ptr(),
                                    v=v.data_ptr(), q_stride=512, k_stride=256, v_stride=256, out=out.data_ptr(),
                                    out_stride=512, cu_q=cu.data_ptr(), cu_k=cu.data_ptr(), causal=1)
        for key, x in kw.items():
            setattr(a, key, x)
        return tdg.lib().tdg_prompt_attention(symm.h, ctypes.byref(a), None)

    bad = tdg.TDG_ERR_INVALID
    assert rc() == tdg.TDG_OK
    assert rc(Tq=-1) == bad and rc(Tk=-1) == bad and rc(Tq=1 << 31) == bad and rc(B=65536) == bad
    assert rc(Hq=5) == bad and rc(Hkv=0) == bad and rc(D=96) == bad and rc(Hq=258, q_stride=1 << 16, out_stride=1 << 16) == bad
    assert rc(q=None) == bad and rc(k=None) == bad and rc(out=None) == bad and rc(cu_q=None) == bad
    assert rc(q=q.data_ptr() + 4) == bad and rc(q_stride=508) == bad and rc(k_stride=248) == bad and rc(v_stride=260) == bad
    assert rc(out_stride=504) == bad and rc(out=q.data_ptr()) == bad and rc(out=v.data_ptr()) == bad
    assert rc(causal=2) == bad and rc(scale=-0.5) == bad and rc(scale=float("nan")) == bad
    with pytest.raises(ValueError, match="fit together"):
        tdg.prompt_attention(symm, q, k, v[:29], out, cu, cu)
    with pytest.raises(TypeError, match="bfloat16"):
        tdg.prompt_attention(symm, q.float(), k, v, out, cu, cu)
    with pytest.raises(TypeError, match="int32"):
        tdg.prompt_attention(symm, q, k, v, out, cu.long(), cu)
    torch.cuda.synchronize()
    assert symm.status()["code"] == 0


@pytest.mark.parametrize("D", [64, 128])
def test_output_rows_off_the_32_byte_grid(symm, D):
    # an output that starts 16 bytes off, with a row stride of an odd number of 16-byte units
    c = Case([70, 200], [70, 200], 4, 2, D, seed=3)
    T, n = len(c.q), 4 * D
    buf = torch.full(((T + 1) * (n + 8),), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = torch.as_strided(buf, (T, 4, D), (n + 8, D, 1), 8)
    q, k, v = (to_dev_bf16(x) for x in (c.q, c.k, c.v))
    cu = torch.from_numpy(c.cu_q).cuda()
    tdg.prompt_attention(symm, q, k, v, out, cu, cu)
    torch.cuda.synchronize()
    assert symm.status()["code"] == 0
    c.check((to_bits(out), None))
    rest = torch.ones_like(buf, dtype=torch.bool)
    torch.as_strided(rest, (T, 4, D), (n + 8, D, 1), 8).fill_(False)
    assert torch.isnan(buf[rest].float()).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,nq,nk", [
    (8, 1, [1], [5000]),                                   # few rows, long keys: 8 CTAs share an item
    (7, 1, [1, 17, 40], [3000, 2177, 4000]),
    (4, 2, [3, 0, 64, 5], [2500, 3000, 64, 2]),            # beside sequences of few keys, and rows that see nothing
    (16, 2, [130, 9], [1500, 1300]),
    (2, 2, [700], [700]),
])
def test_keys_shared_by_ctas(symm, D, causal, Hq, Hkv, nq, nk):
    c = Case(nq, nk, Hq, Hkv, D, seed=sum(nk) + D, tail=1)
    got = c.run(symm, causal)
    c.check(got, causal)
    again = c.run(symm, causal)
    assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1], equal_nan=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,nq,nk", [
    (48, 48, LENS + [511, 64, 65, 63, 1000], LENS + [511, 64, 65, 63, 1000]),
    (128, 64, [1, 70, 300, 0, 129, 64, 2, 90, 33, 5, 200, 17], [700, 70, 100, 50, 1000, 0, 65, 222, 33, 64, 1, 128]),
    (32, 8, [1 + 7 * i % 41 for i in range(300)], [1 + 7 * i % 41 for i in range(300)]),  # more than the table's entries
])
def test_many_items(symm, D, causal, Hq, Hkv, nq, nk):
    # several items for each SM: taken by length, and with heads of 64 by two CTAs an SM
    c = Case(nq, nk, Hq, Hkv, D, seed=Hq + D, tail=2)
    bad = 4                              # what one sequence holds is no other's business
    c.k[c.cu_k[bad]:c.cu_k[bad + 1]] = 0x7FC0
    c.v[c.cu_k[bad]:c.cu_k[bad + 1]] = 0x7F80
    got = c.run(symm, causal)
    c.check(got, causal, some=[b for b in range(len(nq)) if b != bad])
    again = c.run(symm, causal)
    assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1], equal_nan=True)


def test_refuses_what_would_overwrite_its_inputs(symm):
    # nothing is launched: every buffer keeps its bytes
    c = Case([30, 20], [30, 20], 4, 2, 128)
    q, k, v = (to_dev_bf16(x) for x in (c.q, c.k, c.v))
    out = torch.full_like(q, 7.0)
    lse = torch.full((50, 4), 7.0, device="cuda")
    cu_q, cu_k = torch.from_numpy(c.cu_q).cuda(), torch.from_numpy(c.cu_k).cuda()

    def rc(**kw):
        a = tdg.PromptAttentionArgs(Tq=50, Tk=50, B=2, Hq=4, Hkv=2, D=128, q=q.data_ptr(), k=k.data_ptr(),
                                    v=v.data_ptr(), q_stride=512, k_stride=256, v_stride=256, out=out.data_ptr(),
                                    out_stride=512, lse=lse.data_ptr(), cu_q=cu_q.data_ptr(), cu_k=cu_k.data_ptr(), causal=1)
        for key, x in kw.items():
            setattr(a, key, x)
        return tdg.lib().tdg_prompt_attention(symm.h, ctypes.byref(a), None)

    bad = tdg.TDG_ERR_INVALID
    kept = [(x, x.clone()) for x in (q, k, v, out, lse, cu_q, cu_k)]
    for x in (q, k, v, out):                                             # lse over rows: their first, their last bytes
        assert rc(lse=x.data_ptr()) == bad and rc(lse=x.data_ptr() + x.numel() * 2 - 4) == bad
    for x in (cu_q, cu_k):                                               # outputs over offsets
        assert rc(lse=x.data_ptr() + 8) == bad and rc(lse=x.data_ptr() - 50 * 4 * 4 + 4) == bad
    for name in ("cu_q", "cu_k"):
        assert rc(**{name: out.data_ptr() + 64}) == bad and rc(**{name: lse.data_ptr() + 50 * 4 * 4 - 4}) == bad
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in kept)
    assert rc(cu_k=cu_q.data_ptr()) == 0 and rc(lse=None) == 0           # inputs may be one another
    torch.cuda.synchronize()
    assert symm.status()["code"] == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cu_q,cu_k,bad", [
    ([0, 50, 40, 90], [0, 50, 60, 90], [1]),           # backwards in the queries: rows 40 .. 49 lie in two sequences
    ([0, 30, 60, 90], [0, 50, 40, 90], [1]),           # backwards in the keys
    ([0, 30, 60, 91], [0, 30, 60, 90], [2]),           # past the last query
    ([0, 30, 60, 90], [0, 30, 60, 95], [2]),           # past the last key
    ([-1, 30, 60, 90], [0, 30, 60, 90], [0]),
    ([0, 30, 60, 90], [0, 30, 2 ** 31 - 1, 90], [1, 2]),
    ([0, -2 ** 31, 60, 90], [0, 30, 60, 90], [0, 1]),
])
def test_bad_offsets_leave_the_others_right(symm, D, cu_q, cu_k, bad):
    c = Case([30, 30, 30], [30, 30, 30], 4, 2, D, seed=D)
    _check_bad_offsets(symm, c, cu_q, cu_k, bad)


@pytest.mark.parametrize("D,Hq,Hkv,n", [(128, 4, 1, 300), (64, 48, 48, 40), (128, 8, 8, 100)])
def test_bad_offsets_among_many(symm, D, Hq, Hkv, n):
    # more sequences than the item table has entries; items by length, with heads of 64 by two CTAs an SM
    g = np.random.default_rng(n)
    lens = g.integers(1, 20 if n == 300 else 300, n).tolist()
    c = Case(lens, lens, Hq, Hkv, D, seed=n)
    cu_q, cu_k = c.cu_q.tolist(), c.cu_k.tolist()
    cu_k[n // 2] = len(c.k) + 7                         # the end of one sequence and the beginning of the next
    cu_q[-1] = len(c.q) + 1
    _check_bad_offsets(symm, c, cu_q, cu_k, [n // 2 - 1, n // 2, n - 1])


def _check_bad_offsets(symm, c, cu_q, cu_k, bad):
    q, k, v = (to_dev_bf16(x) for x in (c.q, c.k, c.v))
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    out.view(torch.int16).fill_(0x7FC1)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    tdg.prompt_attention(symm, q, k, v, out, torch.tensor(cu_q, dtype=torch.int32, device="cuda"),
                         torch.tensor(cu_k, dtype=torch.int32, device="cuda"), lse=lse)
    torch.cuda.synchronize()
    st = symm.status()
    assert st["code"] == tdg.TDG_ERR_DEVICE and st["where"] == "cu" and st["index"] in bad
    out, lse = to_bits(out), lse.cpu().numpy()
    times = np.zeros(len(c.q), int)
    good = [b for b in range(len(cu_q) - 1) if b not in bad]
    for b in good:
        times[cu_q[b]:cu_q[b + 1]] += 1
    for b in good:
        rows, keys = np.arange(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        want = oracle.attention(*(oracle.bf16_to_f64(x) for x in (c.q[rows], c.k[keys], c.v[keys])))
        once = times[rows] == 1
        want = {name: x[once] for name, x in want.items()}
        check_attention(out[rows[once]], want, c.D, f"sequence {b}")
        check_lse(lse[rows[once]], want, c.D, f"lse of sequence {b}")
    assert np.all(out[times == 0] == 0x7FC1) and np.all(lse[times == 0] == 7)       # rows of no valid sequence
