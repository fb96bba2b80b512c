"""The oracle of the attention operators, pinned by brute force and closed forms."""
import math

import numpy as np
import pytest

import oracle
from tile_centric_comm_gb300 import synth


def _bits(x):
    return synth.f32_to_bf16_bits(np.ascontiguousarray(x, np.float32))


def test_e4m3_values_and_rounding():
    v = oracle.e4m3_to_f64(np.arange(256))
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1.0 and v[0x7E] == 448.0
    assert np.isnan(v[0x7F]) and np.isnan(v[0xFF]) and v[0x81] == -(2.0 ** -9)
    assert np.all(np.diff(v[:0x7F]) > 0)
    codes = np.array([i for i in range(256) if i & 0x7F != 0x7F])
    assert np.array_equal(oracle.f64_to_e4m3(v[codes]), codes)
    # ties go to the even code, everything else to the nearest, large values to 448
    mid = (v[:0x7E] + v[1:0x7F]) / 2
    want = np.array([i if i % 2 == 0 else i + 1 for i in range(0x7E)])
    assert np.array_equal(oracle.f64_to_e4m3(mid), want)
    assert np.array_equal(oracle.f64_to_e4m3(mid * (1 + 1e-9)), np.arange(1, 0x7F))
    assert oracle.f64_to_e4m3([1e9, math.inf, -math.inf]).tolist() == [0x7E, 0x7E, 0xFE]


@pytest.mark.parametrize("inter", [False, True])
def test_rope_turns_each_pair(inter):
    g = np.random.default_rng(1)
    T, H, D, rot, P = 3, 2, 64, 32, 11
    x = _bits(g.standard_normal((T, H, D)))
    ang = g.standard_normal((P, rot // 2))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    pos = g.integers(0, P, (3, T)).astype(np.int32)
    sec = (5, 0, 11)
    out, mag = oracle.rope(x, cs, pos, sec, inter)
    xv = oracle.bf16_to_f64(x)
    for t in range(T):
        for i in range(rot // 2):
            a = 0 if i < 5 else 2
            c, s = float(cs[pos[a, t], i]), float(cs[pos[a, t], rot // 2 + i])
            d0, d1 = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
            z = (xv[t, :, d0] + 1j * xv[t, :, d1]) * (c + 1j * s)
            np.testing.assert_allclose(out[t, :, d0] + 1j * out[t, :, d1], z, rtol=1e-14, atol=1e-14)
            assert np.all(mag[t, :, d0] >= np.abs(out[t, :, d0]))
    assert np.array_equal(out[..., rot:], xv[..., rot:])


def test_attention_against_a_direct_sum():
    g = np.random.default_rng(2)
    Lq, Lk, Hq, Hkv, D = 4, 6, 4, 2, 8
    q, k, v = g.standard_normal((Lq, Hq, D)), g.standard_normal((Lk, Hkv, D)), g.standard_normal((Lk, Hkv, D))
    for causal in (True, False):
        r = oracle.attention(q, k, v, causal, 0.3)
        for i in range(Lq):
            n = i + Lk - Lq + 1 if causal else Lk
            for h in range(Hq):
                w = [math.exp(0.3 * float(q[i, h] @ k[j, h // 2])) for j in range(n)]
                want = sum(w[j] * v[j, h // 2] for j in range(n)) / sum(w)
                np.testing.assert_allclose(r["out"][i, h], want, rtol=1e-12, atol=1e-13)
                assert abs(r["lse"][i, h] - math.log(sum(w))) < 1e-12


def test_attention_rows_that_see_nothing():
    g = np.random.default_rng(3)
    q, k = g.standard_normal((5, 2, 4)), g.standard_normal((3, 1, 4))
    r = oracle.attention(q, k, k, True)          # 5 queries, 3 keys: the first two see nothing
    assert np.all(r["out"][:2] == 0) and np.all(np.isneginf(r["lse"][:2]))
    np.testing.assert_allclose(r["out"][2], np.repeat(k[:1, 0][:, None], 2, 1)[0])   # one key: its value
    r = oracle.attention(q, k[:0], k[:0], False)
    assert np.all(r["out"] == 0) and np.all(np.isneginf(r["lse"]))


def test_cache_rows_and_gather():
    table = np.array([[3, 0, -7], [2, 1, 4]])
    assert oracle.cache_rows(table, [5, 9], 4) == [(0, 0), (4, 0)]
    assert oracle.cache_rows(table, [5, 9], 4, [0, 2, 5]) == [(3, 3), (0, 0), (1, 2), (1, 3), (4, 0)]
    pool = np.arange(5 * 2 * 4 * 1).reshape(5, 2, 4, 1)
    got = oracle.gather_pages(pool, table[0], 5)
    assert got[4, 0, 0] == pool[0, 0, 0, 0] and got[1, 1, 0] == pool[3, 1, 1, 0] and got.shape == (5, 2, 1)
