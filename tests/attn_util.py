"""Helpers for the tests of the attention operators: a paged cache in a
symmetric heap with a scattered page table, and the error bounds.

Bounds (u = 2^-8, the unit roundoff of bf16's 8 significant bits; all sums and statistics float32):
  - an attention output is rounded once (u |out| at most), and its weights are
    rounded to bf16 before the product with v (u sum_j w_j |v_j| at most), so
    |err| <= 2u sum_j w_j |v_j|, plus the scores' float32 error: with
    S = scale sum_d |q_d k_d|, D products summed in float32 are within
    D 2^-23 S, which moves a weight by that relative amount;
  - log-sum-exp: the scores' error, plus 2^-20 of its size for exponential and
    logarithm;
  - a rotated element is a float32 expression of two products (2^-22 of their
    sizes) rounded once to bf16, or divided by the scale and rounded to 8 bits
    (2^-4 relative, 2^-10 below the smallest normal).
"""
from __future__ import annotations

import numpy as np
import torch

import oracle
from gpu_util import align, bf16_f64, to_bits, to_dev_bf16
from tile_centric_comm_gb300 import synth, tdg

U = 2.0 ** -8


def bits(x):
    return synth.f32_to_bf16_bits(np.ascontiguousarray(x, np.float32))


def check_attention(got_bits, want, D, what=""):
    got = bf16_f64(got_bits)
    tol = (2 * U + D * 2.0 ** -23 * want["smag"][..., None]) * want["mag"] + 1e-30
    bad = ~(np.abs(got - want["out"]) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside the bound, first at "
                           f"{np.argwhere(bad)[0].tolist()}: {got[bad][0]} for {want['out'][bad][0]}")


def check_lse(got, want, D, what=""):
    got = np.asarray(got, np.float64)
    empty = np.isneginf(want["lse"])
    assert np.array_equal(np.isneginf(got), empty), f"{what}: empty rows differ"
    tol = D * 2.0 ** -23 * want["smag"][~empty] + 2.0 ** -20 * (np.abs(want["lse"][~empty]) + 1)
    assert np.all(np.abs(got[~empty] - want["lse"][~empty]) <= tol), what


class Cache:
    """A cache whose sequences' pages are scattered over the ranks; every slot
    behind a length, and every page of nobody, holds NaN."""

    def __init__(self, W, lens, Hkv, D, page, e4m3=False, seed=0, extra_entries=0, fill=True):
        g = self.g = np.random.default_rng(seed)
        self.W, self.lens, self.Hkv, self.D, self.page, self.e4m3 = W, list(lens), Hkv, D, page, e4m3
        need = [-(-n // page) for n in lens]
        self.pages = -(-(sum(need) + 2) // W)
        entries = max(need + [1]) + extra_entries
        order = g.permutation(W * self.pages)
        self.table = np.full((len(need), entries), -7, np.int32)   # unused entries are no page ids
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        pool = tdg.paged_pool_bytes(self.pages, page, Hkv, D, e4m3)
        self.v_off = align(pool)
        self.part_off = align(self.v_off + pool)
        self.symm = tdg.Symm(W, self.part_off + align(tdg.paged_decode_part_bytes(Hkv, Hkv, D)), 64)
        self.k_scale = (g.random(Hkv) * 0.02 + 0.01).astype(np.float32)
        self.v_scale = (g.random(Hkv) * 0.02 + 0.01).astype(np.float32)
        self.scales = [torch.from_numpy(s).cuda() for s in (self.k_scale, self.v_scale)]
        self.cache = tdg.PagedCache(self.pages, page, Hkv, D, 0, self.v_off, e4m3=e4m3,
                                    k_scale=self.scales[0] if e4m3 else None,
                                    v_scale=self.scales[1] if e4m3 else None)
        shape = (W * self.pages, Hkv, page, D)
        nan = 0x7F if e4m3 else 0x7FC1
        self.k = np.full(shape, nan, np.uint8 if e4m3 else np.uint16)
        self.v = self.k.copy()
        if fill:
            for b, n in enumerate(lens):
                for j in range(n):
                    for dst in (self.k, self.v):
                        x = g.standard_normal((Hkv, D))
                        dst[self.table[b, j // page], :, j % page] = \
                            g.integers(0, 0x70, (Hkv, D)) | (g.integers(0, 2, (Hkv, D)) << 7) if e4m3 else bits(x)
        self.upload()
        self.table_d = torch.from_numpy(self.table).cuda()
        self.lens_d = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def upload(self):
        for r in range(self.W):
            for src, dst in zip((self.k, self.v), self.cache.pools(self.symm, r)):
                part = np.ascontiguousarray(src[r * self.pages:(r + 1) * self.pages])
                dst.view(torch.uint8).copy_(torch.from_numpy(part.view(np.uint8)).view(dst.view(torch.uint8).shape))

    def download(self):
        """The pools as they are now: codes, (W * pages, Hkv, page, D)."""
        out = []
        for i in range(2):
            parts = [self.cache.pools(self.symm, r)[i].view(torch.uint8).cpu().numpy() for r in range(self.W)]
            out.append(np.concatenate(parts).view(self.k.dtype))
        return out

    def values(self, codes, scale):
        x = oracle.e4m3_to_f64(codes) if self.e4m3 else oracle.bf16_to_f64(codes)
        return x * scale.astype(np.float64)[None, :, None] if self.e4m3 else x

    def sequence(self, b, n=None):
        """Keys and values of sequence b's first n tokens, float64 (n, Hkv, D)."""
        n = self.lens[b] if n is None else n
        return (self.values(oracle.gather_pages(self.k, self.table[b], n), self.k_scale),
                self.values(oracle.gather_pages(self.v, self.table[b], n), self.v_scale))


def strided_rows(parts, device="cuda"):
    """Several (T, heads, D) bf16 bit arrays as columns of one buffer's rows."""
    T = parts[0].shape[0]
    D = parts[0].shape[2]
    heads = [p.shape[1] for p in parts]
    buf = torch.empty((T, sum(heads) + 1, D), dtype=torch.bfloat16, device=device)
    buf.view(torch.int16).fill_(0x7FC1)
    out, at = [], 0
    for p, n in zip(parts, heads):
        view = buf[:, at:at + n]
        view.copy_(to_dev_bf16(p))
        out.append(view)
        at += n
    return buf, out


__all__ = ["U", "bits", "check_attention", "check_lse", "Cache", "strided_rows", "to_bits", "to_dev_bf16", "bf16_f64"]
