"""Helpers for the tests of the 8-bit operators and the MoE gradients: plain
implementations in 64 bits and the error bounds.

Bounds (u = 2^-24, the unit roundoff of float32):
  - a product: a block's 128 products of codes are exact in float32 and summed
    in it (at most 2u of the running magnitude an addition), the product of two
    scales rounded once, the multiply-add with the blocks before once each, a
    cut K joined by at most 8 additions; so |err| <= 2u (128 + blocks + 10) mag
    with mag = sum |scales| sum |a| |b|, plus half a step of bf16 (2^-8 |out|)
    where the output has that type;
  - codes of bf16 values are those of the correctly rounded float32 quotient:
    bit for bit;
  - a gated value g r u, r the reciprocal (1 ulp: 2u) of 1 + e (u), e = 2^t
    (2 ulp: 4u), t = -g log2(e): the constant and the product rounded, u |t|
    each, which moves e by 2u |t| ln 2 = 2u |g| relative, and two products (u
    each).  e counts in full for negative g and by e / (1 + e) for positive,
    where |g| e / (1 + e) < 0.28: 9u + 2u max(-g, 0.28), taken as 2^-20 +
    2^-23 max(-g, 0); its scale as much, and its code half a step off the
    quotient (2^-4 relative, 2^-10 below the smallest normal) plus twice that.
"""
from __future__ import annotations

import torch

E4M3 = torch.float8_e4m3fn
LEAST = 2.0 ** -100


def blocks(n):
    return -(-n // 128)


def padded(x, *multiples):
    """x with its last axes filled up with zeros to the multiples."""
    pad = []
    for size, m in zip(reversed(x.shape), reversed(multiples)):
        pad += [0, -size % m]
    return torch.nn.functional.pad(x, pad)


def quantised(x, rows=1):
    """The codes (bit patterns) and scales of bf16 or float64 rows (n, K), blocks rows x 128:
    in 64 bits, rounded to float32 where the definition says so."""
    n, K = x.shape
    v = padded(x.double(), rows, 128)
    v = v.view(v.shape[0] // rows, rows, v.shape[1] // 128, 128).transpose(1, 2)
    top = torch.nan_to_num(v.abs(), nan=0.0, posinf=torch.inf).flatten(2).amax(-1)
    scale = (top.float().double() / 448).float().clamp(min=LEAST)
    q = (v / scale.double()[..., None, None]).float()
    codes = torch.where(q.isnan(), q, q.clamp(-448, 448)).to(E4M3)
    codes = codes.transpose(1, 2).reshape(scale.shape[0] * rows, -1)[:n, :K]
    return codes.contiguous().view(torch.uint8), scale


def values(codes, scale):
    """float64 values of codes (n, K), scale one for each row or 128 rows and block."""
    n, K = codes.shape
    if scale.shape[0] != n:
        scale = scale.repeat_interleave(128, 0)[:n]
    return codes.double() * scale.double().repeat_interleave(128, 1)[:, :K]


def product(a, a_scale, b, b_scale):
    """(out, mag) in 64 bits."""
    x, w = values(a, a_scale), values(b, b_scale)
    return x @ w.T, x.abs() @ w.abs().T


def check_product(got, want, mag, K, what=""):
    tol = 2.0 ** -23 * (128 + blocks(K) + 10) * mag + 1e-37
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0].item()} for {want[bad][0].item()}")


def random_codes(g, *shape, most=448.0):
    """Codes over the whole range of the type: signs, subnormals, the largest."""
    x = torch.randn(*shape, generator=g, device="cuda") * torch.exp2(torch.randint(-9, 6, shape, generator=g, device="cuda").float())
    return x.clamp(-most, most).to(E4M3)


def random_scales(g, *shape):
    return torch.exp2(torch.rand(*shape, generator=g, device="cuda") * 6 - 8)


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)
