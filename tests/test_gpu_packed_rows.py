"""8-bit operands as columns of one buffer: a row's codes beside its scales
(as rows are sent between ranks), its input and its product."""
import pytest
import torch

from expert_util import E4M3, blocks, check_product, generator, product, quantised, random_codes, random_scales
from tile_centric_comm_gb300 import tdg

pytestmark = pytest.mark.gpu
POISON = 0x5A


@pytest.fixture(scope="module")
def symm():
    return tdg.Symm(1, 1024, 16)


class Packed:
    """Rows of bytes; columns of any type, 16 bytes of filler between them."""

    def __init__(self, n, **columns):
        self.at, width = {}, 16
        for name, (count, kind) in columns.items():
            self.at[name] = width, count, kind
            width += -(-count * kind.itemsize // 16) * 16 + 16
        self.bytes = torch.full((n, width), POISON, dtype=torch.uint8, device="cuda")

    def __getattr__(self, name):
        at, count, kind = self.at[name]
        return self.bytes[:, at:at + count * kind.itemsize].view(kind)

    def filler(self):
        keep = torch.ones(self.bytes.shape[1], dtype=torch.bool, device="cuda")
        for at, count, kind in self.at.values():
            keep[at:at + count * kind.itemsize] = False
        return self.bytes[:, keep]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("n,K", [(1, 16), (2, 272), (700, 2048)])
def test_codes_beside_their_scales_and_input(symm, n, K, gated):
    p = Packed(n, x=(2 * K if gated else K, torch.bfloat16), codes=(K, E4M3), scale=(blocks(K), torch.float32))
    x = torch.randn(n, 2 * K if gated else K, generator=generator(K), device="cuda").to(torch.bfloat16)
    p.x.copy_(x)
    tdg.quantise_rows(symm, p.x, p.codes, p.scale, gated=gated)
    codes, scale = torch.empty(n, K, dtype=E4M3, device="cuda"), torch.empty(n, blocks(K), device="cuda")
    tdg.quantise_rows(symm, x, codes, scale, gated=gated)
    if not gated:
        assert torch.equal(codes.view(torch.uint8), quantised(x)[0])
    assert torch.equal(p.codes.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(p.scale, scale) and torch.equal(p.x, x)
    assert bool((p.filler() == POISON).all())


# narrow tiles, wide ones, K divided over CTAs and over pairs
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K", [(2, 136, 144), (40, 256, 2048), (250, 5112, 2576), (2000, 7160, 528)])
def test_products_beside_their_operand(symm, M, N, K, f32):
    p = Packed(M, a=(K, E4M3), scale=(blocks(K), torch.float32), out=(N, torch.float32 if f32 else torch.bfloat16))
    g = generator(M)
    p.a.copy_(random_codes(g, M, K))
    p.scale.copy_(random_scales(g, M, blocks(K)))
    b, b_scale = random_codes(g, N, K), random_scales(g, blocks(N), blocks(K))
    before = p.a.clone(), p.scale.clone()
    tdg.scaled_gemm(symm, p.a, p.scale, b, b_scale, p.out)
    want, mag = product(*before, b, b_scale)
    check_product(p.out, want, mag, K)
    assert torch.equal(p.a.view(torch.uint8), before[0].view(torch.uint8)) and torch.equal(p.scale, before[1])
    assert bool((p.filler() == POISON).all())


def test_columns_that_overlap_are_refused(symm):
    n, K = 8, 256
    buf = torch.zeros(n, 2048, dtype=torch.uint8, device="cuda")

    def columns(at, count, kind):
        return buf[:, at:at + count * kind.itemsize].view(kind)
    x, codes, scale = columns(0, K, torch.bfloat16), columns(512, K, E4M3), columns(768, 2, torch.float32)
    tdg.quantise_rows(symm, x, codes, scale)
    for args in ((x, columns(496, K, E4M3), scale), (x, codes, columns(764, 2, torch.float32)), (x, codes, columns(508, 2, torch.float32)),
                 (x, codes, columns(600, 2, torch.float32)), (columns(528, K, torch.bfloat16), codes, scale),
                 # rows that lie otherwise than the codes': told by their whole range
                 (x, buf.view(-1)[512:512 + n * K].view(n, K).view(E4M3), columns(1024, 2, torch.float32))):
        with pytest.raises(tdg.TdgError) as e:
            tdg.quantise_rows(symm, *args)
        assert e.value.code == tdg.TDG_ERR_INVALID
    b, b_scale = torch.zeros(128, K, dtype=torch.uint8, device="cuda").view(E4M3), torch.zeros(1, 2, device="cuda")
    tdg.scaled_gemm(symm, codes, scale, b, b_scale, columns(784, 128, torch.bfloat16))
    for at in (256 + 16, 752, 768, 512):
        with pytest.raises(tdg.TdgError) as e:
            tdg.scaled_gemm(symm, codes, scale, b, b_scale, columns(at, 128, torch.bfloat16))
        assert e.value.code == tdg.TDG_ERR_INVALID
    torch.cuda.synchronize()
    assert symm.status()["code"] == 0
