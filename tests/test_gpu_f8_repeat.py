"""F8 products and the gated block give the same bits from call to call, at sizes
that fill the device."""
import pytest
import torch

import f8_ref as ref
import weight_only_quantized_w8a16_amd as qg

pytestmark = pytest.mark.gpu

BF, SF = torch.bfloat16, torch.float32
F8 = torch.float8_e4m3fn


def random_codes(g, *shape):
    c = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    c[(c & 0x7F) == 0x7F] = 0x3A
    return c.view(F8)


def scales(g, *shape):
    return torch.rand(shape, generator=g, device="cuda") + 0.5


@pytest.mark.parametrize("m,n,k,b_block", [(1, 131072, 2048, 128), (13, 18944, 3584, 128), (333, 3584, 18944, 128),
                                           (2000, 18944, 3584, 128), (100, 400, 9232, 1), (5000, 2064, 2064, 1)])
def test_product_repeats_its_bits(m, n, k, b_block):
    g = torch.Generator(device="cuda").manual_seed(m)
    args = (random_codes(g, m, k), scales(g, ref.blocks(k), m), random_codes(g, n, k),
            scales(g, *((ref.blocks(n), ref.blocks(k)) if b_block == 128 else (ref.blocks(k), n))))
    first = qg.gemm_f8(*args, b_block=b_block, out_dtype=SF)
    assert torch.isfinite(first).all()
    for _ in range(8):
        assert torch.equal(qg.gemm_f8(*args, b_block=b_block, out_dtype=SF), first)


@pytest.mark.parametrize("rows", [48, 12288])
def test_product_by_expert_repeats_its_bits(rows):
    g = torch.Generator(device="cuda").manual_seed(rows)
    E, n, k = 64, 2816, 2048
    share = torch.bincount(torch.randint(0, E, (rows,), generator=g, device="cuda"), minlength=E)
    off = torch.cat([share.new_zeros(1), share.cumsum(0)]).int()
    args = (random_codes(g, rows, k), scales(g, 16, rows), off, random_codes(g, E, n, k), scales(g, E, 22, 16))
    first = qg.gemm_f8_grouped(*args, out_dtype=SF)
    assert torch.isfinite(first).all()
    for _ in range(8):
        assert torch.equal(qg.gemm_f8_grouped(*args, out_dtype=SF), first)


@pytest.mark.parametrize("m,inter,k", [(1, 13312, 2048), (100, 1408, 2048), (2000, 9472, 3584)])
def test_gated_block_repeats_its_bits(m, inter, k):
    g = torch.Generator(device="cuda").manual_seed(m)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)   # noqa: E731
    xq, xs, xt, xts = qg.quantize_f8(r(m, k), transposed=True)
    wq, ws, wt, wts = qg.quantize_f8(r(2 * inter, k) * 0.02, block=128, transposed=True)
    ws, wts = ws * 1.25, wts * 1.25
    dh = r(m, inter)

    def step():
        h, gu = qg.gated_f8(xq, xs, wq, ws, return_gu=True)
        return (h, gu, qg.gated_f8(xq, xs, wq, ws, out_dtype=SF),
                *qg.gated_f8_backward(dh, gu, xt, xts, wt, wts, dx_dtype=SF, dw_dtype=SF))
    first = step()
    assert all(torch.isfinite(t).all() for t in first)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(step(), first))
