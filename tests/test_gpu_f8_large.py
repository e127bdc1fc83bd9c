"""F8 operators at their largest sizes on the GPU: rows past 2^30 and operands
past 2 GiB, sampled outputs against the plain forms."""
import numpy as np
import pytest
import torch

import f8_ref as ref
import weight_only_quantized_w8a16_amd as qg

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32
F8 = torch.float8_e4m3fn


def room(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB of device memory")


def dev(a):
    a = torch.from_numpy(np.ascontiguousarray(a)).to("cuda")
    return a.float() if a.dtype == torch.float64 else a


def exact_pair(rng, rows, k, block):
    """Codes of -2 .. 2 and power-of-two scales: every sum is exact in fp32."""
    c = ref.encode(rng.integers(-2, 3, (rows, k)).astype(np.float64))
    shape = (ref.blocks(k), rows) if block == 1 else (ref.blocks(rows), ref.blocks(k))
    return c, np.exp2(rng.integers(-1, 2, shape))


@pytest.mark.parametrize("tile", ["auto", "stream", "T256", "T128", "T64"])
def test_rows_past_2_30(tile):
    """More rows than 2^30: the scales of a second 128 k start past 2^32 bytes.  Three parts of the rows, at both ends
    and in the middle, have values; the others hold what the memory held."""
    room(225)
    qg.set_override(f8_tile=tile)
    rng = np.random.default_rng(7)
    m, n, k, part = 2 ** 30 + 64, 32, 144, 300
    A = torch.empty((m, k), dtype=torch.uint8, device="cuda")
    AS = torch.empty((2, m), device="cuda")
    C = torch.empty((m, n), dtype=BF, device="cuda")
    cb, sb = zip(*(exact_pair(rng, n, k, 128) for _ in range(3)))
    starts = (0, m // 2 - 77, m - part)
    a = []
    for s in starts:
        c, scale = exact_pair(rng, part, k, 1)
        A[s:s + part] = dev(c)
        AS[:, s:s + part] = dev(scale)
        a.append(ref.values(c, scale))
    codes, scales = dev(np.stack(cb)).view(F8), dev(np.stack(sb))
    try:
        qg.gemm_f8(A.view(F8), AS, codes[0], scales[0], out=C)
        for s, x in zip(starts, a):
            want = x @ ref.values(cb[0], sb[0], 128).T
            assert torch.equal(C[s:s + part].cpu(), torch.from_numpy(want).to(BF))
        # by expert: the parts are the first, the second and the last expert's
        off = dev(np.array([0, part, m - part, m], np.int32))
        qg.gemm_f8_grouped(A.view(F8), AS, off, codes, scales, out=C)
        for e, (s, x) in enumerate(zip(starts, a)):
            want = x @ ref.values(cb[e], sb[e], 128).T
            assert torch.equal(C[s:s + part].cpu(), torch.from_numpy(want).to(BF))
    finally:
        del A, AS, C
        torch.cuda.empty_cache()


# -- operands past 2 GiB --------------------------------------------------------------

TILES = ["stream", "T256", "T128", "T64"]


def big_codes(g, *shape):
    """Codes of -2, -1, 1 and 2."""
    c = torch.randint(0, 4, shape, generator=g, device="cuda", dtype=torch.uint8)
    return (c & 1).mul_(8).add_(0x38).add_((c & 2).mul_(64)).view(F8)


def big_scales(g, *shape):
    return torch.randint(-1, 2, shape, generator=g, device="cuda").float().exp2_()


def rows_of(codes, scales, rows):
    """Values of some rows, scales by rows."""
    s = scales[:, rows].double().t().repeat_interleave(128, 1)[:, :codes.shape[1]]
    return codes.view(torch.uint8)[rows].view(F8).double() * s


def channels_of(codes, scales, rows):
    """The same, scales by blocks."""
    s = scales[rows // 128].double().repeat_interleave(128, 1)[:, :codes.shape[1]]
    return codes.view(torch.uint8)[rows].view(F8).double() * s


def sample(g, n, count=400):
    """Rows to look at: both ends and some between."""
    return torch.cat([torch.arange(min(n, 70), device="cuda"), torch.arange(n - min(n, 70), n, device="cuda"),
                      torch.randint(0, n, (count,), generator=g, device="cuda")])


def check(C, a, b, rows, cols):
    want = a @ b.t()
    assert torch.equal(C[rows][:, cols].double(), want.to(C.dtype).double())


@pytest.fixture
def gen():
    room(40)
    yield torch.Generator(device="cuda").manual_seed(1)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("m,n,k", [(3, 262160, 8208), (300, 262160, 8208), (262170, 144, 8208)])
def test_products_of_operands_past_2gib(gen, m, n, k, tile):
    qg.set_override(f8_tile=tile)
    a, b = big_codes(gen, m, k), big_codes(gen, n, k)
    assert max(a.numel(), b.numel()) > 2 ** 31
    sa, sb = big_scales(gen, ref.blocks(k), m), big_scales(gen, ref.blocks(n), ref.blocks(k))
    C = qg.gemm_f8(a, sa, b, sb, out_dtype=SF)
    rows, cols = sample(gen, m), sample(gen, n)
    check(C, rows_of(a, sa, rows), channels_of(b, sb, cols), rows, cols)


@pytest.mark.parametrize("split", [1, 2])
@pytest.mark.parametrize("tile", TILES)
def test_results_past_4gib(gen, tile, split):
    qg.set_override(f8_tile=tile, f8_split=split)
    m, n, k = 131100, 9232, 272
    a, b = big_codes(gen, m, k), big_codes(gen, n, k)
    rows, cols = sample(gen, m), sample(gen, n)
    for block, sb in ((128, big_scales(gen, ref.blocks(n), ref.blocks(k))), (1, big_scales(gen, ref.blocks(k), n))):
        sa = big_scales(gen, ref.blocks(k), m)
        C = qg.gemm_f8(a, sa, b, sb, out_dtype=SF, b_block=block)
        assert C.numel() * 4 > 2 ** 32
        check(C, rows_of(a, sa, rows), (channels_of if block == 128 else rows_of)(b, sb, cols), rows, cols)


@pytest.mark.parametrize("tile", TILES)
def test_experts_past_2gib(gen, tile):
    qg.set_override(f8_tile=tile)
    E, n, k = 9, 16400, 16400
    off = np.cumsum([0, 3, 0, 70, 1, 40, 0, 130, 16, 20])
    m = int(off[-1])
    a, b = big_codes(gen, m, k), big_codes(gen, E, n, k)
    assert b.numel() > 2 ** 31
    sa, sb = big_scales(gen, ref.blocks(k), m), big_scales(gen, E, ref.blocks(n), ref.blocks(k))
    C = qg.gemm_f8_grouped(a, sa, dev(off.astype(np.int32)), b, sb, out_dtype=SF)
    cols = sample(gen, n)
    for e in range(E):
        rows = torch.arange(off[e], off[e + 1], device="cuda")
        check(C, rows_of(a, sa, rows), channels_of(b[e], sb[e], cols), rows, cols)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("m,inter,k", [(65600, 16512, 144), (40, 131200, 8208)])
def test_gated_past_2gib(gen, m, inter, k, tile):
    qg.set_override(f8_tile=tile)
    a, b = big_codes(gen, m, k), big_codes(gen, 2 * inter, k)
    sa, sb = big_scales(gen, ref.blocks(k), m), big_scales(gen, ref.blocks(2 * inter), ref.blocks(k))
    h, gu = qg.gated_f8(a, sa, b, sb, out_dtype=SF, return_gu=True)
    assert max(b.numel(), gu.numel() * 4) > 2 ** 31
    rows, cols = sample(gen, m), sample(gen, inter)
    av, g, u = rows_of(a, sa, rows), channels_of(b, sb, cols), channels_of(b, sb, cols + inter)
    check(gu, av, g, rows, cols)
    check(gu, av, u, rows, cols + inter)
    g, u = av @ g.t(), av @ u.t()
    want = g * torch.sigmoid(g) * u
    # the sigmoid's roundings, as in the tests of small sizes
    tol = (7 * g.abs() + 8) * 2.0 ** -23 * want.abs() + 2.0 ** -126 * (g * u).abs() + 2.0 ** -140
    assert bool(((h[rows][:, cols].double() - want).abs() <= tol).all())


@pytest.mark.parametrize("tile", TILES)
def test_backward_past_2gib(gen, tile):
    """With g = 0: act = 0 and act' = 1/2, so D = [dH u / 2 | 0] keeps its bits."""
    qg.set_override(f8_tile=tile)
    m, inter, k = 65600, 16512, 48
    dh, gu = big_codes(gen, m, inter).to(BF), big_codes(gen, m, 2 * inter).to(BF)
    gu[:, :inter] = 0
    assert dh.numel() * 2 > 2 ** 31 and gu.numel() > 2 ** 31
    xt, xts = big_codes(gen, k, m), big_scales(gen, ref.blocks(m), k)
    wt, wts = big_codes(gen, k, 2 * inter), big_scales(gen, 1, ref.blocks(2 * inter))
    dx, dw = qg.gated_f8_backward(dh, gu, xt, xts, wt, wts, dx_dtype=SF, dw_dtype=SF)
    rows, chans = sample(gen, m), sample(gen, inter)
    d = dh[rows].double() * gu[rows, inter:].double() / 2
    every = torch.arange(k, device="cuda")
    check(dx, d, channels_of(wt, wts, every)[:, :inter], rows, every)
    d = (dh[:, chans].double() * gu[:, inter:][:, chans].double() / 2).t()
    check(dw, d, rows_of(xt, xts, every), chans, every)
    assert not dw[inter:].any()


@pytest.mark.parametrize("block", [1, 128])
def test_conversions_past_2gib(gen, block):
    m, k = 262170, 8208
    x = torch.randn(m, k, generator=gen, device="cuda", dtype=BF)
    assert x.numel() > 2 ** 31
    got = qg.quantize_f8(x, block=block, transposed=True)
    alone = qg.quantize_f8(x, block=block)
    for a, b in zip(got, alone):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    back = qg.dequant_f8(*alone, BF, block=block)
    for r0 in (0, 128 * 700, 128 * 2047, 128 * 2048):        # whole blocks of rows, the last one short
        part = x[r0:r0 + 128].double().cpu().numpy()
        codes, scales = ref.quantize(part, block)
        assert np.array_equal(alone[0][r0:r0 + 128].view(torch.uint8).cpu().numpy(), codes)
        mine = alone[1][:, r0:r0 + 128] if block == 1 else alone[1][r0 // 128:r0 // 128 + 1]
        assert np.array_equal(mine.double().cpu().numpy(), scales)
        assert torch.equal(back[r0:r0 + 128].cpu(), torch.from_numpy(ref.values(codes, scales, block)).to(BF))
    for c0 in (0, 128 * 63, 128 * 64):
        part = ref.pad16(x[:, c0:c0 + 128].double().cpu().numpy().T[:(16 if block == 1 else 128)])
        codes, scales = ref.quantize(part, block)
        assert np.array_equal(got[2][c0:c0 + len(part)].view(torch.uint8).cpu().numpy(), codes)
        mine = got[3][:, c0:c0 + len(part)] if block == 1 else got[3][c0 // 128:c0 // 128 + 1]
        assert np.array_equal(mine.double().cpu().numpy(), scales)
