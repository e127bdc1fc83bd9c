"""MX4 operators on the GPU against plain 64-bit forms (mx4_ref): conversions
bit for bit, products bit for bit on inputs whose sums are exact in fp32 and
within the rounding bound on random ones."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
import weight_only_quantized_w8a16_amd as qg

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


def host(t):
    return t.detach().double().cpu().numpy()


def same(t, expect):
    """Equal values, NaN equal to NaN, and equal signs (of zeros too)."""
    got, expect = t.detach().cpu(), expect.to(t.dtype)
    nan = torch.isnan(expect)
    assert torch.equal(torch.isnan(got), nan)
    a, b = got.masked_fill(nan, 0), expect.masked_fill(nan, 0)
    assert torch.equal(a, b) and torch.equal(torch.signbit(a), torch.signbit(b))


def random_weight(rng, n, k, lo=118, hi=124):
    """Packed-free MX4 weight: codes 0..15 and scale bytes in [lo, hi]."""
    return (rng.integers(0, 16, (n, k), dtype=np.uint8),
            rng.integers(lo, hi + 1, (n, k // 32), dtype=np.uint8))


def tiled(codes, scales):
    tc, ts = ref.tile(codes, scales)
    return dev(tc), dev(ts)


# -- conversions -----------------------------------------------------------------

def block_inputs(rng, rows, k, dtype):
    """Rows over many magnitudes, with ties, zeros, tiny and huge blocks."""
    x = rng.standard_normal((rows, k)) * np.exp2(rng.integers(-12, 13, (rows, k // 32)).repeat(32, 1))
    t = torch.from_numpy(x).to(dtype)
    b = t.view(rows, k // 32, 32)
    fi = torch.finfo(dtype)
    for i, blk in enumerate(b.view(-1, 32)):
        kind = i % 11
        if kind == 1:
            blk.zero_()
            blk[3] = -0.0
        elif kind == 2:   # ties: quarters and halves of the grid
            blk.copy_(torch.from_numpy(rng.integers(-32, 33, 32) / 4.0).to(dtype))
        elif kind == 3:
            blk.mul_(0).add_(fi.max)
            blk[5] = -fi.max
        elif kind == 4:   # the smallest numbers, subnormal ones among them
            blk.copy_(torch.from_numpy(rng.integers(-9, 10, 32).astype(np.float64) *
                                       float(fi.smallest_normal) * fi.eps).to(dtype))
        elif kind == 5:
            blk.copy_(torch.from_numpy(rng.standard_normal(32) * float(fi.smallest_normal) * 4).to(dtype))
    return t


def spoil(t):
    """A NaN, an infinity of each sign, one per chosen block."""
    b = t.view(-1, 32)
    for i, v in ((0, float("nan")), (1, float("inf")), (2, float("-inf"))):
        if i < b.shape[0]:
            b[i, (7 * i + 31) % 32] = v
    return t


@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("rows,k", [(1, 32), (3, 96), (5, 1152), (64, 256), (1, 8192)])
def test_quantize_portable_bit_exact(dtype, rows, k):
    for bad in (False, True):
        x = block_inputs(np.random.default_rng(rows * k), rows, k, dtype)
        if bad:
            x = spoil(x)
        codes, scales = qg.quantize_mx4(x.cuda())
        c, s = ref.quantize(x.double().numpy())
        assert np.array_equal(scales.cpu().numpy(), s)
        assert np.array_equal(codes.cpu().numpy(), ref.pack(c))


@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("rows,k", [(1, 128), (15, 640), (16, 512), (17, 1152), (100, 384)])
def test_quantize_tiled_bit_exact(dtype, rows, k):
    x = spoil(block_inputs(np.random.default_rng(rows * k), rows, k, dtype))
    codes, scales = qg.quantize_mx4(x.cuda(), tiled=True)
    tc, ts = ref.tile(*ref.quantize(x.double().numpy()))
    assert np.array_equal(scales.cpu().numpy(), ts)
    assert np.array_equal(codes.cpu().numpy(), tc)


@pytest.mark.parametrize("dtype", [BF, HF, SF])
def test_dequant_every_code_and_scale(dtype):
    # row s: scale byte s, every code in both nibbles
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 8))
    codes[:, 64:] = codes[:, 64:][:, ::-1]
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 4, 1)
    want = torch.from_numpy(ref.values(codes, scales))
    same(qg.dequant_mx4(dev(ref.pack(codes)), dev(scales), dtype), want.to(dtype))
    same(qg.dequant_mx4(*tiled(codes, scales), dtype, tiled=True), want.to(dtype))


@pytest.mark.parametrize("rows,k", [(1, 128), (19, 640), (32, 1536)])
def test_repack_formula_and_inverse(rows, k):
    codes, scales = random_weight(np.random.default_rng(k), rows, k, 0, 255)
    c, s = dev(ref.pack(codes)), dev(scales)
    tc, ts = qg.repack_mx4(c, s)
    wc, ws = ref.tile(codes, scales)
    assert np.array_equal(tc.cpu().numpy(), wc) and np.array_equal(ts.cpu().numpy(), ws)
    uc, us = qg.unrepack_mx4(tc, ts, rows)
    assert torch.equal(uc, c) and torch.equal(us, s)
    want = torch.from_numpy(ref.values(codes, scales))
    same(qg.dequant_mx4(tc, ts, SF, tiled=True, rows=rows), want.float())
    same(qg.dequant_mx4(c, s, SF), want.float())


def test_conversions_leave_neighbours_alone():
    # outputs are slices of larger buffers; the rows around them stay
    rows, k = 5, 256
    x = torch.randn(rows, k, device="cuda", dtype=BF)
    out = torch.full((rows + 2, k), 7.0, device="cuda", dtype=BF)
    codes, scales = qg.quantize_mx4(x, tiled=True)
    L = qg.lib()
    assert L.qdequant_mx4(codes.data_ptr(), scales.data_ptr(), out[1:].data_ptr(), rows, k, 1, 1,
                          torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert bool((out[0] == 7).all()) and bool((out[-1] == 7).all())
    assert torch.equal(out[1:-1], qg.dequant_mx4(codes, scales, BF, tiled=True, rows=rows))


# -- products ----------------------------------------------------------------------

# m, n, k: one row to several row tiles, one column tile to several, odd counts
# of both, every remainder of k modulo 512
KERNELS = ["stream", "T256", "T256N", "T128", "T64", "T32"]
SHAPES = [(1, 16, 128), (1, 2048, 2048), (2, 48, 256), (3, 80, 384), (16, 272, 640), (17, 96, 512),
          (31, 528, 896), (64, 144, 1152), (100, 400, 1024), (129, 656, 768), (300, 272, 1664)]


def exact_case(rng, m, n, k, act):
    """Small integers times grid values: every partial sum is a multiple of
    2^-3 below 2^24 * 2^-3, so fp32 sums are exact in any order."""
    codes, scales = random_weight(rng, n, k, 125, 127)
    if act == "a4":
        ac, asc = random_weight(rng, m, k, 127, 128)
        a = ref.values(ac, asc)
    else:
        ac = asc = None
        a = rng.integers(-4, 5, (m, k)).astype(np.float64)
    bias = rng.integers(-8, 9, n).astype(np.float64)
    w = ref.values(codes, scales)
    c = a @ w.T
    assert (np.abs(a) @ np.abs(w).T).max() < 2 ** 21 - 16
    return codes, scales, ac, asc, a, w, bias, c


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_a16_exact_sums(m, n, k, dtype):
    codes, scales, _, _, a, w, bias, c = exact_case(np.random.default_rng(m + n + k), m, n, k, "a16")
    B = tiled(codes, scales)
    A = torch.from_numpy(a).to(dtype).cuda()
    same(qg.gemm_mx4a16(A, *B), ref.rne(c, dtype))
    out = torch.full((m, n), float("nan"), dtype=dtype, device="cuda")
    got = qg.gemm_mx4a16(A, *B, bias=dev(bias).to(HF), out=out)
    assert got.data_ptr() == out.data_ptr()
    same(out, ref.rne(c + bias, dtype))


@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_a4_exact_sums(m, n, k, dtype):
    codes, scales, ac, asc, a, w, bias, c = exact_case(np.random.default_rng(m + n + k), m, n, k, "a4")
    A, B = tiled(ac, asc), tiled(codes, scales)
    same(qg.gemm_mx4a4(*A, *B, m=m, out_dtype=dtype), ref.rne(c, dtype))
    out = torch.full((m, n), float("nan"), dtype=dtype, device="cuda")
    qg.gemm_mx4a4(*A, *B, m=m, bias=dev(bias).to(BF), out=out)
    same(out, ref.rne(c + bias, dtype))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k", [(1, 272, 2048), (7, 528, 1408), (33, 144, 3584), (150, 400, 512)])
def test_a16_random_within_rounding(m, n, k, dtype):
    rng = np.random.default_rng(k)
    A = torch.from_numpy(rng.standard_normal((m, k))).to(dtype)
    codes, scales = random_weight(rng, n, k)
    bias = torch.from_numpy(0.1 * rng.standard_normal(n)).to(dtype)
    a, w = A.double().numpy(), ref.values(codes, scales)
    c = a @ w.T + bias.double().numpy()
    got = host(qg.gemm_mx4a16(A.cuda(), *tiled(codes, scales), bias=bias.cuda()))
    assert (np.abs(got - c) <= ref.product_bound(a, w, c, dtype)).all()


@pytest.mark.parametrize("dtype", [BF, SF])
@pytest.mark.parametrize("m,n,k", [(1, 272, 2048), (7, 528, 1408), (33, 144, 3584), (150, 400, 512)])
def test_a4_random_within_rounding(m, n, k, dtype):
    # quantised on the way in, scales of both operands far apart
    rng = np.random.default_rng(k + 1)
    x = torch.from_numpy(rng.standard_normal((m, k)) * np.exp2(rng.integers(-6, 7, (m, k // 32)).repeat(32, 1)))
    x = x.to(BF)
    codes, scales = random_weight(rng, n, k, 100, 124)
    a, w = ref.values(*ref.quantize(x.double().numpy())), ref.values(codes, scales)
    c = a @ w.T
    got = host(qg.gemm_mx4a4(*qg.quantize_mx4(x.cuda(), tiled=True), *tiled(codes, scales), m=m,
                             out_dtype=dtype))
    assert (np.abs(got - c) <= ref.product_bound(a, w, c, dtype)).all()


def test_a16_weight_extremes():
    # bf16: every finite scale byte, one live block per channel, one-hot
    # activations: C is the weight's own value.  fp16: the value rounded.
    n, k = 256, 128
    codes = np.zeros((n, k), dtype=np.uint8)
    codes[:, 32:64] = np.arange(32, dtype=np.uint8) % 16
    scales = np.full((n, 4), 127, dtype=np.uint8)
    scales[:, 1] = np.arange(n)
    w = ref.values(codes, scales)
    # limit: the last scale whose largest weight, 6 * 2^(s - 127), is finite in
    # dtype (below 2^128, below 65520); past it the channel holds infinities,
    # and those times the activations' zeros make NaN of all its outputs.
    for dtype, limit in ((BF, 252), (HF, 140)):
        A = torch.zeros(16, k, dtype=dtype)
        for r in range(16):
            A[r, 32 + r] = 1.0
        got = qg.gemm_mx4a16(A.cuda(), *tiled(codes, scales)).cpu()
        want = torch.from_numpy(w[:, 32:48].T.copy()).to(dtype)
        live = (torch.arange(n) <= limit).expand(16, n)
        fine = live & (want.abs().double() >= 2.0 ** -126)   # sums below may be flushed to zero
        assert torch.equal(got[fine], want[fine])
        assert bool((got[live & ~fine].float().abs() <= 2.0 ** -126).all())
        assert bool(torch.isnan(got[:, 255].float()).all())


def test_nan_scale_spoils_its_own_outputs_only():
    rng = np.random.default_rng(5)
    for m in (3, 200):
        codes, scales = random_weight(rng, 144, 640)
        scales[37, 13] = 255
        ac, asc = random_weight(rng, m, 640, 126, 127)
        asc[1, 3] = 255
        got = qg.gemm_mx4a4(*tiled(ac, asc), *tiled(codes, scales), m=m, out_dtype=SF)
        bad = torch.zeros(m, 144, dtype=torch.bool)
        bad[1], bad[:, 37] = True, True
        assert torch.equal(torch.isnan(got).cpu(), bad)
        A = torch.from_numpy(rng.standard_normal((m, 640))).to(BF)
        A[2, 5] = float("inf")
        got = qg.gemm_mx4a16(A.cuda(), *tiled(codes, scales)).cpu()
        assert bool(torch.isnan(got[:, 37]).all())
        rest = torch.cat([got[:, :37], got[:, 38:]], 1)
        assert bool(torch.isfinite(torch.cat([rest[:2], rest[3:]])).all())


def test_leading_dimensions_and_empty():
    rng = np.random.default_rng(9)
    B = tiled(*random_weight(rng, 64, 256))
    A = torch.randn(2, 3, 256, device="cuda", dtype=BF)
    C = qg.gemm_mx4a16(A, *B)
    assert C.shape == (2, 3, 64)
    assert torch.equal(C.reshape(6, 64), qg.gemm_mx4a16(A.reshape(6, 256), *B))
    assert qg.gemm_mx4a16(A[:0], *B).shape == (0, 3, 64)
    q = qg.quantize_mx4(A[0][:0], tiled=True)
    assert qg.gemm_mx4a4(*q, *B).shape == (0, 64)
    assert qg.dequant_mx4(*q, tiled=True).shape == (0, 256)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_every_kernel_exact_sums(m, n, k, kernel):
    # one kernel forced for sizes it would not be chosen for, too
    qg.set_override(mx4_tile=kernel)
    rng = np.random.default_rng(m + n + k)
    codes, scales, _, _, a, w, bias, c = exact_case(rng, m, n, k, "a16")
    for dtype in (BF, HF):
        got = qg.gemm_mx4a16(torch.from_numpy(a).to(dtype).cuda(), *tiled(codes, scales), bias=dev(bias).to(BF))
        same(got, ref.rne(c + bias, dtype))
    codes, scales, ac, asc, a, w, bias, c = exact_case(rng, m, n, k, "a4")
    for dtype in (BF, HF, SF):
        got = qg.gemm_mx4a4(*tiled(ac, asc), *tiled(codes, scales), m=m, bias=dev(bias).to(HF), out_dtype=dtype)
        same(got, ref.rne(c + bias, dtype))


@pytest.mark.parametrize("act", ["a16", "a4"])
def test_several_tiles_a_workgroup_exact_sums(act):
    """More tiles than workgroups run at a time, of every size: each walks
    over tile borders, the last rows and columns ragged."""
    m, n, k = 4100, 4368, 640
    codes, scales, ac, asc, a, w, bias, c = exact_case(np.random.default_rng(m), m, n, k, act)
    B, bias_d = qg.repack_mx4(dev(ref.pack(codes)), dev(scales)), dev(bias).to(BF)
    for kernel in KERNELS[1:]:
        qg.set_override(mx4_tile=kernel)
        if act == "a16":
            same(qg.gemm_mx4a16(torch.from_numpy(a).to(BF).cuda(), *B, bias=bias_d), ref.rne(c + bias, BF))
        else:
            A = qg.repack_mx4(dev(ref.pack(ac)), dev(asc))
            for dtype in (HF, SF):
                same(qg.gemm_mx4a4(*A, *B, m=m, bias=bias_d, out_dtype=dtype), ref.rne(c + bias, dtype))


@pytest.mark.parametrize("m,k", [(1, 128), (13, 640), (20, 384)])
@pytest.mark.parametrize("rounds", [1, 2, 3, 4, 5, 6, 7, 9, 11])
def test_streaming_every_width_exact_sums(rounds, m, k):
    """Column tiles for so many rounds of one per CU, so each number of column
    tiles a workgroup takes, the last workgroup's not all there."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    n = 16 * (cus * rounds // ((m + 15) // 16) - 1)
    qg.set_override(mx4_tile="stream")
    rng = np.random.default_rng(rounds * m)
    codes, scales, _, _, a, w, bias, c = exact_case(rng, m, n, k, "a16")
    B = qg.repack_mx4(dev(ref.pack(codes)), dev(scales))
    for dtype in (BF, HF):
        got = qg.gemm_mx4a16(torch.from_numpy(a).to(dtype).cuda(), *B, bias=dev(bias).to(BF))
        same(got, ref.rne(c + bias, dtype))
    codes, scales, ac, asc, a, w, bias, c = exact_case(rng, m, n, k, "a4")
    B = qg.repack_mx4(dev(ref.pack(codes)), dev(scales))
    for dtype in (BF, HF, SF):
        got = qg.gemm_mx4a4(*tiled(ac, asc), *B, m=m, bias=dev(bias).to(HF), out_dtype=dtype)
        same(got, ref.rne(c + bias, dtype))


@pytest.mark.parametrize("kernel", KERNELS[1:])
@pytest.mark.parametrize("m,n,k,slices", [(1, 16, 1024, 2), (70, 272, 1664, 4), (300, 144, 3584, 3)])
def test_k_slices_exact_sums(m, n, k, slices, kernel):
    # windows of 512 k shared out unevenly, the last slice and window partial;
    # with less workspace the same call runs unsplit, to the same bits
    qg.set_override(mx4_tile=kernel, mx4_split=slices)
    rng = np.random.default_rng(m + k)
    for act, bits in (("a16", 16), ("a4", 4)):
        codes, scales, ac, asc, a, w, bias, c = exact_case(rng, m, n, k, act)
        assert qg.mx4_workspace_size(m, n, k, bits) >= 2 * m * n * 4
        for ws in (None, torch.empty(0, dtype=torch.uint8, device="cuda")):
            if act == "a16":
                got = qg.gemm_mx4a16(torch.from_numpy(a).to(BF).cuda(), *tiled(codes, scales),
                                     bias=dev(bias).to(BF), workspace=ws)
            else:
                got = qg.gemm_mx4a4(*tiled(ac, asc), *tiled(codes, scales), m=m, bias=dev(bias).to(BF),
                                    workspace=ws)
            same(got, ref.rne(c + bias, BF))


# -- grouped -----------------------------------------------------------------------

SIZES = [[1], [0, 5, 0], [16, 0, 17, 1, 0], [3, 40, 130, 0, 0, 2], [0, 0, 0, 0],
         [1] * 70, [0] * 64 + [9] + [0] * 3 + [33], [260, 1, 129], [600, 0, 3]]


def grouped_case(rng, sizes, n, k, before=0, behind=0):
    E = len(sizes)
    codes, scales = random_weight(rng, E * n, k, 125, 127)
    off = before + np.concatenate([[0], np.cumsum(sizes)])
    rows = int(off[-1]) + behind
    a = rng.integers(-4, 5, (rows, k)).astype(np.float64)
    bias = rng.integers(-8, 9, (E, n)).astype(np.float64)
    w = ref.values(codes, scales).reshape(E, n, k)
    c = np.full((rows, n), 9.0)
    for e in range(E):
        c[off[e]:off[e + 1]] = a[off[e]:off[e + 1]] @ w[e].T + bias[e]
    B, S = qg.repack_mx4(dev(ref.pack(codes)), dev(scales))
    return (a, torch.from_numpy(off.astype(np.int32)).cuda(), B.view(E, n, k // 2),
            S.view(E, n // 16, -1, 64, 4), bias, c)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{sum(s)}")
@pytest.mark.parametrize("n,k,before,behind", [(48, 256, 0, 0), (272, 640, 3, 5)])
def test_grouped_exact_sums(sizes, n, k, before, behind, dtype):
    a, off, B, S, bias, c = grouped_case(np.random.default_rng(sum(sizes) + n), sizes, n, k, before, behind)
    A = torch.from_numpy(a).to(dtype).cuda()
    out = torch.full((a.shape[0], n), 9.0, dtype=dtype, device="cuda")
    got = qg.gemm_mx4a16_grouped(A, off, B, S, dev(bias).to(BF), out=out)
    assert got.data_ptr() == out.data_ptr()
    same(out, ref.rne(c, dtype))   # rows of no expert keep their 9


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("sizes", [SIZES[2], SIZES[3], SIZES[6], SIZES[7]], ids=lambda s: f"{len(s)}x{sum(s)}")
def test_grouped_every_kernel_exact_sums(sizes, kernel):
    qg.set_override(mx4_tile=kernel)
    a, off, B, S, bias, c = grouped_case(np.random.default_rng(len(sizes)), sizes, 272, 640, 2, 7)
    for dtype in (BF, HF):
        out = torch.full((a.shape[0], 272), 9.0, dtype=dtype, device="cuda")
        qg.gemm_mx4a16_grouped(torch.from_numpy(a).to(dtype).cuda(), off, B, S, dev(bias).to(BF), out=out)
        same(out, ref.rne(c, dtype))


@pytest.mark.parametrize("rows,kernel", [(150, "auto"), (1500, "auto"), (6000, "auto"), (6000, "T256")])
def test_grouped_many_experts(rows, kernel):
    """300 experts, most of them without rows, some with many."""
    qg.set_override(mx4_tile=kernel)
    rng = np.random.default_rng(rows)
    share = rng.exponential(size=300) ** 6
    sizes = rng.multinomial(rows, share / share.sum())
    a, off, B, S, bias, c = grouped_case(rng, sizes, 144, 128, 1, 1)
    out = torch.full((a.shape[0], 144), 9.0, dtype=BF, device="cuda")
    qg.gemm_mx4a16_grouped(torch.from_numpy(a).to(BF).cuda(), off, B, S, dev(bias).to(BF), out=out)
    same(out, ref.rne(c, BF))


def test_grouped_several_tiles_a_workgroup():
    n, k = 4368, 640
    a, off, B, S, bias, c = grouped_case(np.random.default_rng(8), [700, 0, 1500, 3, 900, 400], n, k, 2, 3)
    A = torch.from_numpy(a).to(BF).cuda()
    for kernel in KERNELS[1:5]:
        qg.set_override(mx4_tile=kernel)
        out = torch.full((a.shape[0], n), 9.0, dtype=BF, device="cuda")
        same(qg.gemm_mx4a16_grouped(A, off, B, S, dev(bias).to(BF), out=out), ref.rne(c, BF))


@pytest.mark.parametrize("kernel", KERNELS)
def test_grouped_bad_offsets_stay_inside(kernel):
    qg.set_override(mx4_tile=kernel)
    # decreasing and out-of-range offsets: nothing outside the rows is written
    n, k, rows = 48, 256, 40
    rng = np.random.default_rng(2)
    B, S = qg.repack_mx4(dev(ref.pack(random_weight(rng, 4 * n, k)[0])), dev(np.full((4 * n, k // 32), 120, np.uint8)))
    A = torch.randn(rows, k, device="cuda", dtype=BF)
    for off in ([0, 30, 10, 20, 40], [-5, 10, 2 ** 30, 7, 3], [2 ** 31 - 1, -2 ** 31, 50, 60, 70]):
        buf = torch.full((rows + 64, n), 9.0, dtype=BF, device="cuda")
        qg.gemm_mx4a16_grouped(A, torch.tensor(off, dtype=torch.int32, device="cuda"), B.view(4, n, -1),
                               S.view(4, n // 16, -1, 64, 4), out=buf[32:32 + rows])
        assert bool((buf[:32] == 9).all()) and bool((buf[32 + rows:] == 9).all())


# -- together ------------------------------------------------------------------------

def test_expert_layer():
    """Routed rows through gate/up and down experts, as a model runs them."""
    rng = np.random.default_rng(11)
    T, H, I, E, topk = 37, 256, 128, 6, 2
    x = torch.from_numpy(rng.standard_normal((T, H))).to(BF)
    w1 = torch.from_numpy(0.05 * rng.standard_normal((E * 2 * I, H))).to(BF)
    w2 = torch.from_numpy(0.05 * rng.standard_normal((E * H, I))).to(BF)
    ids = torch.from_numpy(np.stack([rng.permutation(E)[:topk] for _ in range(T)]))
    order = torch.argsort(ids.flatten(), stable=True)
    src = order // topk
    counts = torch.bincount(ids.flatten(), minlength=E)
    off = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).to(torch.int32)

    def weight(w):
        c, s = qg.quantize_mx4(w.cuda(), tiled=True)
        return c.view(E, -1, c.shape[1]), s.view(E, -1, *s.shape[1:])

    h = qg.gemm_mx4a16_grouped(x[src].cuda(), off.cuda(), *weight(w1))
    act = (torch.nn.functional.silu(h[:, :I].float()) * h[:, I:].float()).to(BF)
    y = qg.gemm_mx4a16_grouped(act, off.cuda(), *weight(w2))
    v1 = ref.values(*ref.quantize(w1.double().numpy())).reshape(E, 2 * I, H)
    v2 = ref.values(*ref.quantize(w2.double().numpy())).reshape(E, H, I)
    xs, hh, aa, yy = x[src].double().numpy(), host(h), host(act), host(y)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        c = xs[r] @ v1[e].T
        assert (np.abs(hh[r] - c) <= ref.product_bound(xs[r], v1[e], c, BF)).all()
        c = aa[r] @ v2[e].T
        assert (np.abs(yy[r] - c) <= ref.product_bound(aa[r], v2[e], c, BF)).all()


@pytest.mark.parametrize("m", [3, 96])
def test_captured_and_replayed(m):
    """Quantise, both products and the grouped one in a captured graph, with
    new inputs and eager work between the replays."""
    rng = np.random.default_rng(m)
    n, k = 208, 1152
    B = tiled(*random_weight(rng, n, k))
    Bg, Sg = B[0].unsqueeze(0).repeat(3, 1, 1), B[1].unsqueeze(0).repeat(3, 1, 1, 1, 1)
    x = torch.randn(m, k, device="cuda", dtype=BF)
    off = torch.tensor([0, 1, 1, m], dtype=torch.int32, device="cuda")

    def step():
        q = qg.quantize_mx4(x, tiled=True)
        return (*q, qg.gemm_mx4a4(*q, *B, m=m), qg.gemm_mx4a16(x, *B),
                qg.gemm_mx4a16_grouped(x, off, Bg, Sg), qg.dequant_mx4(*q, BF, tiled=True, rows=m))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for i in range(4):
        x.copy_(torch.randn(m, k, device="cuda", dtype=BF))
        off.copy_(torch.tensor([0, i % 2, min(2 * i, m), m], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)


def test_two_graphs_with_k_slices():
    """Two captured graphs of a product with K slices, replayed in turn and on
    two streams at once: neither's partials touch the other's."""
    rng = np.random.default_rng(21)
    m, n, k = 128, 256, 4096
    qg.set_override(mx4_tile="T64", mx4_split=3)
    assert qg.mx4_workspace_size(m, n, k, 16) > 0
    B = [tiled(*random_weight(rng, n, k)) for _ in range(2)]
    x = [torch.randn(m, k, device="cuda", dtype=BF) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i in range(2):
            qg.gemm_mx4a16(x[i], *B[i])
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            outs.append(qg.gemm_mx4a16(x[i], *B[i]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for r in range(4):
        for i in range(2):
            x[i].copy_(torch.randn(m, k, device="cuda", dtype=BF))
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i] if r % 2 else torch.cuda.current_stream()):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], qg.gemm_mx4a16(x[i], *B[i]))


# -- operands of 2 GiB and more --------------------------------------------------------

def some_rows(rows, *more):
    return sorted({0, 1, 255, 256, rows // 2, rows - 257, rows - 256, rows - 17, rows - 1, *more})


def device_weight(n, k, seed):
    """Random tiled codes and scales (bytes 124 .. 126) made on the device."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.randint(124, 127, (n // 16, (k + 511) // 512, 64, 4), dtype=torch.uint8, device="cuda", generator=g)
    return c, s


def device_rows(c, s, rows):
    """Their values in the given rows, fp64."""
    out = []
    for r in rows:
        t = r // 16
        v = qg.dequant_mx4(c[16 * t:16 * t + 16], s[t:t + 1], tiled=True)
        out.append(host(v)[r % 16])
    return np.stack(out)


def test_a16_activations_past_2gib():
    m, n, k = 65536 + 300, 80, 16384 + 128
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    A = torch.empty(m, k, dtype=BF, device="cuda").random_(-4, 5, generator=g)
    assert A.numel() * 2 > 2 ** 31
    B = device_weight(n, k, 6)
    C = qg.gemm_mx4a16(A, *B)
    r = some_rows(m)
    # |sum| <= k * 4 * 3 < 2^18 in steps of 2^-4: exact in fp32
    same(C[r], ref.rne(host(A[r]) @ device_rows(*B, range(n)).T, BF))


def test_a4_activations_past_2gib():
    m, n, k = 131072 + 300, 48, 32768 + 128
    A, B = device_weight(m + 4, k, 7), device_weight(n, k, 8)
    assert A[0].numel() > 2 ** 31
    C = qg.gemm_mx4a4(*A, *B, m=m, out_dtype=SF)
    most = (2 ** 31 - 1) // (k // 2) // 256 * 256   # rows of one launch
    r = some_rows(m, most - 1, most, most + 1)
    a, w = device_rows(*A, r), device_rows(*B, range(n))
    c = a @ w.T
    # products in steps of 2^-8, |sum| < 2^19: fp32 rounds each addition
    assert (np.abs(host(C[r]) - c) <= ref.product_bound(a, w, c, SF)).all()


@pytest.mark.parametrize("m", [1, 20])
def test_weights_past_2gib(m):
    n, k = 131072 + 48, 32768 + 128
    B = device_weight(n, k, 9)
    assert B[0].numel() > 2 ** 31
    r = some_rows(n)
    w = device_rows(*B, r)
    rng = np.random.default_rng(m)
    a = rng.integers(-4, 5, (m, k)).astype(np.float64)
    C = qg.gemm_mx4a16(torch.from_numpy(a).to(BF).cuda(), *B)
    same(C[:, r], ref.rne(a @ w.T, BF))   # |sum| < 2^19 in steps of 2^-4
    q = qg.quantize_mx4(torch.from_numpy(a).to(BF).cuda(), tiled=True)   # -4 .. 4 are codes' values
    C = qg.gemm_mx4a4(*q, *B, m=m)
    same(C[:, r], ref.rne(a @ w.T, BF))


def test_two_streams_at_once():
    rng = np.random.default_rng(3)
    B = tiled(*random_weight(rng, 512, 1024))
    x = [torch.randn(m, 1024, device="cuda", dtype=BF) for m in (5, 80)]
    want = [qg.gemm_mx4a16(a, *B) for a in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    got = []
    for s, a in zip(streams, x):
        with torch.cuda.stream(s):
            got.append([qg.gemm_mx4a16(a, *B) for _ in range(5)])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, t) for t in g)
