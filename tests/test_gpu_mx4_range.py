"""MX4 products at the ends of their ranges: values and scales, long k on the
streaming kernel, long k by expert, forced tiles that do not fit."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
import weight_only_quantized_w8a16_amd as qg
from test_gpu_mx4 import exact_case, grouped_case, same, tiled, dev

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32
KERNELS = ["stream", "T256", "T256N", "T128", "T64", "T32"]


def test_forced_tile_past_a_launch_is_ignored():
    # 4096 x 2049 tiles of 32 x 64, 512 threads each, are more than 2^32 - 1
    # threads: the forced choice does not fit and the automatic one runs
    m, n, k = 131072, 64 * 2049, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    A = torch.empty(m, k, dtype=BF, device="cuda").random_(-4, 5, generator=g)
    c = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.randint(124, 127, (n // 16, 1, 64, 4), dtype=torch.uint8, device="cuda", generator=g)
    qg.set_override(mx4_tile="T32")
    C = qg.gemm_mx4a16(A, c, s)
    rows = [0, 1, 31, 32, m // 2, m - 33, m - 1]
    w = qg.dequant_mx4(c, s, tiled=True)
    # integers times values of step 2^-4, |sum| <= 128 * 4 * 3: exact in fp32 in
    # any order, so the fp32 product is the same before its one rounding
    assert torch.equal(C[rows], (A[rows].float() @ w.t()).to(BF))


# -- values and scales -----------------------------------------------------------

# power of the activations, first scale byte; in fp16 the weights are rounded
@pytest.mark.parametrize("dtype,power,first", [
    (BF, 0, 0), (BF, 20, 0), (BF, 100, 0),            # subnormal weights; subnormal and normal results
    (BF, -130, 200), (BF, -24, 120),                  # subnormal activations
    (HF, 0, 100), (HF, 10, 100), (HF, 15, 100),       # weights below fp16's range, subnormal, and above
    (HF, -24, 120), (HF, -14, 127)])                  # subnormal activations; infinite weights
@pytest.mark.parametrize("kernel", KERNELS)
def test_a16_subnormal_and_extreme_values(kernel, dtype, power, first):
    """One activation of 2^power a row against every code and 32 scale bytes
    from `first` on.  One product a sum, the others zero (or NaN, where fp16
    makes the weight infinite): exact in fp32, so the result is the product
    rounded once, subnormal or not."""
    n, k = 256, 128
    codes = np.zeros((n, k), dtype=np.uint8)
    codes[:, 32:48] = np.arange(16)
    scales = np.full((n, 4), 127, dtype=np.uint8)
    scales[:, 1] = first + np.arange(n) % 32
    w = ref.rne(ref.values(codes, scales), dtype).double().numpy()
    A = torch.zeros(16, k, dtype=dtype)
    A[range(16), range(32, 48)] = 2.0 ** power
    with np.errstate(invalid="ignore"):               # zero times infinity
        c = A.double().numpy() @ w.T
    qg.set_override(mx4_tile=kernel)
    got = qg.gemm_mx4a16(A.cuda(), *tiled(codes, scales)).cpu()
    want = ref.rne(c, dtype)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(1.0), want.nan_to_num(1.0))


@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("kernel", KERNELS)
def test_a4_every_pair_of_scales(kernel, dtype):
    """1.5 * 2^(sa - 127) times 3 * 2^(sb - 127) for every two scale bytes: one
    rounding to fp32 (to infinity above its range, subnormal or zero below it)
    and one to the output type."""
    m = n = 256
    k = 128
    ac, bc = np.zeros((m, k), dtype=np.uint8), np.zeros((n, k), dtype=np.uint8)
    ac[:, 32], bc[:, 32] = 3, 5
    sa, sb = np.full((m, 4), 127, dtype=np.uint8), np.full((n, 4), 127, dtype=np.uint8)
    sa[:, 1], sb[:, 1] = np.arange(m), np.arange(n)
    c = np.ldexp(4.5, (np.arange(m) - 127)[:, None] + (np.arange(n) - 127))
    c[255, :], c[:, 255] = np.nan, np.nan
    qg.set_override(mx4_tile=kernel)
    got = qg.gemm_mx4a4(*tiled(ac, sa), *tiled(bc, sb), m=m, out_dtype=dtype)
    same(got, ref.rne(c, SF).to(dtype))


@pytest.mark.parametrize("kernel", KERNELS)
def test_a4_scales_far_apart_and_opposite(kernel):
    """Row r's scales grow by 2^d where column r's shrink by it: on the diagonal
    every product is a plain one, and the sum exact (steps of 2^-2, at most
    36 * 128)."""
    m = n = 240
    k = 128
    rng = np.random.default_rng(13)
    ac = rng.integers(0, 16, (m, k), dtype=np.uint8)
    bc = rng.integers(0, 16, (n, k), dtype=np.uint8)
    d = rng.integers(-127, 128, (m, 4))
    sa, sb = (127 + d).astype(np.uint8), (127 - d).astype(np.uint8)
    qg.set_override(mx4_tile=kernel)
    got = qg.gemm_mx4a4(*tiled(ac, sa), *tiled(bc, sb), m=m, out_dtype=SF)
    c = (ref.TABLE[ac] * ref.TABLE[bc]).sum(1)
    assert torch.equal(got.diagonal().cpu(), ref.rne(c, SF))


# -- long k ------------------------------------------------------------------------

def stream_case(rng, m, n, k, act):
    """exact_case; with MX4 activations its sums go in steps of 2^-4 and reach
    12 * 6 * k, which has to stay below 2^20."""
    assert act == "a16" or 72 * k < 2 ** 20
    return exact_case(rng, m, n, k, act)


def both_products(rng, m, n, k):
    codes, scales, _, _, a, w, bias, c = stream_case(rng, m, n, k, "a16")
    B, bias_d = qg.repack_mx4(dev(ref.pack(codes)), dev(scales)), dev(bias).to(BF)
    for dtype in (BF, HF):
        same(qg.gemm_mx4a16(torch.from_numpy(a).to(dtype).cuda(), *B, bias=bias_d), ref.rne(c + bias, dtype))
    codes, scales, ac, asc, a, w, bias, c = stream_case(rng, m, n, k, "a4")
    B = qg.repack_mx4(dev(ref.pack(codes)), dev(scales))
    same(qg.gemm_mx4a4(*tiled(ac, asc), *B, m=m, out_dtype=SF), ref.rne(c, SF))


@pytest.mark.parametrize("k", [1152, 2176, 3584, 4224])
@pytest.mark.parametrize("n", [272, 3584])
@pytest.mark.parametrize("m", [1, 7, 16])
def test_streaming_long_k_exact_sums(m, n, k):
    """One column tile a workgroup: more 128-k blocks than its eight waves take
    in one pass of two, the last pass not all there."""
    qg.set_override(mx4_tile="stream")
    both_products(np.random.default_rng(m + n + k), m, n, k)


@pytest.mark.parametrize("rounds", [2, 3, 4, 5, 6])
def test_streaming_wide_long_k_exact_sums(rounds):
    """More column tiles a workgroup, one block of each wave at a time."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    qg.set_override(mx4_tile="stream")
    both_products(np.random.default_rng(rounds), 5, 16 * (cus * rounds - 3), 1152)


def grouped_matches(sizes, n, k, dtypes=(BF, HF)):
    a, off, B, S, bias, c = grouped_case(np.random.default_rng(n + k), sizes, n, k, 1, 2)
    for dtype in dtypes:
        out = torch.full((a.shape[0], n), 9.0, dtype=dtype, device="cuda")
        qg.gemm_mx4a16_grouped(torch.from_numpy(a).to(dtype).cuda(), off, B, S, dev(bias).to(BF), out=out)
        same(out, ref.rne(c, dtype))   # rows of no expert keep their 9


@pytest.mark.parametrize("n,k", [(272, 1152), (272, 2176), (272, 3584), (2400, 1152), (4368, 1152)])
def test_grouped_streaming_long_k_exact_sums(n, k):
    # one, two and four column tiles a workgroup
    qg.set_override(mx4_tile="stream")
    grouped_matches([3, 0, 17, 1], n, k)


@pytest.mark.parametrize("k", [1152, 2048, 3584])
@pytest.mark.parametrize("kernel", KERNELS[1:5])
def test_grouped_tiles_long_k_exact_sums(kernel, k):
    qg.set_override(mx4_tile=kernel)
    grouped_matches([140, 0, 70, 1], 272, k)
