"""MX4 products at the ends of their ranges: values and scales, long k on the
streaming kernel, long k by expert, forced tiles that do not fit."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
import weight_only_quantized_w8a16_amd as qg

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
