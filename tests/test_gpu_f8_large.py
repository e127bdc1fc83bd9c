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
