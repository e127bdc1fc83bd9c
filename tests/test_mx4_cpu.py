"""MX4 operators without a GPU: arguments refused on the host (these calls
never reach a launch) and the reference forms themselves."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
import weight_only_quantized_w8a16_amd as qg

OK, NULL, SHAPE, GROUP, DTYPE, ALIGN, WORKSPACE, UNSUP, HIP, MODE = range(10)
FAKE = 0x100000          # 16-byte-aligned stand-in address; never dereferenced
BF16, FP16, FP32 = 1, 2, 3


def quant(**kw):
    a = dict(X=FAKE, c=FAKE, s=FAKE, rows=3, k=256, layout=0, dt=BF16)
    a.update(kw)
    return qg.lib().qquantize_mx4(a["X"], a["c"], a["s"], a["rows"], a["k"], a["layout"], a["dt"], None)


def dequant(**kw):
    a = dict(X=FAKE, c=FAKE, s=FAKE, rows=3, k=256, layout=0, dt=BF16)
    a.update(kw)
    return qg.lib().qdequant_mx4(a["c"], a["s"], a["X"], a["rows"], a["k"], a["layout"], a["dt"], None)


CONVERT = [
    (dict(rows=-1), SHAPE), (dict(k=-32), SHAPE), (dict(X=None), NULL), (dict(c=None), NULL),
    (dict(s=None), NULL), (dict(dt=0), DTYPE), (dict(dt=9), DTYPE), (dict(layout=2), MODE),
    (dict(layout=-1), MODE), (dict(k=48), UNSUP), (dict(k=160, layout=1), UNSUP),
    (dict(X=FAKE + 8), ALIGN), (dict(c=FAKE + 8), ALIGN), (dict(s=FAKE + 2, layout=1), ALIGN),
    (dict(rows=0, X=None), OK), (dict(k=0, c=None), OK),
]


@pytest.mark.parametrize("kw,status", CONVERT)
def test_conversion_refusals(kw, status):
    assert quant(**kw) == status
    assert dequant(**kw) == status


@pytest.mark.parametrize("fn", ["qrepack_mx4", "qunrepack_mx4"])
@pytest.mark.parametrize("args,status", [
    ((FAKE, FAKE, FAKE, FAKE, -1, 128), SHAPE), ((None, FAKE, FAKE, FAKE, 1, 128), NULL),
    ((FAKE, None, FAKE, FAKE, 1, 128), NULL), ((FAKE, FAKE, None, FAKE, 1, 128), NULL),
    ((FAKE, FAKE, FAKE, None, 1, 128), NULL), ((FAKE, FAKE, FAKE, FAKE, 1, 96), UNSUP),
    ((FAKE + 8, FAKE, FAKE, FAKE, 1, 128), ALIGN), ((FAKE, FAKE, FAKE + 8, FAKE, 1, 128), ALIGN),
    ((None, None, None, None, 0, 128), OK),
])
def test_repack_refusals(fn, args, status):
    assert getattr(qg.lib(), fn)(*args, None) == status


def a16(**kw):
    a = dict(A=FAKE, B=FAKE, s=FAKE, bias=None, C=FAKE, m=4, n=32, k=256, act=BF16, bdt=0, ws=None, wsb=0)
    a.update(kw)
    return qg.lib().qgemm_mx4a16(a["A"], a["B"], a["s"], a["bias"], a["C"], a["m"], a["n"], a["k"],
                                 a["act"], a["bdt"], a["ws"], a["wsb"], None)


def a4(**kw):
    a = dict(A=FAKE, AS=FAKE, B=FAKE, s=FAKE, bias=None, C=FAKE, m=4, n=32, k=256, act=BF16, bdt=0,
             ws=None, wsb=0)
    a.update(kw)
    return qg.lib().qgemm_mx4a4(a["A"], a["AS"], a["B"], a["s"], a["bias"], a["C"], a["m"], a["n"],
                                a["k"], a["act"], a["bdt"], a["ws"], a["wsb"], None)


def grouped(**kw):
    a = dict(A=FAKE, off=FAKE, B=FAKE, s=FAKE, bias=None, C=FAKE, m=4, n=32, k=256, E=3, act=BF16, bdt=0)
    a.update(kw)
    return qg.lib().qgemm_mx4a16_grouped(a["A"], a["off"], a["B"], a["s"], a["bias"], a["C"], a["m"],
                                         a["n"], a["k"], a["E"], a["act"], a["bdt"], None)


PRODUCT = [
    (dict(m=-1), SHAPE), (dict(n=-16), SHAPE), (dict(k=0), SHAPE), (dict(A=None), NULL),
    (dict(B=None), NULL), (dict(s=None), NULL), (dict(C=None), NULL), (dict(bdt=BF16), NULL),
    (dict(act=0), DTYPE), (dict(act=4), DTYPE), (dict(bias=FAKE, bdt=0), DTYPE),
    (dict(bias=FAKE, bdt=FP32), DTYPE), (dict(n=24), UNSUP), (dict(k=192), UNSUP),
    (dict(A=FAKE + 8), ALIGN), (dict(B=FAKE + 8), ALIGN), (dict(C=FAKE + 8), ALIGN),
    (dict(s=FAKE + 2), ALIGN), (dict(bias=FAKE + 1, bdt=BF16), ALIGN),
    (dict(m=0, A=None), OK), (dict(n=0, B=None), OK),
]


@pytest.mark.parametrize("kw,status", PRODUCT)
def test_product_refusals(kw, status):
    assert a16(**kw) == status
    assert a4(**kw) == status
    assert grouped(**kw) == status


@pytest.mark.parametrize("fn,kw,status", [
    (a16, dict(act=FP32), DTYPE), (grouped, dict(act=FP32), DTYPE), (a4, dict(AS=None), NULL),
    (a4, dict(AS=FAKE + 2), ALIGN), (a16, dict(ws=FAKE + 16, wsb=4096), ALIGN),
    (a4, dict(ws=FAKE + 16, wsb=4096), ALIGN), (grouped, dict(off=None), NULL),
    (grouped, dict(off=FAKE + 2), ALIGN), (grouped, dict(E=0), SHAPE), (grouped, dict(E=-1), SHAPE),
    (grouped, dict(E=65537), UNSUP),
])
def test_product_refusals_of_one_form(fn, kw, status):
    assert fn(**kw) == status


@pytest.mark.parametrize("args", [(0, 64, 128, 16), (4, 0, 128, 16), (4, 64, 0, 16), (4, 24, 128, 16),
                                  (4, 64, 96, 4), (4, 64, 128, 8)])
def test_workspace_size_of_refused_problems_is_zero(args):
    assert qg.mx4_workspace_size(*args) == 0


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


@pytest.mark.parametrize("call", [
    lambda: qg.quantize_mx4(torch.zeros(2, 64, dtype=torch.float64)),
    lambda: qg.quantize_mx4(torch.zeros(2, 48)),
    lambda: qg.quantize_mx4(torch.zeros(2, 160), tiled=True),
    lambda: qg.quantize_mx4(torch.zeros(2, 64)),                                 # not on the device
    lambda: qg.dequant_mx4(u8(2, 32), u8(2, 3)),
    lambda: qg.dequant_mx4(u8(2, 32), u8(2, 2), torch.int8),
    lambda: qg.dequant_mx4(u8(2, 32), u8(2, 2), rows=3),
    lambda: qg.dequant_mx4(u8(24, 64), u8(2, 1, 64, 4), tiled=True),
    lambda: qg.repack_mx4(u8(4, 32), u8(4, 2)),                                  # k = 64
    lambda: qg.unrepack_mx4(u8(16, 64), u8(1, 2, 64, 4)),
    lambda: qg.gemm_mx4a16(torch.zeros(2, 128), u8(16, 64), u8(1, 1, 64, 4)),    # fp32 A
    lambda: qg.gemm_mx4a16(torch.zeros(2, 256).half(), u8(16, 64), u8(1, 1, 64, 4)),
    lambda: qg.gemm_mx4a16(torch.zeros(2, 128).half(), u8(24, 64), u8(1, 1, 64, 4)),
    lambda: qg.gemm_mx4a16(torch.zeros(2, 128).half(), u8(16, 64), u8(1, 1, 64, 4),
                           bias=torch.zeros(8).half()),
    lambda: qg.gemm_mx4a16(torch.zeros(2, 128).half(), u8(16, 64), u8(1, 1, 64, 4),
                           out=torch.zeros(2, 16)),
    lambda: qg.gemm_mx4a4(u8(16, 64), u8(1, 1, 64, 4), u8(16, 128), u8(1, 1, 64, 4)),
    lambda: qg.gemm_mx4a4(u8(16, 64), u8(1, 1, 64, 4), u8(16, 64), u8(1, 1, 64, 4), m=17),
    lambda: qg.gemm_mx4a4(u8(16, 64), u8(1, 1, 64, 4), u8(16, 64), u8(1, 1, 64, 4),
                          out_dtype=torch.float64),
    lambda: qg.gemm_mx4a16_grouped(torch.zeros(2, 128).half(), torch.zeros(3, dtype=torch.int64),
                                   u8(2, 16, 64), u8(2, 1, 1, 64, 4)),
    lambda: qg.gemm_mx4a16_grouped(torch.zeros(2, 128).half(), torch.zeros(4, dtype=torch.int32),
                                   u8(2, 16, 64), u8(2, 1, 1, 64, 4)),
    lambda: qg.gemm_mx4a16_grouped(torch.zeros(2, 128).half(), torch.zeros(3, dtype=torch.int32),
                                   u8(2, 16, 64), u8(2, 1, 1, 64, 4), bias=torch.zeros(2, 8).half()),
])
def test_wrapper_refusals(call):
    with pytest.raises(qg.QGemmError):
        call()


@pytest.mark.parametrize("call", [
    lambda e: qg.quantize_mx4(e(1, 2 ** 32 + 128, dtype=torch.bfloat16), tiled=True),
    lambda e: qg.quantize_mx4(e(2 ** 32 + 1, 32, dtype=torch.float16)),
    lambda e: qg.dequant_mx4(e(1, 2 ** 31 + 64, dtype=torch.uint8), e(1, 2 ** 27 + 4, dtype=torch.uint8)),
    lambda e: qg.repack_mx4(e(2 ** 32 + 16, 64, dtype=torch.uint8), e(2 ** 32 + 16, 4, dtype=torch.uint8)),
    lambda e: qg.gemm_mx4a16(e(2 ** 32 + 1, 128, dtype=torch.float16), e(16, 64, dtype=torch.uint8),
                             e(1, 1, 64, 4, dtype=torch.uint8)),
    lambda e: qg.gemm_mx4a16_grouped(e(4, 128, dtype=torch.float16), e(65538, dtype=torch.int32),
                                     e(65537, 16, 64, dtype=torch.uint8),
                                     e(65537, 1, 1, 64, 4, dtype=torch.uint8)),
])
def test_sizes_past_the_librarys(call):
    # sizes that a 32-bit integer would wrap (no memory behind them)
    with pytest.raises(qg.QGemmError) as e:
        call(lambda *shape, dtype: torch.empty(shape, dtype=dtype, device="meta"))
    assert e.value.status == 7


def test_workspace_size_of_unusable_sizes():
    for m, n, k, bits in [(2 ** 31 - 1, 256, 4096, 16), (64, 256, 2 ** 31 - 128, 4), (0, 256, 4096, 16),
                          (64, 250, 4096, 16), (64, 256, 4096, 8), (2 ** 31 - 1, 256, 4096, 4)]:
        assert qg.mx4_workspace_size(m, n, k, bits) == 0


def test_reference_quantizer_examples():
    # one block: largest 7 -> scale 2^0; ties go to the even code
    x = np.zeros((1, 32))
    x[0, :12] = [7.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, -6.5, 0.26, -5.01]
    c, s = ref.quantize(x)
    assert s[0, 0] == 127
    assert list(ref.values(c, s)[0, :12]) == [6, 4, 4, 2, 2, 1, 1, 0, 0, -6, 0.5, -6]
    assert c[0, 8] == 8                                     # the sign of -0.25 stays
    assert ref.quantize(np.zeros((1, 32)))[1][0, 0] == 0
    x[0, 3] = np.nan
    c, s = ref.quantize(x)
    assert s[0, 0] == 255 and not c.any()


def test_reference_layout_round_trip():
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 16, (16, 256), dtype=np.uint8)
    tc, ts = ref.tile(codes, rng.integers(0, 255, (16, 8), dtype=np.uint8))
    # lane 16 j + nl of block kb: bytes of row nl, k 128 kb + 32 j ..
    assert np.array_equal(tc.reshape(2, 64, 16)[1, 16 * 2 + 5], ref.pack(codes[5:6, 128 + 64:128 + 96])[0])
    assert ts.shape == (1, 1, 64, 4) and not ts[..., 2:].any()
