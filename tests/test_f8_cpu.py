"""F8 operators without a GPU: arguments refused on the host (these calls never
reach a launch) and the reference forms themselves."""
import numpy as np
import pytest
import torch

import f8_ref as ref
import weight_only_quantized_w8a16_amd as qg

OK, NULL, SHAPE, GROUP, DTYPE, ALIGN, WORKSPACE, UNSUP, HIP, MODE = range(10)
FAKE = 0x100000          # 256-byte-aligned stand-in address; never dereferenced
BF16, FP16, FP32 = 1, 2, 3
BIG = 2 ** 31 - 255


def quant(**kw):
    a = dict(X=FAKE, stack=1, rows=3, k=272, dt=BF16, block=1, Q=FAKE, S=FAKE, QT=None, ST=None)
    a.update(kw)
    return qg.lib().qquantize_f8(*(a[x] for x in ("X", "stack", "rows", "k", "dt", "block", "Q", "S", "QT", "ST")), None)


def dequant(**kw):
    a = dict(Q=FAKE, S=FAKE, X=FAKE, stack=1, rows=3, k=272, block=1, dt=BF16)
    a.update(kw)
    return qg.lib().qdequant_f8(*(a[x] for x in ("Q", "S", "X", "stack", "rows", "k", "block", "dt")), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), SHAPE), (dict(k=-16), SHAPE), (dict(stack=0), SHAPE), (dict(stack=2), SHAPE),
    (dict(X=None), NULL), (dict(Q=None), NULL), (dict(S=None), NULL), (dict(dt=0), DTYPE), (dict(dt=4), DTYPE),
    (dict(block=0), MODE), (dict(block=64), MODE), (dict(block=127, k=24), MODE), (dict(k=24), UNSUP),
    (dict(k=8), UNSUP), (dict(rows=BIG), UNSUP), (dict(X=FAKE + 8), ALIGN), (dict(Q=FAKE + 8), ALIGN),
    (dict(S=FAKE + 2), ALIGN), (dict(rows=0, X=None), OK), (dict(k=0, Q=None), OK),
])
def test_conversion_refusals(kw, status):
    assert quant(**kw) == status
    assert dequant(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(QT=FAKE), NULL), (dict(ST=FAKE), NULL), (dict(Q=None, S=None), NULL),
    (dict(QT=FAKE + 8, ST=FAKE), ALIGN), (dict(QT=FAKE, ST=FAKE + 2), ALIGN), (dict(k=2 ** 31 - 128), UNSUP),
])
def test_quantize_refusals(kw, status):
    assert quant(**kw) == status


def gemm(**kw):
    a = dict(A=FAKE, AS=FAKE, B=FAKE, BS=FAKE, bias=None, C=FAKE, m=4, n=32, k=272, block=128, out=BF16, bdt=0,
             ws=None, wsb=0)
    a.update(kw)
    return qg.lib().qgemm_f8(*(a[x] for x in ("A", "AS", "B", "BS", "bias", "C", "m", "n", "k", "block", "out", "bdt",
                                              "ws", "wsb")), None)


def grouped(**kw):
    a = dict(A=FAKE, AS=FAKE, off=FAKE, B=FAKE, BS=FAKE, bias=None, C=FAKE, m=4, n=32, k=272, E=3, out=BF16, bdt=0)
    a.update(kw)
    return qg.lib().qgemm_f8_grouped(*(a[x] for x in ("A", "AS", "off", "B", "BS", "bias", "C", "m", "n", "k", "E",
                                                      "out", "bdt")), None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), SHAPE), (dict(n=-16), SHAPE), (dict(k=0), SHAPE), (dict(A=None), NULL), (dict(AS=None), NULL),
    (dict(B=None), NULL), (dict(BS=None), NULL), (dict(C=None), NULL), (dict(bdt=BF16), NULL),
    (dict(out=0), DTYPE), (dict(out=4), DTYPE), (dict(bias=FAKE, bdt=0), DTYPE), (dict(bias=FAKE, bdt=FP32), DTYPE),
    (dict(n=24), UNSUP), (dict(k=40), UNSUP), (dict(m=BIG), UNSUP), (dict(n=2 ** 31 - 128), UNSUP),
    (dict(k=2 ** 31 - 128), UNSUP), (dict(A=FAKE + 8), ALIGN), (dict(B=FAKE + 8), ALIGN), (dict(C=FAKE + 8), ALIGN),
    (dict(AS=FAKE + 2), ALIGN), (dict(BS=FAKE + 2), ALIGN), (dict(bias=FAKE + 1, bdt=BF16), ALIGN),
    (dict(m=0, A=None), OK), (dict(n=0, B=None), OK),
])
def test_product_refusals(kw, status):
    assert gemm(**kw) == status
    assert grouped(**kw) == status


@pytest.mark.parametrize("fn,kw,status", [
    (gemm, dict(block=0), MODE), (gemm, dict(block=64, n=24), MODE), (gemm, dict(ws=FAKE + 16, wsb=4096), ALIGN),
    (grouped, dict(off=None), NULL), (grouped, dict(off=FAKE + 2), ALIGN), (grouped, dict(E=0), SHAPE),
    (grouped, dict(E=-1), SHAPE), (grouped, dict(E=65537), UNSUP),
])
def test_product_refusals_of_one_form(fn, kw, status):
    assert fn(**kw) == status


def gated(**kw):
    a = dict(A=FAKE, AS=FAKE, B=FAKE, BS=FAKE, H=FAKE, GU=None, m=4, inter=128, k=272, act=0, out=BF16)
    a.update(kw)
    return qg.lib().qgated_f8(*(a[x] for x in ("A", "AS", "B", "BS", "H", "GU", "m", "inter", "k", "act", "out")), None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), SHAPE), (dict(inter=-128), SHAPE), (dict(k=0), SHAPE), (dict(A=None), NULL), (dict(AS=None), NULL),
    (dict(B=None), NULL), (dict(BS=None), NULL), (dict(H=None), NULL), (dict(out=0), DTYPE), (dict(act=2), MODE),
    (dict(act=-1), MODE), (dict(inter=192), UNSUP), (dict(k=24), UNSUP), (dict(inter=2 ** 30), UNSUP),
    (dict(A=FAKE + 8), ALIGN), (dict(B=FAKE + 8), ALIGN), (dict(H=FAKE + 8), ALIGN), (dict(GU=FAKE + 8), ALIGN),
    (dict(AS=FAKE + 2), ALIGN), (dict(BS=FAKE + 2), ALIGN), (dict(m=0, A=None), OK), (dict(inter=0, B=None), OK),
])
def test_gated_refusals(kw, status):
    assert gated(**kw) == status


def backward(**kw):
    a = dict(dH=FAKE, GU=FAKE, XT=FAKE, XS=FAKE, WT=FAKE, WS=FAKE, dX=FAKE, dW=FAKE, m=4, inter=128, k=272, act=0,
             dt=BF16, dxt=BF16, dwt=FP32, ws=None, wsb=0)
    a.update(kw)
    return qg.lib().qgated_f8_backward(*(a[x] for x in ("dH", "GU", "XT", "XS", "WT", "WS", "dX", "dW", "m", "inter",
                                                        "k", "act", "dt", "dxt", "dwt", "ws", "wsb")), None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), SHAPE), (dict(inter=-128), SHAPE), (dict(k=0), SHAPE), (dict(dH=None), NULL), (dict(GU=None), NULL),
    (dict(XT=None), NULL), (dict(XS=None), NULL), (dict(WT=None), NULL), (dict(WS=None), NULL), (dict(dt=FP32), DTYPE),
    (dict(dxt=0), DTYPE), (dict(dwt=9), DTYPE), (dict(act=7), MODE), (dict(inter=64), UNSUP), (dict(k=40), UNSUP),
    (dict(dH=FAKE + 8), ALIGN), (dict(GU=FAKE + 8), ALIGN), (dict(XT=FAKE + 8), ALIGN), (dict(WT=FAKE + 8), ALIGN),
    (dict(dX=FAKE + 8), ALIGN), (dict(dW=FAKE + 8), ALIGN), (dict(XS=FAKE + 2), ALIGN), (dict(WS=FAKE + 2), ALIGN),
    (dict(), WORKSPACE), (dict(ws=FAKE, wsb=255), WORKSPACE), (dict(ws=FAKE + 16, wsb=1 << 30), ALIGN),
    (dict(m=0, dW=None, dH=None), OK), (dict(inter=0, dX=None), OK), (dict(dX=None, dW=None, dH=None), OK),
    # what a NULL result does not need is not looked at
    (dict(dX=None, WT=None, WS=None, dxt=0), WORKSPACE), (dict(dW=None, XT=None, XS=None, dwt=0), WORKSPACE),
])
def test_backward_refusals(kw, status):
    assert backward(**kw) == status


@pytest.mark.parametrize("args", [(0, 64, 128, 128), (4, 0, 128, 128), (4, 64, 0, 128), (4, 24, 128, 128),
                                  (4, 64, 24, 1), (4, 64, 128, 2), (2 ** 31, 64, 128, 1), (-1, 64, 128, 1)])
def test_workspace_size_of_refused_problems_is_zero(args):
    assert qg.f8_workspace_size(*args) == 0


@pytest.mark.parametrize("args", [(0, 128, 128), (4, 64, 128), (4, 128, 24), (4, 0, 128), (4, 128, 0), (-1, 128, 128),
                                  (4, 2 ** 30, 128)])
def test_backward_workspace_size_of_refused_problems_is_zero(args):
    assert qg.gated_f8_backward_workspace_size(*args) == 0
    assert qg.gated_f8_backward_workspace_size(4, 128, 272) > 0


def f8(*shape):
    return torch.zeros(shape, dtype=torch.uint8).view(torch.float8_e4m3fn)


def f32(*shape):
    return torch.zeros(shape)


A, AS = f8(2, 144), f32(2, 2)
B, BS = f8(32, 144), f32(1, 2)
W, WS = f8(256, 144), f32(2, 2)
DH, GU, XT, XS, WT, WTS = (f32(2, 128).half(), f32(2, 256).half(), f8(144, 16), f32(1, 144), f8(144, 256), f32(2, 2))


@pytest.mark.parametrize("call,status", [
    (lambda: qg.quantize_f8(torch.zeros(2, 64, dtype=torch.float64)), DTYPE),
    (lambda: qg.quantize_f8(f32(2, 24)), UNSUP),
    (lambda: qg.quantize_f8(f32(2, 32), block=32), MODE),
    (lambda: qg.quantize_f8(f32(32), block=128), SHAPE),
    (lambda: qg.quantize_f8(f32(2, 32)), NULL),                                # not on the device
    (lambda: qg.dequant_f8(A, f32(2, 3)), SHAPE),
    (lambda: qg.dequant_f8(A, AS.half()), DTYPE),
    (lambda: qg.dequant_f8(A, AS, torch.int8), DTYPE),
    (lambda: qg.dequant_f8(B, BS, block=1), SHAPE),
    (lambda: qg.dequant_f8(f8(2, 24), f32(1, 2)), UNSUP),
    (lambda: qg.dequant_f8(A.view(torch.uint8), AS), DTYPE),
    (lambda: qg.dequant_f8(f8(3, 2, 144), f32(2, 6)), SHAPE),
    (lambda: qg.gemm_f8(A, AS, f8(32, 128), f32(1, 1)), SHAPE),
    (lambda: qg.gemm_f8(A, AS, B, BS, b_block=1), SHAPE),
    (lambda: qg.gemm_f8(A, AS, B, BS, b_block=3), MODE),
    (lambda: qg.gemm_f8(A, AS, B, BS, bias=f32(32)), DTYPE),
    (lambda: qg.gemm_f8(A, AS, B, BS, bias=f32(16).half()), SHAPE),
    (lambda: qg.gemm_f8(A, AS, B, BS, out=f32(2, 16)), SHAPE),
    (lambda: qg.gemm_f8(A, AS, B, BS, out_dtype=torch.float64), DTYPE),
    (lambda: qg.gemm_f8(A, AS, B, BS), NULL),                                  # not on the device
    (lambda: qg.gemm_f8_grouped(A, AS, torch.zeros(3, dtype=torch.int64), f8(2, 32, 144), f32(2, 1, 2)), DTYPE),
    (lambda: qg.gemm_f8_grouped(A, AS, torch.zeros(4, dtype=torch.int32), f8(2, 32, 144), f32(2, 1, 2)), SHAPE),
    (lambda: qg.gemm_f8_grouped(A, AS, torch.zeros(1, dtype=torch.int32), f8(0, 32, 144), f32(0, 1, 2)), SHAPE),
    (lambda: qg.gemm_f8_grouped(A, AS, torch.zeros(3, dtype=torch.int32), f8(2, 32, 144), f32(2, 1, 2),
                                bias=f32(2, 16).half()), SHAPE),
    (lambda: qg.gated_f8(A, AS, W, WS, act="relu"), MODE),
    (lambda: qg.gated_f8(A, AS, f8(128, 144), f32(1, 2)), UNSUP),
    (lambda: qg.gated_f8(A, AS, f8(256, 128), f32(2, 1)), SHAPE),
    (lambda: qg.gated_f8(A, AS, W, WS, out=f32(2, 256)), SHAPE),
    (lambda: qg.gated_f8_backward(DH.float(), GU.float(), XT, XS, WT, WTS), DTYPE),
    (lambda: qg.gated_f8_backward(DH, GU.bfloat16(), XT, XS, WT, WTS), DTYPE),
    (lambda: qg.gated_f8_backward(DH, GU[:, :128], XT, XS, WT, WTS), SHAPE),
    (lambda: qg.gated_f8_backward(DH, GU, f8(144, 32), XS, WT, WTS), SHAPE),
    (lambda: qg.gated_f8_backward(DH, GU, f8(128, 16), f32(1, 128), WT, WTS), SHAPE),
    (lambda: qg.gated_f8_backward(DH, GU, XT, XS, f8(144, 128), f32(2, 1)), SHAPE),
    (lambda: qg.gated_f8_backward(DH, GU, XT, None, WT, WTS), NULL),
    (lambda: qg.gated_f8_backward(DH, GU, XT, XS, WT, None), NULL),
    (lambda: qg.gated_f8_backward(DH, GU, None, None, None, None), NULL),
    (lambda: qg.gated_f8_backward(DH, GU, XT, XS, WT, WTS, act="tanh"), MODE),
    (lambda: qg.gated_f8_backward(DH, GU, XT, XS, WT, WTS, dx_dtype=torch.int8), DTYPE),
    (lambda: qg.gated_f8_backward(DH, GU, XT, XS, WT, WTS, dw_dtype=torch.float64), DTYPE),
])
def test_wrapper_refusals(call, status):
    with pytest.raises(qg.QGemmError) as e:
        call()
    assert e.value.status == status


@pytest.mark.parametrize("call", [
    lambda e: qg.quantize_f8(e(2 ** 32 + 1, 32, dtype=torch.float16)),
    lambda e: qg.quantize_f8(e(1, 2 ** 32 + 16, dtype=torch.float16), block=128),
    lambda e: qg.dequant_f8(e(1, 2 ** 31 + 16, dtype=torch.float8_e4m3fn), e(2 ** 24 + 1, 1, dtype=torch.float32)),
    lambda e: qg.gemm_f8_grouped(e(4, 128, dtype=torch.float8_e4m3fn), e(1, 4, dtype=torch.float32),
                                 e(65538, dtype=torch.int32), e(65537, 16, 128, dtype=torch.float8_e4m3fn),
                                 e(65537, 1, 1, dtype=torch.float32)),
])
def test_sizes_past_the_librarys(call):
    # sizes that a 32-bit integer would wrap (no memory behind them)
    with pytest.raises(qg.QGemmError) as e:
        call(lambda *shape, dtype: torch.empty(shape, dtype=dtype, device="meta"))
    assert e.value.status == UNSUP


# -- the reference forms ---------------------------------------------------------

def test_reference_codes_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(ref.decode(codes)))
    assert np.array_equal(np.nan_to_num(t), np.nan_to_num(ref.decode(codes)))
    v = torch.randn(4096, generator=torch.Generator().manual_seed(1)) * 100
    v = torch.cat([v.clamp(-448, 448), torch.arange(-448.0, 449.0) / 2, torch.arange(-64, 65) * 2.0 ** -11])
    assert np.array_equal(ref.encode(v.double().numpy()), v.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_reference_scales():
    top = [0.0, 448.0, 448.5, 1.75, 1.7500001, 1.0, 2.0 ** -140, 3.0e38, np.inf, np.nan]
    got = ref.scale_of(top)
    assert list(got[:8]) == [1.0, 1.0, 2.0, 2.0 ** -8, 2.0 ** -7, 2.0 ** -8, 2.0 ** -126, 2.0 ** 120]
    assert np.isnan(got[8:]).all()


def test_reference_transposed_blocks_agree():
    x = np.random.default_rng(0).standard_normal((200, 272))
    c, s = ref.quantize(x, 128)
    ct, st = ref.quantize(ref.pad16(x.T), 128)
    assert np.array_equal(ct[:, :200], c.T) and not ct[:, 200:].any() and np.array_equal(st, s.T)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_reference_slope_against_differences(act):
    g, h = np.linspace(-8, 8, 161), 1e-5
    d = (ref.gate(g + h, act)[0] - ref.gate(g - h, act)[0]) / (2 * h)
    # central differences: h^2 / 6 times a third derivative below 10, and 2^-53 * 8 / h of rounding
    assert np.abs(d - ref.gate(g, act)[1]).max() < 1e-9
