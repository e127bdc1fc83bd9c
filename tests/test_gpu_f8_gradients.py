"""The F8 gated block's gradients against differences, by a bound that no gradient of
another size or sign meets, and its values where the sigmoid is tiny."""
import numpy as np
import pytest
import torch

import f8_ref as ref
import weight_only_quantized_w8a16_amd as qg

pytestmark = pytest.mark.gpu

BF, SF = torch.bfloat16, torch.float32
F8 = torch.float8_e4m3fn


def dev(a):
    a = torch.from_numpy(np.ascontiguousarray(a)).to("cuda")
    return a.float() if a.dtype == torch.float64 else a


def values(codes, scales, block=1):
    return ref.values(codes.view(torch.uint8).cpu().numpy(), scales.double().cpu().numpy(), block)


def cuts(a, b):
    """How far the products' sums may be off: seven cuts of 2^-13 of the largest of every eight products, and
    the fp32 sums (k additions of 2^-23 each, the scales' product and its application)."""
    k = a.shape[1]
    x, y = np.abs(a), np.abs(b)
    most = sum((x[:, None, g:g + 8] * y[None, :, g:g + 8]).max(-1) for g in range(0, k, 8))
    return 7 * 2.0 ** -13 * most + (k + 2) * 2.0 ** -23 * (x @ y.T)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_against_differences(act):
    """Every element of dX and dW against central differences of sum(dH * H) in 64 bits, as one vector."""
    rng = np.random.default_rng(11)
    m, inter, k = 24, 128, 144
    x, w = rng.standard_normal((m, k)), rng.standard_normal((2 * inter, k)) * 0.15
    q, s, xt, xts = qg.quantize_f8(dev(x), transposed=True)
    wq, ws, wt, wts = qg.quantize_f8(dev(w), block=128, transposed=True)
    xv, wv, xtv = values(q, s), values(wq, ws, 128), values(xt, xts)[:, :m].T
    dh = torch.from_numpy(rng.standard_normal((m, inter))).to(BF)
    _, gu = qg.gated_f8(q, s, wq, ws, act, BF, return_gu=True)
    dx, dw = qg.gated_f8_backward(dh.cuda(), gu, xt, xts, wt, wts, act, SF, SF)
    h = dh.double().numpy()

    def terms(a, b):
        """The sum's terms, one for each row and channel."""
        z = a @ b.T
        return h * ref.gate(z[:, :inter], act)[0] * z[:, inter:]

    # a column of X at a time in all rows, which share no term; of the gate's and of the up channels, likewise
    e = 1e-5
    want_x, want_w = np.empty_like(xv), np.empty_like(wv)
    for j in range(k):
        step = np.zeros_like(xv)
        step[:, j] = e
        want_x[:, j] = (terms(xv + step, wv) - terms(xv - step, wv)).sum(1) / (2 * e)
        for half in (slice(0, inter), slice(inter, 2 * inter)):
            step = np.zeros_like(wv)
            step[half, j] = e
            want_w[half, j] = (terms(xv, wv + step) - terms(xv, wv - step)).sum(0) / (2 * e)

    # D's error, element by element.  GU is off by the products' cuts and half a step of bf16 (2^-8):
    z = xv @ wv.T
    dz = cuts(xv, wv) + 2.0 ** -8 * (np.abs(z) + cuts(xv, wv))
    g, u, dg, du = z[:, :inter], z[:, inter:], dz[:, :inter], dz[:, inter:]
    value, slope = ref.gate(g, act)
    d = np.concatenate([h * u * slope, h * value], 1)
    # with |act''| <= 2 and |act'| <= 2 on the way
    moved = np.concatenate([np.abs(h) * (2 * dg * (np.abs(u) + du) + np.abs(slope) * du),
                            np.abs(h) * (np.abs(slope) * dg + dg ** 2)], 1)
    # then e4m3's half step: 2^-4 of the value, and 2^-10 of a scale that is below 2^-7 of the largest value
    size = np.abs(d) + moved
    off = moved + 2.0 ** -4 * size + 2.0 ** -17 * size.max()
    # ||E W|| <= ||E|| times W's largest singular value; dW multiplies by X^T's own codes, not X's
    norm, spectral = np.linalg.norm, lambda a: np.linalg.norm(a, 2)
    for got, want, bound in (
            (dx, want_x, norm(off) * spectral(wv) + norm(cuts(size, wv.T))),
            (dw, want_w, norm(off) * spectral(xtv) + norm(d.T @ (xtv - xv)) + norm(cuts(size.T, xtv.T)))):
        got = got.double().cpu().numpy()
        bound += 1e-6 * norm(want)      # the differences' own error: e^2 / 6 of third derivatives, 2^-53 / e
        assert bound < norm(want) / 2   # so zeros, a wrong sign or half of it would not do
        assert norm(got - want) <= bound


@pytest.mark.parametrize("act,low,high", [("silu", 80, 112), ("gelu", 5, 14)])
def test_gates_whose_sigmoid_is_tiny(act, low, high):
    """g = -s, u = s, down to sigmoids far below the smallest normal number, which may count as zeros."""
    inter, k, m = 128, 16, 257
    s = np.linspace(low, high, m).astype(np.float32)
    ca = ref.encode(np.ones((m, 1)) * np.eye(1, k))
    cb = ref.encode(np.concatenate([-np.ones((inter, 1)), np.ones((inter, 1))]) * np.eye(1, k))
    h = qg.gated_f8(dev(ca).view(F8), dev(s[None]), dev(cb).view(F8), torch.ones(2, 1, device="cuda"), act, SF)
    g = -s.astype(np.float64)
    y = g if act == "silu" else np.sqrt(8 / np.pi) * (g + 0.044715 * g ** 3)
    want = g / (1 + np.exp(-y)) * s
    # the sigmoid: 5 roundings of y, the exponential's argument's and 2 of its own, the reciprocal's, doubled,
    # or all of it below 2^-126; two products in fp32, whose subnormals have steps of 2^-149
    tol = (7 * np.abs(y) + 10) * 2.0 ** -23 * np.abs(want) + 2.0 ** -126 * np.abs(g * s) + 2.0 ** -148 * (1 + s)
    err = np.abs(h.double().cpu().numpy() - want[:, None])
    assert (err <= tol[:, None]).all(), (err / tol[:, None]).max()
