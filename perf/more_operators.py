"""Block-scaled 8-bit float (F8) operators: what one pass computes, on which inputs.

An F8 matrix holds e4m3 codes (sign, 4 exponent bits, 3 mantissa bits, largest
448) and 32-bit scales, value = code's value * scale.  Activations have one
scale per row and 128 of k, kept as [ceil(k / 128), rows]; weights one per
128 x 128 block, [ceil(rows / 128), ceil(k / 128)].

    quantise    scale = the smallest power of two 2^e (e >= -126) with
                (largest magnitude of the block) / 2^e <= 448, 1 for a block of
                zeros; codes = x / 2^e rounded to the nearest e4m3, ties to the
                even code.  Transposed as well: the codes of x^T, its rows
                padded with zeros to a multiple of 16, its blocks those of x^T
    gemm        C = value(quantise(A)) . value(B)^T (+ bias)
    grouped     rows offsets[e] .. offsets[e + 1] - 1 of A with expert e's weight
    gated       with g = value(quantise(A)) . value(B_gate)^T and u that of
                B_up: H = act(g) * u, act(g) = g * sigmoid(y), y = g (silu) or
                2 sqrt(2 / pi) (g + 0.044715 g^3) (gelu); in training also
                GU = [g | u]
    backward    of gated, from dH and GU: dg = dH * u * act'(g), du = dH * act(g),
                D = [dg | du] quantised by rows for dX = value(D) . B and
                transposed for dB = value(D^T) . value(X^T)^T

``run`` makes one pass: with ``own`` set through the package's entry points,
else in elementary torch operations in 32 bits.  ``exact`` computes the same
results in 64 bits from the definition.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
_DEV = "cuda"
_F8 = torch.float8_e4m3fn
_GELU = 2.0 * math.sqrt(2.0 / math.pi)


# -- cases -------------------------------------------------------------------

def listed():
    return [
        # one decode step's activations of a 16-sequence batch, quantised and
        # read back: all latency
        dict(name="quant-16x2048", op="quant", rows=16, k=2048, dtype="bf16", block=1, both=False),
        # a training step's activations, by rows for the forward products and
        # transposed for the weight's gradient
        dict(name="quant-4096x3584-both", op="quant", rows=4096, k=3584, dtype="bf16", block=1,
             both=True),
        # one token through the output head: the largest decode read
        dict(name="gemm-m1-n131072", op="gemm", m=1, n=131072, k=2048, dtype="bf16", bias=False),
        # an odd decode batch through a wide projection with bias
        dict(name="gemm-m13-n18944", op="gemm", m=13, n=18944, k=3584, dtype="fp16", bias=True),
        # a ragged prompt through a down-projection (long sums, few outputs)
        dict(name="gemm-m333-n3584", op="gemm", m=333, n=3584, k=18944, dtype="bf16", bias=True),
        # the largest prompt through a wide projection
        dict(name="gemm-m4096-n18944", op="gemm", m=4096, n=18944, k=3584, dtype="bf16", bias=False),
        # 8 tokens' top-6 experts of 64: most experts see no row or one
        dict(name="grouped-48-e64", op="grouped", rows=48, experts=64, n=2816, k=2048, dtype="bf16",
             bias=False),
        # 2048 tokens' top-6 experts of 64
        dict(name="grouped-12288-e64", op="grouped", rows=12288, experts=64, n=2816, k=2048,
             dtype="bf16", bias=False),
        # one token through a gated block's two projections
        dict(name="gated-m1-i13312", op="gated", m=1, inter=13312, k=2048, dtype="bf16", act="silu",
             save=False),
        # a training step's tokens, the two projections kept for the backward pass
        dict(name="gated-m4096-i18944", op="gated", m=4096, inter=18944, k=3584, dtype="bf16",
             act="silu", save=True),
        # an odd, small batch of tokens back through an expert-sized gated block
        dict(name="backward-m100-i1408", op="backward", m=100, inter=1408, k=2048, dtype="fp16",
             act="gelu"),
        # a training step's tokens back through the widest gated block
        dict(name="backward-m4096-i18944", op="backward", m=4096, inter=18944, k=3584, dtype="bf16",
             act="silu"),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def _multiple(rng, lo, hi, step):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, step * round(_log(rng, lo, hi) / step)))


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "grouped", "gated", "backward"])
    dtype, bias, act = rng.choice(["bf16", "fp16"]), rng.random() < 0.5, rng.choice(["silu", "gelu"])
    while True:
        if op == "quant":
            rows, k = round(_log(rng, 1, 16384)), _multiple(rng, 256, 8192, 16)
            if rows * k <= 18944 * 3584:
                return dict(op=op, rows=rows, k=k, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                            block=rng.choice([1, 128]), both=rng.random() < 0.5)
        elif op == "gemm":
            m, n = round(_log(rng, 1, 4096)), _multiple(rng, 512, 131072, 16)
            k = _multiple(rng, 512, 18944, 16)
            if n * k <= 131072 * 2048 and m * n * k <= 4096 * 18944 * 3584:
                return dict(op=op, m=m, n=n, k=k, dtype=dtype, bias=bias)
        elif op == "grouped":
            rows, experts = round(_log(rng, 1, 12288)), rng.randint(4, 96)
            n, k = _multiple(rng, 512, 4096, 16), _multiple(rng, 512, 4096, 16)
            if experts * n * k <= 64 * 2816 * 2048 and rows * n * k <= 12288 * 2816 * 2048:
                return dict(op=op, rows=rows, experts=experts, n=n, k=k, dtype=dtype, bias=bias)
        else:
            m = round(_log(rng, 1 if op == "gated" else 16, 4096))
            inter, k = _multiple(rng, 256, 18944, 128), _multiple(rng, 512, 8192, 16)
            if inter * k <= 18944 * 3584 and m * inter * k <= 4096 * 18944 * 3584:
                case = dict(op=op, m=m, inter=inter, k=k, dtype=dtype, act=act)
                return dict(case, save=bias) if op == "gated" else case


# -- elementary forms ----------------------------------------------------------

def _blocks(x, rb, kb):
    """x [rows, k], zero-padded -> [rows / rb, rb, k / kb, kb]."""
    r, k = -(-x.shape[0] // rb) * rb, -(-x.shape[1] // kb) * kb
    if (r, k) != tuple(x.shape):
        x = torch.nn.functional.pad(x, (0, k - x.shape[1], 0, r - x.shape[0]))
    return x.reshape(r // rb, rb, k // kb, kb)


def _quantise(x, block):
    """x [rows, k] -> (codes e4m3 [rows, k], scales [rows / block, k / 128])."""
    v = _blocks(x.float(), block, 128)
    bits = v.abs().amax((1, 3)).contiguous().view(torch.int32)
    # amax = 1.f * 2^E: 448 = 1.75 * 2^8, so e = E - 8, one more above 1.75
    e = ((bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000)).clamp(min=-126)
    e = torch.where(bits == 0, torch.zeros_like(e), e)
    scale, inv = ((e + 127) << 23).view(torch.float32), ((127 - e) << 23).view(torch.float32)
    q = (v * inv[:, None, :, None]).to(_F8)
    q = q.view(torch.uint8).reshape(v.shape[0] * block, -1)[:x.shape[0], :x.shape[1]]
    return q.contiguous().view(_F8), scale


def _values(codes, scales, block):
    """Codes [rows, k] and scales [rows / block, k / 128] -> fp32 values."""
    rows, k = codes.shape
    s = scales.repeat_interleave(block, 0)[:rows] if block > 1 else scales
    return codes.float() * s.repeat_interleave(128, 1)[:, :k]


def _pad16(x):
    return torch.nn.functional.pad(x, (0, -x.shape[1] % 16))


def _act(g, kind):
    """act(g) and its derivative."""
    if kind == "silu":
        s, dy = torch.sigmoid(g), 1.0
    else:
        s, dy = torch.sigmoid(_GELU * (g + 0.044715 * g * g * g)), _GELU * (1.0 + 0.134145 * g * g)
    return g * s, s + g * s * (1.0 - s) * dy


def _finish(acc, bias, dtype):
    return (acc if bias is None else acc + bias.float()).to(dtype)


# -- inputs --------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    return g


def _activations(g, rows, k, dtype):
    """Rows of a normalised hidden state: unit normal, a few channels larger."""
    x = torch.randn(rows, k, generator=g, device=_DEV)
    loud = torch.rand(k, generator=g, device=_DEV) < 0.01
    return torch.where(loud, x * 8.0, x).to(dtype)


def _weights(g, n, k):
    """Codes and scales of a normal weight with unequal channels, the scales
    (largest magnitude) / 448 as checkpoints have them."""
    w = torch.randn(n, k, generator=g, device=_DEV)
    w *= 0.02 * (0.5 + torch.rand(n, 1, generator=g, device=_DEV))
    v = _blocks(w, 128, 128)
    scale = v.abs().amax((1, 3)) / 448.0
    q = (v / scale[:, None, :, None]).clamp(-448.0, 448.0).to(_F8).view(torch.uint8)
    return q.reshape(v.shape[0] * 128, -1)[:n, :k].contiguous().view(_F8), scale


def _transposed(codes):
    return codes.view(torch.uint8).t().contiguous().view(_F8)


def _expert_sizes(g, rows, experts):
    """Rows of each expert: drawn by unequal shares, some experts without any."""
    share = torch.randn(experts, generator=g, device=_DEV).exp()
    pick = torch.multinomial(share, rows, replacement=True, generator=g)
    return torch.bincount(pick, minlength=experts)


def prepare(case, seed):
    g = _gen(seed)
    op, dtype = case["op"], _DT[case["dtype"]]
    st = dict(case=case)
    if op == "quant":
        st["x"] = _activations(g, case["rows"], case["k"], dtype)
    elif op in ("gemm", "grouped"):
        n, k, experts = case["n"], case["k"], case.get("experts", 0)
        rows = case["rows"] if experts else case["m"]
        st["x"] = _activations(g, rows, k, dtype)
        if experts:
            pairs = [_weights(g, n, k) for _ in range(experts)]
            st["w"] = torch.stack([w.view(torch.uint8) for w, _ in pairs]).view(_F8)
            st["s"] = torch.stack([s for _, s in pairs])
            sizes = _expert_sizes(g, rows, experts)
            st["sizes"] = sizes.tolist()
            st["offsets"] = torch.zeros(experts + 1, dtype=torch.int32, device=_DEV)
            st["offsets"][1:] = sizes.cumsum(0)
        else:
            st["w"], st["s"] = _weights(g, n, k)
        st["bias"] = None
        if case["bias"]:
            lead = (experts,) if experts else ()
            st["bias"] = (0.02 * torch.randn(*lead, n, generator=g, device=_DEV)).to(dtype)
    else:
        m, inter, k = case["m"], case["inter"], case["k"]
        x = _activations(g, m, k, dtype)
        w, s = _weights(g, 2 * inter, k)
        if op == "gated":
            st["x"], st["w"], st["s"] = x, w, s
        else:
            st["dh"] = (0.1 * torch.randn(m, inter, generator=g, device=_DEV)).to(dtype)
            st["gu"] = torch.randn(m, 2 * inter, generator=g, device=_DEV).to(dtype)
            # what the forward pass leaves: x^T quantised, the weight transposed
            st["xt"], sxt = _quantise(_pad16(x.t()), 1)
            st["sxt"] = sxt.t().contiguous()
            st["wt"], st["swt"] = _transposed(w), s.t().contiguous()
    return st


# -- one pass --------------------------------------------------------------------

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import weight_only_quantized_w8a16_amd as qg
    case = st["case"]
    op = case["op"]
    if op == "quant":
        x, block = st["x"], case["block"]
        out = qg.quantize_f8(x, block=block, transposed=case["both"])
        return [qg.dequant_f8(out[i], out[i + 1], x.dtype, block=block)
                for i in range(0, len(out), 2)]
    if op == "backward":
        dtype = st["dh"].dtype
        dx, dw = qg.gated_f8_backward(st["dh"], st["gu"], st["xt"], st["sxt"], st["wt"], st["swt"],
                                      act=case["act"], dx_dtype=dtype, dw_dtype=dtype)
        return dict(dx=dx, dw=dw)
    x = st["x"]
    a, sa = qg.quantize_f8(x)
    if op == "gemm":
        return qg.gemm_f8(a, sa, st["w"], st["s"], bias=st["bias"], out_dtype=x.dtype)
    if op == "grouped":
        return qg.gemm_f8_grouped(a, sa, st["offsets"], st["w"], st["s"], bias=st["bias"],
                                  out_dtype=x.dtype)
    return qg.gated_f8(a, sa, st["w"], st["s"], act=case["act"], out_dtype=x.dtype,
                       return_gu=case["save"])


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "quant":
        x, block = st["x"], case["block"]
        q, s = _quantise(x, block)
        out = [_values(q, s, block).to(x.dtype)]
        if case["both"]:
            q, s = _quantise(_pad16(x.t()), block)
            out.append(_values(q, s, block).to(x.dtype))
        return out
    if op == "backward":
        dtype, inter = st["dh"].dtype, case["inter"]
        dh, g, u = st["dh"].float(), st["gu"][:, :inter].float(), st["gu"][:, inter:].float()
        h, slope = _act(g, case["act"])
        d = torch.cat([dh * u * slope, dh * h], 1)
        q, s = _quantise(d, 1)
        dx = _values(q, s, 1) @ _values(st["wt"], st["swt"], 128).t()
        q, s = _quantise(_pad16(d.t()), 1)
        dw = _values(q, s, 1) @ _values(st["xt"], st["sxt"].t(), 1).t()
        return dict(dx=dx.to(dtype), dw=dw.to(dtype))
    x = st["x"]
    a = _values(*_quantise(x, 1), 1)
    if op == "grouped":
        out = torch.empty(x.shape[0], case["n"], dtype=x.dtype, device=x.device)
        r0 = 0
        for e, size in enumerate(st["sizes"]):
            if size:
                b = None if st["bias"] is None else st["bias"][e]
                out[r0:r0 + size] = _finish(a[r0:r0 + size] @ _values(st["w"][e], st["s"][e], 128).t(),
                                            b, x.dtype)
            r0 += size
        return out
    c = a @ _values(st["w"], st["s"], 128).t()
    if op == "gemm":
        return _finish(c, st["bias"], x.dtype)
    inter = case["inter"]
    h = (_act(c[:, :inter], case["act"])[0] * c[:, inter:]).to(x.dtype)
    return (h, c.to(x.dtype)) if case["save"] else h


def work(case):
    op, size = case["op"], _SIZE[case["dtype"]]
    if op == "quant":
        elems, forms = case["rows"] * case["k"], 1 + case["both"]
        return {"bytes": elems * (size + forms * (2 + size)), "flops": 2 * forms * elems}
    if op in ("gated", "backward"):
        m, inter, k = case["m"], case["inter"], case["k"]
        flops = 2 * m * 2 * inter * k
        if op == "gated":
            saved = 2 * inter * case["save"]
            return {"bytes": 2 * inter * k + m * (k + inter + saved) * size, "flops": flops}
        # dH, GU, x^T, the weight -> dX, dB
        return {"bytes": m * 3 * inter * size + m * k + 2 * inter * k + (m + 2 * inter) * k * size,
                "flops": 2 * flops}
    n, k = case["n"], case["k"]
    rows = case["rows"] if op == "grouped" else case["m"]
    weights = n * k * (min(case["experts"], rows) if op == "grouped" else 1)
    return {"bytes": weights + rows * (k + n) * size, "flops": 2 * rows * n * k}


# -- 64-bit results from the definition --------------------------------------------

def _power64(e):
    """2^e as a 64-bit float, from its exponent field."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_quantised(x, block):
    """The values of x's nearest codes, in 64 bits."""
    v = _blocks(x.double(), block, 128)
    top = v.abs().amax((1, 3), keepdim=True)
    man, e = torch.frexp(top)                                # top = man * 2^e, man in [0.5, 1)
    e = torch.where(man > 448.0 / 512.0, e - 8, e - 9).clamp(min=-126)
    scale = _power64(torch.where(top == 0, torch.zeros_like(e), e))
    a = v / scale
    fine = (torch.frexp(a)[1] - 1).clamp(min=-6) - 3         # the exponent of a step of e4m3
    step = _power64(fine)
    out = torch.round(a / step) * step * scale
    return out.reshape(v.shape[0] * block, -1)[:x.shape[0], :x.shape[1]]


def _exact_values(codes, scales, block):
    """e4m3 from its fields, times its scale, in 64 bits."""
    c = codes.view(torch.uint8).long()
    e, man = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, man * 2.0 ** -9, (1.0 + man / 8.0) * _power64(e - 7))
    r, k = torch.arange(c.shape[0], device=c.device), torch.arange(c.shape[1], device=c.device)
    return torch.where(c >= 128, -mag, mag) * scales.double()[(r // block)[:, None], (k // 128)[None]]


def _exact_act(g, kind):
    y, dy = g, torch.ones_like(g)
    if kind == "gelu":
        c = math.sqrt(8.0 / math.pi)
        y, dy = c * (g + 0.044715 * g ** 3), c * (1.0 + 3 * 0.044715 * g ** 2)
    s = 1.0 / (1.0 + torch.exp(-y))
    return g * s, s * (1.0 + g * dy / (1.0 + torch.exp(y)))


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "quant":
        x = st["x"]
        out = [_exact_quantised(x, case["block"])]
        if case["both"]:
            out.append(_exact_quantised(_pad16(x.t()), case["block"]))
        return out
    if op == "backward":
        inter = case["inter"]
        dh, g, u = st["dh"].double(), st["gu"][:, :inter].double(), st["gu"][:, inter:].double()
        h, slope = _exact_act(g, case["act"])
        d = torch.cat([dh * u * slope, dh * h], 1)
        dx = _exact_quantised(d, 1) @ _exact_values(st["wt"], st["swt"], 128).t()
        dw = _exact_quantised(_pad16(d.t()), 1) @ _exact_values(st["xt"], st["sxt"].t(), 1).t()
        return dict(dx=dx, dw=dw)
    x = st["x"]
    a = _exact_quantised(x, 1)
    if op == "grouped":
        out = torch.empty(x.shape[0], case["n"], dtype=torch.float64, device=x.device)
        r0 = 0
        for e, size in enumerate(st["sizes"]):
            if size:
                out[r0:r0 + size] = a[r0:r0 + size] @ _exact_values(st["w"][e], st["s"][e], 128).t()
                if st["bias"] is not None:
                    out[r0:r0 + size] += st["bias"][e].double()
            r0 += size
        return out
    c = a @ _exact_values(st["w"], st["s"], 128).t()
    if op == "gemm":
        return c if st["bias"] is None else c + st["bias"].double()
    inter = case["inter"]
    h = _exact_act(c[:, :inter], case["act"])[0] * c[:, inter:]
    return (h, c) if case["save"] else h
