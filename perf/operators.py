"""Microscaled 4-bit (MX4) operators: what one pass computes, on which inputs.

An MX4 matrix holds 4-bit floats (sign, 2 exponent bits, 1 mantissa bit: the
magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6) in blocks of 32 along a row, each block
with one power-of-two scale 2^(s - 127), s an unsigned byte (255: NaN).

    quantise    s = max(floor(log2 of the block's largest magnitude) - 2 + 127, 0);
                codes = x / 2^(s - 127) rounded to the nearest magnitude, ties
                to the even code, beyond 6 to 6
    read back   value = code's value * 2^(s - 127)
    mx4a16      C = A . value(B)^T (+ bias), A in 16 bits
    mx4a4       C = value(quantise(A)) . value(B)^T (+ bias)
    grouped     rows offsets[e] .. offsets[e + 1] - 1 of A times expert e's
                weight: C[r] = A[r] . value(B[e])^T (+ bias[e])

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


# -- cases -------------------------------------------------------------------

def listed():
    return [
        # one decode step's activations of a 16-sequence batch, quantised and
        # read back: all latency
        dict(name="roundtrip-16x2048", op="roundtrip", rows=16, k=2048, dtype="bf16", tiled=True),
        # a whole up-projection weight, quantised at load and read back
        dict(name="roundtrip-13312x2048", op="roundtrip", rows=13312, k=2048, dtype="fp16",
             tiled=False),
        # one token through a square projection: the smallest product
        dict(name="a16-m1-n2048", op="a16", m=1, n=2048, k=2048, dtype="bf16", bias=False),
        # one token through the output head: the largest decode read
        dict(name="a16-m1-n131072", op="a16", m=1, n=131072, k=2048, dtype="bf16", bias=False),
        # an odd decode batch through a wide up-projection with bias
        dict(name="a16-m13-n18944", op="a16", m=13, n=18944, k=3584, dtype="fp16", bias=True),
        # a short prompt, or many sequences' tokens, through a square projection
        dict(name="a16-m100-n3584", op="a16", m=100, n=3584, k=3584, dtype="bf16", bias=True),
        # a long prompt through an up-projection
        dict(name="a16-m2048-n13312", op="a16", m=2048, n=13312, k=2048, dtype="bf16", bias=False),
        # a decode batch, activations quantised on the way in
        dict(name="a4-m8-n18944", op="a4", m=8, n=18944, k=3584, dtype="bf16", bias=False),
        # a ragged prompt through a down-projection (long sums, few outputs)
        dict(name="a4-m333-n3584", op="a4", m=333, n=3584, k=18944, dtype="bf16", bias=True),
        # the largest prompt through a wide up-projection
        dict(name="a4-m4096-n18944", op="a4", m=4096, n=18944, k=3584, dtype="fp16", bias=False),
        # 8 tokens' top-6 experts of 64: most experts see no row or one
        dict(name="grouped-48-e64", op="grouped", rows=48, experts=64, n=2816, k=2048,
             dtype="bf16", bias=False),
        # 2048 tokens' top-6 experts of 64
        dict(name="grouped-12288-e64", op="grouped", rows=12288, experts=64, n=2816, k=2048,
             dtype="bf16", bias=False),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def _multiple(rng, lo, hi, step):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, step * round(_log(rng, lo, hi) / step)))


def draw(rng):
    op = rng.choice(["roundtrip", "a16", "a16", "a4", "a4", "grouped"])
    dtype = rng.choice(["bf16", "fp16"])
    bias = rng.random() < 0.5
    while True:
        if op == "roundtrip":
            rows, tiled = round(_log(rng, 1, 16384)), rng.random() < 0.5
            k = _multiple(rng, 256, 8192, 128 if tiled else 32)
            if rows * k <= 13312 * 2048:
                return dict(op=op, rows=rows, k=k, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                            tiled=tiled)
        elif op == "a16":
            m, n = round(_log(rng, 1, 2048)), _multiple(rng, 512, 131072, 16)
            k = _multiple(rng, 512, 18944, 128)
            if n * k <= 131072 * 2048 and m * n * k <= 2048 * 13312 * 2048:
                return dict(op=op, m=m, n=n, k=k, dtype=dtype, bias=bias)
        elif op == "a4":
            m, n = round(_log(rng, 1, 4096)), _multiple(rng, 512, 32768, 16)
            k = _multiple(rng, 512, 18944, 128)
            if n * k <= 18944 * 3584 and m * n * k <= 4096 * 18944 * 3584:
                return dict(op=op, m=m, n=n, k=k, dtype=dtype, bias=bias)
        else:
            rows, experts = round(_log(rng, 1, 12288)), rng.randint(4, 96)
            n, k = _multiple(rng, 512, 4096, 16), _multiple(rng, 512, 4096, 128)
            if experts * n * k <= 64 * 2816 * 2048 and rows * n * k <= 12288 * 2816 * 2048:
                return dict(op=op, rows=rows, experts=experts, n=n, k=k, dtype=dtype, bias=bias)


# -- elementary forms ----------------------------------------------------------

def _quantise(x):
    """x [rows, k] -> (codes uint8 [rows, k] in 0..15, scale bytes uint8 [rows, k / 32])."""
    v = x.float().reshape(x.shape[0], -1, 32)
    field = (v.abs().amax(-1).view(torch.int32) >> 23) & 0xFF    # biased exponent
    s = (field - 2).clamp(min=0)
    inv = ((254 - s) << 23).view(torch.float32)                  # 2^(127 - s), exact
    a = (v.abs() * inv.unsqueeze(-1)).clamp(max=6.0)
    # steps of 0.5 up to 2, of 1 up to 4, of 2 up to 6; torch.round takes ties
    # to the even multiple, which is the even code
    small = torch.round(a * 2.0)
    mid = torch.round(a) + 2.0
    big = torch.round(a * 0.5) + 4.0
    mag = torch.where(a < 2.0, small, torch.where(a < 4.0, mid, big)).to(torch.uint8)
    sign = (v.view(torch.int32) < 0).to(torch.uint8) << 3
    return (mag | sign).reshape(x.shape), s.to(torch.uint8)


def _values(codes, s):
    """Codes [..., k] and scale bytes [..., k / 32] -> fp32 values."""
    c = codes.to(torch.int32)
    e, man = (c >> 1) & 3, (c & 1).float()
    mag = torch.where(e == 0, 0.5 * man, (1.0 + 0.5 * man) * (1 << e).float() * 0.5)
    val = torch.where((c & 8) != 0, -mag, mag)
    s = s.to(torch.int32)
    scale = (s << 23).view(torch.float32).masked_fill(s == 0, 2.0 ** -127)
    return (val.reshape(*codes.shape[:-1], -1, 32) * scale.unsqueeze(-1)).reshape(codes.shape)


def _unpack(packed):
    return torch.stack([packed & 15, packed >> 4], dim=-1).reshape(*packed.shape[:-1], -1)


def _pack(codes):
    c = codes.reshape(*codes.shape[:-1], -1, 2)
    return (c[..., 0] | (c[..., 1] << 4)).contiguous()


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
    """Packed codes and scale bytes of a normal weight with unequal channels."""
    w = torch.randn(n, k, generator=g, device=_DEV)
    w *= 0.02 * (0.5 + torch.rand(n, 1, generator=g, device=_DEV))
    codes, s = _quantise(w)
    return _pack(codes), s


def _expert_sizes(g, rows, experts):
    """Rows of each expert: drawn by unequal shares, some experts without any."""
    share = torch.randn(experts, generator=g, device=_DEV).exp()
    pick = torch.multinomial(share, rows, replacement=True, generator=g)
    return torch.bincount(pick, minlength=experts)


def prepare(case, seed):
    g = _gen(seed)
    dtype = _DT[case["dtype"]]
    st = dict(case=case)
    if case["op"] == "roundtrip":
        st["x"] = _activations(g, case["rows"], case["k"], dtype)
        return st
    n, k = case["n"], case["k"]
    experts = case.get("experts", 0)
    lead = (experts,) if experts else ()
    rows = case["rows"] if experts else case["m"]
    st["x"] = _activations(g, rows, k, dtype)
    packed, scales = _weights(g, n * max(experts, 1), k)
    st["bias"] = None
    if case["bias"]:
        st["bias"] = (0.02 * torch.randn(*lead, n, generator=g, device=_DEV)).to(dtype)
    if experts:
        sizes = _expert_sizes(g, rows, experts)
        st["sizes"] = sizes.tolist()
        st["offsets"] = torch.zeros(experts + 1, dtype=torch.int32, device=_DEV)
        st["offsets"][1:] = sizes.cumsum(0)
    if own:   # the weight in the order the products read it, laid out once
        import weight_only_quantized_w8a16_amd as qg
        w, s = qg.repack_mx4(packed, scales)   # experts are consecutive matrices
        st["w"], st["s"] = (w.reshape(experts, n, -1), s.reshape(experts, n // 16, -1, 64, 4)) \
            if experts else (w, s)
    else:
        st["w"], st["s"] = packed.reshape(*lead, n, -1), scales.reshape(*lead, n, -1)
    return st


# -- one pass --------------------------------------------------------------------

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import weight_only_quantized_w8a16_amd as qg
    case, x = st["case"], st["x"]
    if case["op"] == "roundtrip":
        codes, scales = qg.quantize_mx4(x, tiled=case["tiled"])
        return qg.dequant_mx4(codes, scales, x.dtype, tiled=case["tiled"], rows=x.shape[0])
    if case["op"] == "a16":
        return qg.gemm_mx4a16(x, st["w"], st["s"], st["bias"])
    if case["op"] == "a4":
        codes, scales = qg.quantize_mx4(x, tiled=True)
        return qg.gemm_mx4a4(codes, scales, st["w"], st["s"], m=x.shape[0], bias=st["bias"],
                             out_dtype=x.dtype)
    return qg.gemm_mx4a16_grouped(x, st["offsets"], st["w"], st["s"], st["bias"])


def _run_plain(st):
    case, x = st["case"], st["x"]
    if case["op"] == "roundtrip":
        return _values(*_quantise(x)).to(x.dtype)
    if case["op"] == "grouped":
        out = torch.empty(x.shape[0], case["n"], dtype=x.dtype, device=x.device)
        r0 = 0
        for e, size in enumerate(st["sizes"]):
            if size:
                w = _values(_unpack(st["w"][e]), st["s"][e])
                b = None if st["bias"] is None else st["bias"][e]
                out[r0:r0 + size] = _finish(x[r0:r0 + size].float() @ w.t(), b, x.dtype)
            r0 += size
        return out
    a = x.float() if case["op"] == "a16" else _values(*_quantise(x))
    w = _values(_unpack(st["w"]), st["s"])
    return _finish(a @ w.t(), st["bias"], x.dtype)


def work(case):
    size = _SIZE[case["dtype"]]
    if case["op"] == "roundtrip":
        elems = case["rows"] * case["k"]
        return {"bytes": elems * (2 * size + 0.5 + 1 / 32), "flops": 2 * elems}
    n, k = case["n"], case["k"]
    rows = case["rows"] if case["op"] == "grouped" else case["m"]
    weights = n * k
    if case["op"] == "grouped":   # experts that can have a row at all
        weights *= min(case["experts"], rows)
    return {"bytes": weights * (0.5 + 1 / 32) + rows * (k + n) * size, "flops": 2 * rows * n * k}


# -- 64-bit results from the definition --------------------------------------------

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _power64(e):
    """2^e as a 64-bit float, from its exponent field."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_roundtrip(x):
    """Nearest grid value of each element of its block, in 64 bits."""
    v = x.double().reshape(x.shape[0], -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    e = torch.frexp(top)[1] - 1 - 2                     # floor(log2) - 2
    e = torch.where(top == 0, torch.full_like(e, -127), e).clamp(min=-127)
    scale = _power64(e)
    a = v.abs() / scale
    best = torch.zeros_like(a)
    for i in range(1, 8):
        mid = (_GRID[i - 1] + _GRID[i]) / 2
        up = (a >= mid) if i % 2 == 0 else (a > mid)    # a tie goes to the even code
        best = torch.where(up, torch.full_like(a, _GRID[i]), best)
    return (torch.sign(v) * best * scale).reshape(x.shape)


def _exact_weight(packed, scales):
    table = torch.tensor(_GRID + tuple(-q for q in _GRID), dtype=torch.float64, device=packed.device)
    w = torch.empty(packed.shape[0], 2 * packed.shape[1], dtype=torch.float64, device=packed.device)
    w[:, 0::2] = table[(packed & 15).long()]
    w[:, 1::2] = table[(packed >> 4).long()]
    return w * _power64(scales.long() - 127).repeat_interleave(32, dim=1)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    x = st["x"]
    if case["op"] == "roundtrip":
        return _exact_roundtrip(x)
    a = _exact_roundtrip(x) if case["op"] == "a4" else x.double()
    if case["op"] != "grouped":
        c = a @ _exact_weight(st["w"], st["s"]).t()
        return c if st["bias"] is None else c + st["bias"].double()
    out = torch.empty(x.shape[0], case["n"], dtype=torch.float64, device=x.device)
    r0 = 0
    for e, size in enumerate(st["sizes"]):
        if size:
            out[r0:r0 + size] = a[r0:r0 + size] @ _exact_weight(st["w"][e], st["s"][e]).t()
            if st["bias"] is not None:
                out[r0:r0 + size] += st["bias"][e].double()
        r0 += size
    return out
