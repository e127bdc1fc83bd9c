"""F8 products on the paths that small problems do not take: every width of the
streaming kernel, and several tiles a workgroup by expert and gated."""
import numpy as np
import pytest
import torch

import f8_ref as ref
import weight_only_quantized_w8a16_amd as qg

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32
F8 = torch.float8_e4m3fn
TILES = ["T256", "T128", "T64"]


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


def exact_pair(rng, rows, k, block, lead=()):
    """(codes, scales, values in 64 bits) on the GPU: codes of -2 .. 2 and power-of-two scales, whose sums are
    exact in fp32."""
    g = torch.from_numpy(rng.integers(-2, 3, (*lead, rows, k)).astype(np.float32)).cuda()
    shape = (ref.blocks(k), rows) if block == 1 else (ref.blocks(rows), ref.blocks(k))
    s = torch.from_numpy(np.exp2(rng.integers(-1, 2, (*lead, *shape))).astype(np.float32)).cuda()
    wide = s.double()
    if block == 1:
        wide = wide.transpose(-1, -2)
    else:
        wide = wide.repeat_interleave(128, -2)[..., :rows, :]
    return g.to(F8), s, g.double() * wide.repeat_interleave(128, -1)[..., :k]


def same(got, want):
    assert got.shape == want.shape
    assert torch.equal(got.double(), want.to(got.dtype).double())


# -- the streaming kernel ------------------------------------------------------------

@pytest.mark.parametrize("rounds", [1, 2, 3, 4, 5, 6, 7, 8, 10, 12])
@pytest.mark.parametrize("m", [3, 19])
@pytest.mark.parametrize("dtype", [BF, SF])
def test_streamed_by_rounds(rounds, m, dtype):
    # the column tiles a workgroup go by the rounds of tiles over the CUs; one tile short of full rounds, so the
    # last workgroup's tiles are cut short
    qg.set_override(f8_tile="stream")
    rng = np.random.default_rng(rounds)
    slabs, k = (m + 15) // 16, 144
    tiles = cus() * rounds // slabs - 1
    assert -(-tiles * slabs // cus()) == rounds
    n = 16 * tiles
    (a, sa, av), (b, sb, bv) = exact_pair(rng, m, k, 1), exact_pair(rng, n, k, 128)
    bias = torch.from_numpy(rng.integers(-8, 9, n) / 4.0).to(HF).cuda()
    whole = torch.full((m + 1, n), 5.0, dtype=dtype, device="cuda")
    same(qg.gemm_f8(a, sa, b, sb, bias=bias, out=whole[:m]), av @ bv.t() + bias.double())
    assert (whole[m] == 5.0).all()


@pytest.mark.parametrize("n", [16, 144, 208, 272, 400, 1040, 1072])
@pytest.mark.parametrize("dtype", [BF, SF])
def test_streamed_by_expert(n, dtype):
    # 70 experts of no to 20 rows: one, two and four column tiles a workgroup
    qg.set_override(f8_tile="stream")
    rng = np.random.default_rng(n)
    sizes = [(7 * e) % 21 if e % 5 == 0 else e % 3 for e in range(70)]
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    rows, k = int(off[-1]), 272
    a, sa, av = exact_pair(rng, rows, k, 1)
    b, sb, bv = exact_pair(rng, n, k, 128, (70,))
    want = torch.cat([av[off[e]:off[e + 1]] @ bv[e].t() for e in range(70)])
    same(qg.gemm_f8_grouped(a, sa, torch.from_numpy(off).cuda(), b, sb, out_dtype=dtype), want)


def gate(g, act):
    y = g if act == "silu" else np.sqrt(8 / np.pi) * (g + 0.044715 * g ** 3)
    return g * torch.sigmoid(y), y


def check_gated(m, inter, k, act, dtype, seed):
    rng = np.random.default_rng(seed)
    (a, sa, av), (b, sb, bv) = exact_pair(rng, m, k, 1), exact_pair(rng, 2 * inter, k, 128)
    sb /= 8      # sums around 1 to 10
    gu = av @ (bv / 8).t()
    g, u = gu[:, :inter], gu[:, inter:]
    h, got = qg.gated_f8(a, sa, b, sb, act, dtype, return_gu=True)
    same(got, gu)
    assert torch.equal(qg.gated_f8(a, sa, b, sb, act, dtype), h)
    # act(g) = g s from exact sums: s = 1 / (1 + e^-y) with y's roundings (5 of 2^-24, times y), the
    # exponential's (its argument's again |y| 2^-24, 2 steps of its own) and the reciprocal's, doubled; the
    # products with g and u round once each, the result once to its type
    value, y = gate(g, act)
    want = value * u
    tol = (7 * y.abs() + 8) * 2.0 ** -23 * want.abs() + 2.0 ** -126 * (g * u).abs()
    tol += torch.finfo(dtype).eps / 2 * (want.abs() + tol) + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    err = (h.double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("m,groups", [(3, 1), (20, 2)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [BF, SF])
def test_streamed_gated_of_many_channels(m, groups, act, dtype):
    # more than four rounds of pairs of tiles: two pairs a workgroup
    qg.set_override(f8_tile="stream")
    inter = 128 * (4 * cus() // (8 * groups) + 1)
    assert inter // 16 * groups > 4 * cus()
    check_gated(m, inter, 272, act, dtype, m)


# -- several tiles a workgroup ---------------------------------------------------------

# rows, and the tile's: more tiles than workgroups (two a CU but for the largest)
MANY = [("T256", 2100, 256), ("T128", 1100, 128), ("T64", 600, 64)]


@pytest.mark.parametrize("k", [16, 272, 400])     # one step, an odd number, an even one
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [BF, SF])
@pytest.mark.parametrize("tile,m,rows", MANY)
def test_gated_of_many_tiles(tile, m, rows, act, dtype, k):
    qg.set_override(f8_tile=tile)
    inter, cols = (9216, 128) if tile == "T256" else (9216, 64)
    assert -(-m // rows) * (inter // cols) > 2 * cus()
    check_gated(m, inter, k, act, dtype, k)


@pytest.mark.parametrize("k", [16, 272, 400])
@pytest.mark.parametrize("dtype", [BF, SF])
@pytest.mark.parametrize("tile,m,rows", MANY)
def test_by_expert_of_many_tiles(tile, m, rows, dtype, k):
    # experts without rows, with one, with a whole tile and with several; n past the last whole tile; rows of no expert
    qg.set_override(f8_tile=tile)
    rng = np.random.default_rng(k)
    sizes = [0, m // 3 + 1, 0, 0, 1, rows, m // 5, 0, rows + 1, m // 4, 0]
    E, n = len(sizes), 9232
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32) + 3
    total = int(off[-1]) + 5
    cols, most = (256, 1) if tile == "T256" else (128, 2)      # workgroups a CU
    assert sum(-(-s // rows) for s in sizes) * -(-n // cols) > most * cus()
    a, sa, av = exact_pair(rng, total, k, 1)
    b, sb, bv = exact_pair(rng, n, k, 128, (E,))
    bias = torch.from_numpy(rng.integers(-8, 9, (E, n)) / 4.0).to(BF).cuda()
    want = torch.full((total, n), 77.0, dtype=torch.float64, device="cuda")
    for e in range(E):
        want[off[e]:off[e + 1]] = av[off[e]:off[e + 1]] @ bv[e].t() + bias[e].double()
    for _ in range(2):
        out = torch.full((total, n), 77.0, dtype=dtype, device="cuda")
        same(qg.gemm_f8_grouped(a, sa, torch.from_numpy(off).cuda(), b, sb, bias=bias, out=out), want)


@pytest.mark.parametrize("tile", TILES)
def test_by_expert_of_many_experts_and_tiles(tile):
    # a workgroup's tiles lie in several lots of 64 experts
    qg.set_override(f8_tile=tile)
    rng = np.random.default_rng(3)
    E, n, k = 300, 528, 144
    sizes = rng.integers(0, 4, E)
    sizes[[5, 150, 299]] = 70, 300, 129
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    a, sa, av = exact_pair(rng, int(off[-1]), k, 1)
    b, sb, bv = exact_pair(rng, n, k, 128, (E,))
    want = torch.cat([av[off[e]:off[e + 1]] @ bv[e].t() for e in range(E)])
    same(qg.gemm_f8_grouped(a, sa, torch.from_numpy(off).cuda(), b, sb, out_dtype=SF), want)


# -- the kernel taken ------------------------------------------------------------------

@pytest.mark.parametrize("m,n,k", [(1, 26624, 2048), (16, 37888, 3584), (16, 131072, 512)])
def test_one_slab_of_rows_is_streamed(m, n, k):
    """Up to 16 rows tiles of their own steps are slower: the bits are those of the streaming kernel, whose
    sums run in another order than a tile's."""
    g = torch.Generator(device="cuda").manual_seed(m)
    r = lambda *s: torch.rand(s, generator=g, device="cuda") + 0.5   # noqa: E731
    codes = lambda *s: (torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8) & 0xB7).view(F8)  # noqa: E731
    args = (codes(m, k), r(k // 128, m), codes(n, k), r(n // 128, k // 128))
    calls = (lambda: qg.gemm_f8(*args, out_dtype=SF), lambda: qg.gated_f8(*args, out_dtype=SF))
    got = [c() for c in calls]
    qg.set_override(f8_tile="stream")
    assert all(torch.equal(a, c()) for a, c in zip(got, calls))
    qg.set_override(f8_tile="T64")
    assert not any(torch.equal(a, c()) for a, c in zip(got, calls))
