"""MX4 operators at the ends of their sizes: refused on the host, before a
launch (no GPU; the addresses are stand-ins)."""
import pytest

import weight_only_quantized_w8a16_amd as qg

UNSUP = 7
FAKE = 0x100000          # 16-byte-aligned stand-in address; never dereferenced
BF16, TILED = 1, 1


def conversions(rows, k):
    L = qg.lib()
    return {"quantize": L.qquantize_mx4(FAKE, FAKE, FAKE, rows, k, TILED, BF16, None),
            "dequant": L.qdequant_mx4(FAKE, FAKE, FAKE, rows, k, TILED, BF16, None),
            "repack": L.qrepack_mx4(FAKE, FAKE, FAKE, FAKE, rows, k, None),
            "unrepack": L.qunrepack_mx4(FAKE, FAKE, FAKE, FAKE, rows, k, None)}


@pytest.mark.parametrize("k", [2 ** 31 - 128, 2 ** 31 - 256, 2 ** 31 - 384])
def test_tiled_conversions_refuse_k_whose_windows_pass_32_bits(k):
    # k + 511, of which the 512-k windows are counted, is past 2^31 - 1
    assert set(conversions(1, k).values()) == {UNSUP}


@pytest.mark.parametrize("rows,k", [(2 ** 28, 128), (2 ** 28 + 1, 512), (2 ** 24, 16 * 512)])
def test_tiled_conversions_of_more_pieces_than_a_launch_has(rows, k):
    assert (rows + 15) // 16 * ((k + 511) // 512) >= 2 ** 24
    assert set(conversions(rows, k).values()) == {UNSUP}


@pytest.mark.parametrize("k", [1024, 8192])
def test_products_wider_than_a_launch(k):
    n = 2 ** 30
    L = qg.lib()
    assert L.qgemm_mx4a16(FAKE, FAKE, FAKE, None, FAKE, 4, n, k, BF16, 0, None, 0, None) == UNSUP
    assert L.qgemm_mx4a4(FAKE, FAKE, FAKE, FAKE, None, FAKE, 4, n, k, BF16, 0, None, 0, None) == UNSUP
    assert L.qgemm_mx4a16_grouped(FAKE, FAKE, FAKE, FAKE, None, FAKE, 4, n, k, 2, BF16, 0, None) == UNSUP


@pytest.mark.parametrize("m,n,k", [(2 ** 32 + 64, 256, 4096), (64, 2 ** 32 + 256, 4096), (64, 256, 2 ** 32 + 4096),
                                   (-2 ** 32 + 64, 256, 4096)])
def test_workspace_size_of_sizes_past_32_bits(m, n, k):
    # no problem the library takes; as 32-bit integers they would wrap into one
    qg.set_override(mx4_tile="T64", mx4_split=4)
    assert qg.mx4_workspace_size(64, 256, 4096, 16) > 0
    assert qg.mx4_workspace_size(m, n, k, 16) == 0
