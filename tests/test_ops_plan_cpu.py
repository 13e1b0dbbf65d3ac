"""The 8-bit product's plan on a host without a GPU (256 compute units)."""
import pytest

import fp32_gemm_f32_amd as g


@pytest.mark.parametrize("M,N,K", [(2 ** 31 - 5, 1, 1), (1, 2 ** 31 - 5, 1), (10 ** 9, 20, 3), (10 ** 9, 20, 17),
                                   (300_000_000, 64, 5), (17, 10 ** 9, 7), (40_000, 100_000, 50_001)])
def test_copies_stay_within_their_workspace(M, N, K):
    """Rows are copied to whole chunks of 16 bytes, however short they are: the limit of 4e9 bytes
    counts those."""
    d = g.gemm_i8_plan_describe(M, N, K, num_cus=256)
    k16 = (K + 15) // 16 * 16
    copies = sum(rows * k16 for rows, copied in zip((M, N), d["copies"]) if copied)
    assert copies <= 4e9
    assert d["splits"] > 1 or d["workspace_bytes"] == copies
