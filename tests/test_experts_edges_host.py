"""Refusals of the expert-layer calls at the ends of their ranges (CPU only)."""
import cute_layouts_mma_gb300 as tg


def test_grouped_refuses_rows_that_its_tiles_cannot_count():
    far = [i << 40 for i in range(1, 7)]  # apart by more than any operand
    f = lambda R, N, E: tg.lib().gemm_fp8_block_grouped(R, N, 16, E, *far[:5], far[5], None)
    assert f(2 ** 31 - 511, 8, 1) == tg.GEMM_ERR_INVALID_ARG
    assert f(2 ** 31 - 1, 8, 4) == tg.GEMM_ERR_INVALID_ARG
    assert f(8, 2 ** 31 - 504, 1) == tg.GEMM_ERR_INVALID_ARG
    assert f(8, 2 ** 28 - 56, 8) == tg.GEMM_ERR_INVALID_ARG
