"""Refusals of the expert-layer calls at the ends of their ranges (CPU only)."""
import pytest

import cute_layouts_mma_gb300 as tg
from cute_layouts_mma_gb300 import build


def test_grouped_refuses_rows_that_its_tiles_cannot_count():
    far = [i << 40 for i in range(1, 7)]  # apart by more than any operand
    f = lambda R, N, E: tg.lib().gemm_fp8_block_grouped(R, N, 16, E, *far[:5], far[5], None)
    assert f(2 ** 31 - 511, 8, 1) == tg.GEMM_ERR_INVALID_ARG
    assert f(2 ** 31 - 1, 8, 4) == tg.GEMM_ERR_INVALID_ARG
    assert f(8, 2 ** 31 - 504, 1) == tg.GEMM_ERR_INVALID_ARG
    assert f(8, 2 ** 28 - 56, 8) == tg.GEMM_ERR_INVALID_ARG


LOG = """ptxas info    : Compiling entry function '_ZN2tn21gemm_fp8_block_kernelINS_9Fp8ConfigILi0ELi2ELi256ELi4ELi1ELi2ELi8ELb1EEEEEv' for 'sm_103a'
ptxas info    : Function properties for _ZN2tn21gemm_fp8_block_kernelINS_9Fp8ConfigILi0ELi2ELi256ELi4ELi1ELi2ELi8ELb1EEEEEv
    8 bytes stack frame, 20 bytes spill stores, 48 bytes spill loads
ptxas info    : Used {pair} registers, used 1 barriers, 8 bytes cumulative stack size
ptxas info    : Compiling entry function '_ZN2tn21gemm_fp8_block_kernelINS_9Fp8ConfigILi0ELi1ELi128ELi5ELi1ELi4ELi8ELb1EEEEEv' for 'sm_103a'
ptxas info    : Used 149 registers, used 1 barriers
ptxas info    : Compiling entry function '_ZN2tn21gemm_fp8_block_kernelINS_9Fp8ConfigILi0ELi1ELi256ELi3ELi1ELi2ELi8ELb1EEEEEv' for 'sm_103a'
ptxas info    : Used {single} registers, used 1 barriers
"""


def test_register_split_is_checked_by_the_build():
    """Only the instances that share out their registers need their count, whatever others have."""
    assert build.check_register_split(LOG.format(pair=168, single=168)) == 2
    for counts in ({"pair": 160, "single": 168}, {"pair": 168, "single": 255}):
        with pytest.raises(RuntimeError, match="registers"):
            build.check_register_split(LOG.format(**counts))
    assert build.check_register_split("") == 0
