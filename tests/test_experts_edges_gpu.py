"""Expert-layer calls at the edges of their ranges, on the GPU."""
import pytest
import torch

import cute_layouts_mma_gb300 as tg

import _experts as X

pytestmark = pytest.mark.gpu


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda", 0)


def _done():
    torch.cuda.synchronize()
    assert tg.gemm_last_device_error() == tg.GEMM_OK


def _integer_codes(shape, g):
    return torch.randint(-4, 5, shape, generator=g).float().to(torch.float8_e4m3fn)


# ------------------------------------------------------------------ products

@pytest.mark.parametrize("M,N,K", [(200, 24, 128), (200, 264, 128), (1500, 520, 400), (2050, 4104, 128), (4100, 4104, 2064),
                                   (4100, 4120, 2064), (4100, 4128, 2064)])
@pytest.mark.parametrize("scales", ["tiles", "rows"])
def test_gemm_another_c_and_infinite_rows_at_a_column_remainder(M, N, K, scales):
    """Columns that end inside a warp's: the boxes past them write their staging buffer too,
    NaN where the row's scale is infinite (0 times it), while the last box in range leaves.
    Integer codes and power-of-two scales: a finite row is exact, and a row whose last
    block's scale is infinite is that block's sums' signs times infinity, NaN where one is 0."""
    dev = _dev()
    g = torch.Generator().manual_seed(M + N)
    kb = X.blocks(K)
    A, B = _integer_codes((M, K), g).to(dev), _integer_codes((N, K), g).to(dev)
    SFA = 2.0 ** torch.randint(-2, 3, (M, kb), generator=g).float()
    SFA[::3, -1] = float("inf")
    SFB = 2.0 ** torch.randint(-2, 3, (N if scales == "rows" else X.blocks(N), kb), generator=g).float()
    SFA, SFB = SFA.to(dev), SFB.to(dev)
    C = (torch.randn(M, N, generator=g) * 4).round().to(dev)
    want = C.double()
    for b in range(kb):
        part = A[:, b * 128:(b + 1) * 128].double() @ B[:, b * 128:(b + 1) * 128].double().t()
        want += part * SFA[:, b:b + 1].double() * X.spread(SFB[:, b:b + 1], N, 1).t()
    want = want.float()
    for _ in range(10):
        D = torch.full((M + 1, N), 12345.0, device=dev)
        tg.gemm_fp8_block(A, SFA, B, SFB, C, D[:M])
        _done()
        assert torch.equal(torch.isnan(D[:M]), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(D[:M], nan=0.0), torch.nan_to_num(want, nan=0.0))
        assert (D[M:] == 12345.0).all()
