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


@pytest.mark.parametrize("scales", ["tiles", "rows"])
def test_gemm_of_nearly_two_to_the_31_columns(scales):
    """One row through the widest layer: narrow tiles, and (a scale per row of both) 128 x 128.
    Integer codes and power-of-two scales: sums of 16 products below 2^8 are exact in bf16."""
    dev = _dev()
    if torch.cuda.mem_get_info(dev)[0] < 80 << 30:
        pytest.skip("34 GB of weights")
    N, K, step = 2 ** 31 - 8, 16, 1 << 24
    g = torch.Generator(device=dev).manual_seed(5)
    code = torch.tensor([0x00, 0x38, 0x40, 0xB8, 0xC0], dtype=torch.uint8, device=dev)  # 0, 1, 2, -1, -2
    value = code.view(torch.float8_e4m3fn).float()
    pick = torch.randint(0, 5, (1, K), generator=g, device=dev)
    A, a = code[pick], value[pick]
    B = torch.empty(N, K, dtype=torch.uint8, device=dev)
    for lo in range(0, N, step):
        hi = min(N, lo + step)
        B[lo:hi] = code[torch.randint(0, 5, (hi - lo, K), generator=g, device=dev, dtype=torch.int32)]
    count = N if scales == "rows" else X.blocks(N)
    SFB = torch.empty(count, 1, device=dev)
    for lo in range(0, count, step):
        hi = min(count, lo + step)
        SFB[lo:hi, 0] = 2.0 ** (torch.arange(lo, hi, device=dev) % 5).float()
    SFA = torch.full((1, 1), 0.5, device=dev)
    D = torch.full((2, N), 77.0, dtype=torch.bfloat16, device=dev)
    tg.gemm_fp8_block(A, SFA, B, SFB, None, D[:1])
    _done()
    for lo in range(0, N, step):
        hi = min(N, lo + step)
        sums = (B[lo:hi].view(torch.float8_e4m3fn).float() * a).sum(dim=1)
        n = torch.arange(lo, hi, device=dev)
        want = 0.5 * sums * 2.0 ** ((n if scales == "rows" else n // 128) % 5).float()
        assert torch.equal(D[0, lo:hi].float(), want)
        assert (D[1, lo:hi] == 77.0).all()


@pytest.mark.parametrize("M,N,K", [(3, 136, 272), (100, 264, 4112), (300, 1032, 400), (2050, 2056, 1168), (4100, 4104, 1040)])
@pytest.mark.parametrize("scales", ["tiles", "rows"])
def test_gemm_in_place_keeps_subnormals(M, N, K, scales):
    """Sums, C and their totals below 2^-126, added in place (by the copy engine, where tiles
    leave in boxes) and to another C: exact either way, in units of 2^-149."""
    dev = _dev()
    g = torch.Generator().manual_seed(M + N)
    A, B = _integer_codes((M, K), g).to(dev), _integer_codes((N, K), g).to(dev)
    kb = X.blocks(K)
    SFA = torch.full((M, kb), 2.0 ** -70, device=dev)
    SFB = torch.full((N if scales == "rows" else X.blocks(N), kb), 2.0 ** -79, device=dev)
    C = (torch.randint(-2 ** 22, 2 ** 22, (M, N), generator=g).double() * 2.0 ** -149).float().to(dev)
    want = A.double() @ B.double().t() * 2.0 ** -149 + C.double()
    assert want.abs().max() < 2.0 ** -126 and (want != 0).any()
    D = torch.full_like(C, 9.0)
    tg.gemm_fp8_block(A, SFA, B, SFB, C, D)
    _done()
    assert torch.equal(D.double(), want)
    tg.gemm_fp8_block(A, SFA, B, SFB, C, C)
    _done()
    assert torch.equal(C.double(), want)


# ------------------------------------------------------------------ routing

@pytest.mark.parametrize("T", [3, 2600, 13000])
@pytest.mark.parametrize("E,groups", [(24, 1), (64, 1), (64, 4), (128, 1), (256, 8), (384, 1)])
@pytest.mark.parametrize("above", [30.0, 95.0, 120.0, 3e38])
def test_softmax_weights_of_experts_far_below_the_largest(T, E, groups, above):
    """A bias chooses among experts far below the row's largest logit: the renormalised weights
    are those of the chosen alone, and the gradient is theirs.  Bounds as for other routings:
    exponentials and sums of a few 2^-23 each, and one rounding of a difference below 8."""
    dev = _dev()
    g = torch.Generator().manual_seed(T + E)
    k, scale = 4, 2.5
    x = torch.rand(T, E, generator=g) * 8 - 4
    x[:, 5] = above
    bias = torch.zeros(E)
    bias[-6:] = 2.0 + torch.rand(6, generator=g)
    w = torch.empty(T, k, device=dev)
    ids = torch.empty(T, k, dtype=torch.int32, device=dev)
    tg.expert_route(x.to(dev), bias.to(dev), w, ids, tg.ROUTE_SOFTMAX, groups=groups, top_groups=max(1, groups // 2), group_best=1, scale=scale)
    dw = torch.randn(T, k, generator=g)
    dx = torch.empty(T, E, device=dev)
    tg.expert_route_grad(x.to(dev), ids, dw.to(dev), dx, tg.ROUTE_SOFTMAX, scale=scale)
    _done()
    ids = ids.cpu().long()
    assert torch.equal(ids, bias.sort(descending=True).indices[:k].expand(T, k))
    e = x.double().gather(1, ids).softmax(dim=1)
    want = scale * e
    assert ((w.cpu().double() - want).abs() <= want * (16 + E ** 0.5) * 2.0 ** -23).all()
    dot = (dw.double() * e).sum(dim=1, keepdim=True)
    grad = torch.zeros(T, E, dtype=torch.float64).scatter_(1, ids, want * (dw.double() - dot))
    lim = scale * dw.abs().amax(dim=1, keepdim=True).double() * (k + E ** 0.5 + 16) * 2.0 ** -23
    assert ((dx.cpu().double() - grad).abs() <= lim + grad.abs() * 2.0 ** -24).all()


def test_softmax_weights_of_masked_choices_stay_zero():
    """Chosen by the bias or for want of others, but masked: weight 0, beside ones that are not."""
    dev = _dev()
    x = torch.full((3, 16), -float("inf"))
    x[1, 2], x[1, 9] = -200.0, -201.0
    x[2, 4] = float("inf")
    bias = torch.zeros(16)
    bias[9] = 1.0
    w = torch.empty(3, 4, device=dev)
    ids = torch.empty(3, 4, dtype=torch.int32, device=dev)
    tg.expert_route(x.to(dev), bias.to(dev), w, ids, tg.ROUTE_SOFTMAX)
    _done()
    assert (w[0] == 0).all()
    assert ids[1, :2].tolist() == [9, 2] and (w[1, 2:] == 0).all()
    want = torch.tensor([-201.0, -200.0], dtype=torch.float64).softmax(dim=0)
    assert ((w[1, :2].cpu().double() - want).abs() <= 2.0 ** -19).all()
    assert ids[2, 0].item() == 4 and w[2].tolist() == [1.0, 0.0, 0.0, 0.0]


# ------------------------------------------------------------------ grouping

@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 400, 2 ** 31 - 513])
@pytest.mark.parametrize("dropped", [0, 1])
def test_group_of_nearly_two_to_the_31_pairs(n, dropped):
    """The largest pair counts: ids repeat in turn, so each place has a formula."""
    dev = _dev()
    if torch.cuda.mem_get_info(dev)[0] < 36 << 30:
        pytest.skip("26 GB of pairs")
    E = 3
    period = E + 2 * dropped  # -1 and E are no experts
    counts = [(n - (e + dropped) + period - 1) // period for e in range(E)]
    first = [sum(counts[:e]) for e in range(E + 1)]
    ids = torch.empty(n, 1, dtype=torch.int32, device=dev)
    step = 1 << 27
    for lo in range(0, n, step):
        hi = min(n, lo + step)
        ids[lo:hi, 0] = torch.arange(lo, hi, device=dev) % period - dropped
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    order, position = (torch.full((n,), 5, dtype=torch.int32, device=dev) for _ in range(2))
    tg.expert_group(ids, offsets, order, position)
    _done()
    assert offsets.tolist() == first
    start = torch.tensor(first[:E], device=dev)
    for lo in range(0, n, step):
        hi = min(n, lo + step)
        p = torch.arange(lo, hi, device=dev)
        e = p % period - dropped
        place = torch.where((e >= 0) & (e < E), start[e.clamp(0, E - 1)] + p // period, -1)
        assert torch.equal(position[lo:hi].long(), place)
        e = torch.bucketize(p, torch.tensor(first[1:], device=dev), right=True)  # of the place
        pair = torch.where(e < E, (p - start[e.clamp(max=E - 1)]) * period + e + dropped, -1)
        assert torch.equal(order[lo:hi].long(), pair)


# ------------------------------------------------------------------ quantisation

def _rows_formula(x):
    """Codes and scales of FP8_ROWS by the definition in fp32 (no NaN or infinity), on x's device."""
    b = torch.nn.functional.pad(x.float(), (0, -x.shape[1] % 128)).unflatten(1, (-1, 128))
    a = b.abs().amax(dim=2, keepdim=True).clamp_min(X.FLOOR)
    most = torch.full_like(a, 448.0)
    q = (b * (most / a)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.flatten(1)[:, :x.shape[1]], (a / most)[:, :, 0]


@pytest.mark.parametrize("dtype,K,index", [("bfloat16", 2 ** 31 - 144, None), ("bfloat16", 2 ** 31 - 2064, [0, -1]), ("float32", 2 ** 31 - 1040, [0, 0])])
def test_quantize_rows_of_nearly_two_to_the_31_elements(dtype, K, index):
    dev = _dev()
    if torch.cuda.mem_get_info(dev)[0] < 40 << 30:
        pytest.skip("rows of 2^31 elements")
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.empty(1, K, dtype=getattr(torch, dtype), device=dev)
    step = 1 << 27  # whole blocks
    for lo in range(0, K, step):
        x[:, lo:lo + step].normal_(generator=g)
    R = 1 if index is None else len(index)
    q = torch.full((R + 1, K), 99, dtype=torch.uint8, device=dev)
    sf = torch.full((R + 1, X.blocks(K)), -1.0, device=dev)
    tg.quantize_fp8(x, q[:R], sf[:R], index=None if index is None else torch.tensor(index, dtype=torch.int32, device=dev))
    _done()
    for lo in range(0, K, step):
        hi = min(K, lo + step)
        want_q, want_sf = _rows_formula(x[:, lo:hi])
        at = slice(lo // 128, X.blocks(hi))
        for r in range(R):
            none = index is not None and index[r] < 0
            assert torch.equal(sf[r, at], torch.full_like(want_sf[0], X.FLOOR) / torch.full_like(want_sf[0], 448.0) if none else want_sf[0])
            assert (q[r, lo:hi] == 0).all() if none else torch.equal(q[r, lo:hi], want_q[0])
        assert (q[R, lo:hi] == 99).all()
    assert (sf[R] == -1.0).all()
