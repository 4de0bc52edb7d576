"""Grouped products over ragged segments and their gradients against 64-bit
products: segment lengths around the tile and stage sizes, odd widths and
strides, neighbours that hold Inf or NaN, 8-bit operands named by a row index.
Bounds: ops_util (f32 sums of exact products, then half a step of the output
type)."""
import pytest
import torch

from ops_util import BF16, F32, I32, check, kept_values, offsets_of, rounding, sum_bound
from quantization_nvfp4_quantize_b200 import api

pytestmark = pytest.mark.gpu


def rnd(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF16)


def ref_rows(a, w, off, transpose, fill):
    """(result, sum of |products|) with rows outside the segments at `fill`."""
    y = fill.double().clone()
    s = torch.zeros_like(y)
    for e in range(w.shape[0]):
        lo, hi = int(off[e]), int(off[e + 1])
        m = w[e].double() if transpose else w[e].double().t()
        y[lo:hi] = a[lo:hi].double() @ m
        s[lo:hi] = a[lo:hi].double().abs() @ m.abs()
    return y, s


COUNTS = [
    [1],
    [0, 5, 0],
    [64, 63, 65, 1],
    [255, 0, 256, 257, 3],
    [1] * 17,
    [700, 2, 0, 130],
]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("N,K", [(8, 8), (264, 72), (520, 328), (128, 64)])
def test_products(cuda, counts, N, K, transpose):
    E, M = len(counts), sum(counts) + 9
    off = offsets_of(counts, cuda, start=2)                       # rows before and behind the segments
    w = rnd(1, E, N, K, scale=0.1)
    a = rnd(2, M, N if transpose else K)
    for dtype in (BF16, F32):
        out = torch.full((M, K if transpose else N), 7.0, dtype=dtype, device=cuda)
        got = api.ragged_gemm(a, w, off, transpose=transpose, out=out)
        assert got.data_ptr() == out.data_ptr()
        y, s = ref_rows(a, w, off, transpose, torch.full_like(out, 7.0))
        check(got, y, sum_bound(a.shape[1], s) + rounding(dtype, y), f"{dtype}")


@pytest.mark.parametrize("N", [1, 3, 33, 255, 257])
def test_odd_output_width(cuda, N):
    counts = [70, 0, 200]
    off = offsets_of(counts, cuda)
    w, a = rnd(3, 3, N, 80, scale=0.1), rnd(4, 270, 80)
    for dtype in (BF16, F32):
        got = api.ragged_gemm(a, w, off, out_dtype=dtype)
        y, s = ref_rows(a, w, off, False, torch.zeros(270, N, device=cuda))
        check(got, y, sum_bound(80, s) + rounding(dtype, y))


@pytest.mark.parametrize("transpose", [False, True])
def test_strided_operands(cuda, transpose):
    """Rows on a longer stride; an output whose base and rows are aligned to
    its elements only, inside a buffer that must stay as it is."""
    counts = [100, 33, 300]
    off = offsets_of(counts, cuda)
    N, K = 136, 200
    w = rnd(5, 3, N, K, scale=0.1)
    a = rnd(6, 433, 264)[:, 8:8 + (N if transpose else K)]
    width = K if transpose else N
    for dtype in (BF16, F32):
        buf = torch.full((433, width + 7), 5.0, dtype=dtype, device=cuda)
        out = buf[:, 3:3 + width]
        api.ragged_gemm(a, w, off, transpose=transpose, out=out)
        y, s = ref_rows(a, w, off, transpose, torch.zeros(433, width, device=cuda))
        check(out, y, sum_bound(a.shape[1], s) + rounding(dtype, y))
        assert bool((buf[:, :3] == 5).all()) and bool((buf[:, 3 + width:] == 5).all())


@pytest.mark.parametrize("transpose", [False, True])
def test_products_keep_bad_values_apart(cuda, transpose):
    """Inf and NaN in another expert's rows or weights, or outside the
    segments, reach no result."""
    counts = [70, 60, 90]
    off = offsets_of(counts, cuda, start=5)
    N, K = 200, 104                                                # neither a multiple of the 64-deep stage
    w = rnd(7, 3, N, K, scale=0.1)
    a = rnd(8, 240, N if transpose else K)
    w[1] = float("nan")
    a[75:135] = float("inf")
    a[:5] = float("nan")
    a[225:] = float("nan")
    got = api.ragged_gemm(a, w, off, transpose=transpose, out_dtype=F32)
    ok = torch.cat([torch.arange(5, 75), torch.arange(135, 225)]).to(cuda)
    y, s = ref_rows(a, w, off, transpose, torch.zeros_like(got))
    check(got[ok], y[ok], sum_bound(a.shape[1], s[ok]) + rounding(F32, y[ok]))
    # one bad row spoils itself only
    a2, w2 = rnd(8, 240, a.shape[1]), rnd(7, 3, N, K, scale=0.1)
    a2[100, 3] = float("nan")
    got = api.ragged_gemm(a2, w2, off, transpose=transpose, out_dtype=F32)
    assert bool(torch.isnan(got[100]).all())
    keep = torch.ones(240, dtype=torch.bool, device=cuda)
    keep[100], keep[:5], keep[225:] = False, False, False
    assert bool(torch.isfinite(got[keep]).all())


def ref_wgrad(g, a, off):
    E = off.numel() - 1
    y = torch.zeros(E, g.shape[1], a.shape[1], dtype=torch.float64, device=g.device)
    s = torch.zeros_like(y)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        y[e] = g[lo:hi].double().t() @ a[lo:hi].double()
        s[e] = g[lo:hi].double().abs().t() @ a[lo:hi].double().abs()
    return y, s


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("N,K", [(8, 8), (264, 72), (520, 328), (128, 257)])
def test_weight_gradient(cuda, counts, N, K):
    E, M = len(counts), sum(counts) + 9
    off = offsets_of(counts, cuda, start=2)
    g = rnd(11, M, N, scale=0.1)
    a = rnd(12, M, -(-K // 8) * 8)[:, :K]
    g[:2], a[:2] = float("nan"), float("inf")                      # rows of no segment
    g[-7:], a[-7:] = float("nan"), float("inf")
    y, s = ref_wgrad(g, a, off)
    n = max(counts) + 1
    for dtype in (F32, BF16):
        got = api.ragged_wgrad(g, a, off, out_dtype=dtype)
        check(got, y, sum_bound(n, s) + rounding(dtype, y), f"{dtype}")
        old = rnd(13, E, N, K).to(dtype)
        acc = old.clone()
        api.ragged_wgrad(g, a, off, out=acc, accumulate=True)
        z = y + old.double()
        check(acc, z, sum_bound(n, s) + ULP_ADD * (y.abs() + old.double().abs()) + rounding(dtype, z), f"accumulate {dtype}")


ULP_ADD = 2.0 ** -23                                               # the f32 addition of the old value


def test_weight_gradient_keeps_bad_values_apart(cuda):
    counts = [70, 60, 90, 0, 64]
    off = offsets_of(counts, cuda)
    g, a = rnd(14, 284, 264, scale=0.1), rnd(15, 284, 200)
    g[70:130] = float("nan")
    a[70:130] = float("inf")
    got = api.ragged_wgrad(g, a, off)
    y, s = ref_wgrad(g, a, off)
    for e in (0, 2, 3, 4):
        check(got[e], y[e], sum_bound(100, s[e]) + rounding(F32, y[e]), f"expert {e}")
    assert bool(torch.isnan(got[1]).all())


@pytest.mark.parametrize("E,M,N,K", [(1, 20000, 64, 96), (3, 9001, 256, 264), (2, 5000, 300, 40), (1, 600, 8, 8)])
def test_weight_gradient_split_rows(cuda, E, M, N, K):
    """Few output tiles: rows split over the SMs, partial sums through the
    workspace; the same bits from run to run."""
    assert api._lib.load().moe_ragged_wgrad_workspace_size(M, N, K, E, 0) > 0
    cut = sorted([0] + [int(M * f) for f in (0.13, 0.52)][: E - 1] + [M - 3])
    off = torch.tensor(cut, dtype=I32, device=cuda)
    g, a = rnd(16, M, -(-N // 8) * 8, scale=0.1)[:, :N], rnd(17, M, K)
    y, s = ref_wgrad(g, a, off)
    old = rnd(18, E, N, K).float()
    for dtype in (F32, BF16):
        got = api.ragged_wgrad(g, a, off, out_dtype=dtype)
        check(got, y, sum_bound(M, s) + rounding(dtype, y))
        assert torch.equal(got, api.ragged_wgrad(g, a, off, out_dtype=dtype))
        acc = old.to(dtype)
        z = y + acc.double()
        bound = sum_bound(M, s) + ULP_ADD * (y.abs() + acc.double().abs()) + rounding(dtype, z)
        api.ragged_wgrad(g, a, off, out=acc, accumulate=True)
        check(acc, z, bound)


@pytest.mark.parametrize("counts", COUNTS[1:], ids=str)
@pytest.mark.parametrize("N,K", [(8, 8), (264, 72), (136, 333), (520, 528)])
def test_weight_gradient_from_kept_rows(cuda, counts, N, K):
    """8-bit activations named by a row index: repeated rows, indices outside
    the kept tensor, scales from the smallest to large powers."""
    E, M, T = len(counts), sum(counts) + 4, 50
    off = offsets_of(counts, cuda, start=1)
    x = rnd(21, T, -(-K // 8) * 8)[:, :K].float()
    x = (x * torch.exp2(torch.arange(T, device=cuda).float()[:, None] * 2 - 60)).to(BF16)
    x[3] = 0
    xk = torch.zeros(T, -(-K // 8) * 8, dtype=BF16, device=cuda)[:, :K]
    xk.copy_(x)
    a8 = api.act8_quantize(xk)
    gen = torch.Generator().manual_seed(5)
    rows = torch.randint(0, T, (M,), generator=gen).to(I32).to(cuda)
    rows[2], rows[4] = -1, T
    g = rnd(22, M, N, scale=0.1)
    g[:1], g[-3:] = float("nan"), float("nan")
    full = torch.zeros(M, K, dtype=torch.float64, device=cuda)
    ok = (rows >= 0) & (rows < T)
    full[ok] = kept_values(a8)[rows[ok].long()]
    y, s = ref_wgrad(g, full, off)
    got = api.ragged_wgrad(g, a8, off, a_rows=rows)
    check(got, y, sum_bound(max(counts) + 1, s) + rounding(F32, y))


@pytest.mark.parametrize("kept", [False, True])
def test_weight_gradient_many_stages_and_tiles(cuda, kept):
    """Several tiles per SM pair, each many turns of the stage ring."""
    counts = [4001, 0, 700, 2500, 64, 1]
    off = offsets_of(counts, cuda)
    M, N, K = sum(counts), 1288, 1032
    g, x = rnd(27, M, N, scale=0.1), rnd(28, M, K)
    a = api.act8_quantize(x) if kept else x
    y, s = ref_wgrad(g, kept_values(a) if kept else x, off)
    for _ in range(3):
        check(api.ragged_wgrad(g, a, off), y, sum_bound(4001, s) + rounding(F32, y))


def test_weight_gradient_from_kept_rows_in_order(cuda):
    off = offsets_of([130, 3, 200], cuda)
    a8 = api.act8_quantize(rnd(23, 333, 256))
    g = rnd(24, 333, 264)
    y, s = ref_wgrad(g, kept_values(a8), off)
    check(api.ragged_wgrad(g, a8, off), y, sum_bound(200, s) + rounding(F32, y))


def test_every_kept_code_reads_exactly(cuda):
    """All E4M3 codes times scales from the smallest up, through the weight
    gradient of one row with g = 1."""
    codes = torch.arange(256, dtype=torch.uint8, device=cuda).repeat(4, 1)
    codes[(codes & 0x7F) == 0x7F] = 0
    scales = torch.tensor([[7] * 8, [100] * 8, [127] * 8, [240] * 8], dtype=torch.uint8, device=cuda)
    a8 = api.Act8(codes.contiguous(), scales.contiguous())
    off = torch.tensor([0, 1, 2, 3, 4], dtype=I32, device=cuda)
    g = torch.ones(4, 8, dtype=BF16, device=cuda)
    got = api.ragged_wgrad(g, a8, off)
    want = kept_values(a8)[:, None, :].expand(4, 8, 256)
    # products with 1 are exact in f32 down to its smallest normal
    tiny = torch.finfo(F32).smallest_normal
    assert bool((((got.double() - want).abs()) <= tiny * (want.abs() < tiny)).all())


def test_kept_nan_group_reaches_the_gradient(cuda):
    x = rnd(25, 64, 128)
    x[10, 40] = float("inf")
    got = api.ragged_wgrad(rnd(26, 64, 16), api.act8_quantize(x), offsets_of([64], cuda))
    assert bool(torch.isnan(got[0, :, 32:64]).all())
    assert bool(torch.isfinite(got[0, :, :32]).all()) and bool(torch.isfinite(got[0, :, 64:]).all())


def test_bad_offsets_stay_inside(cuda):
    """Descending or out-of-range bounds read as their running maximum inside
    [0, M]."""
    a, w, g = rnd(31, 100, 64), rnd(32, 4, 64, 64), rnd(33, 100, 64)
    off = torch.tensor([-5, 40, 20, 500, 60], dtype=I32, device=cuda)
    eff = torch.tensor([0, 40, 40, 100, 100], dtype=I32, device=cuda)
    fill = torch.zeros(100, 64, dtype=F32, device=cuda)
    assert torch.equal(api.ragged_gemm(a, w, off, out=fill.clone()), api.ragged_gemm(a, w, eff, out=fill.clone()))
    assert torch.equal(api.ragged_wgrad(g, a, off), api.ragged_wgrad(g, a, eff))


def test_most_experts_and_wide_tables(cuda):
    counts = [(7 * e) % 5 for e in range(256)]
    off = offsets_of(counts, cuda)
    M = sum(counts)
    a, w = rnd(34, M, 64), rnd(35, 256, 72, 64, scale=0.1)
    got = api.ragged_gemm(a, w, off, out_dtype=F32)
    y, s = ref_rows(a, w, off, False, torch.zeros(M, 72, device=cuda))
    check(got, y, sum_bound(64, s) + rounding(F32, y))
    g = rnd(36, M, 72)
    y, s = ref_wgrad(g, a, off)
    check(api.ragged_wgrad(g, a, off), y, sum_bound(8, s) + rounding(F32, y))


def test_long_offsets(cuda):
    """A row buffer whose elements pass 2^31: the last rows' products."""
    M, K = 1_100_000, 2048
    a = torch.empty(M, K, dtype=BF16, device=cuda)
    tail = rnd(37, 300, K)
    a[-300:] = tail
    w = rnd(38, 2, 64, K, scale=0.05)
    off = torch.tensor([M - 300, M - 100, M], dtype=I32, device=cuda)
    out = api.ragged_gemm(a, w, off, out=torch.zeros(M, 64, dtype=F32, device=cuda))
    small = offsets_of([200, 100], cuda)
    y, s = ref_rows(tail, w, small, False, torch.zeros(300, 64, device=cuda))
    check(out[-300:], y, sum_bound(K, s) + rounding(F32, y))
    assert not bool(out[:-300].any())
    g = torch.empty(M, 64, dtype=BF16, device=cuda)
    g[-300:] = rnd(39, 300, 64)
    y, s = ref_wgrad(g[-300:], tail, small)
    check(api.ragged_wgrad(g, a, off), y, sum_bound(M, s) + rounding(F32, y))


def test_captured_and_on_another_stream(cuda):
    off = offsets_of([130, 70], cuda)
    a, w, g = rnd(41, 200, 128), rnd(42, 2, 96, 128), rnd(43, 200, 96)
    y0 = api.ragged_gemm(a, w, off)
    d0 = api.ragged_wgrad(g, a, off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1 = api.ragged_gemm(a, w, off)
        graph = torch.cuda.CUDAGraph()
    side.synchronize()
    with torch.cuda.graph(graph):
        y2 = api.ragged_gemm(a, w, off)
        d2 = api.ragged_wgrad(g, a, off)
    y2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(y0, y2) and torch.equal(d0, d2)
    a.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, api.ragged_gemm(a, w, off)) and torch.equal(d2, api.ragged_wgrad(g, a, off))


def test_gradients_match_differences(cuda):
    """d sum(out * c) along random directions, against the gradients, by
    central differences of the 64-bit product (linear in each factor, so the
    difference is exact but for its own rounding)."""
    counts = [40, 0, 25]
    off = offsets_of(counts, cuda)
    a, w, c = rnd(44, 65, 48), rnd(45, 3, 56, 48), rnd(46, 65, 56)

    def loss(av, wv):
        y = torch.zeros(65, 56, dtype=torch.float64, device=cuda)
        for e in range(3):
            lo, hi = int(off[e]), int(off[e + 1])
            y[lo:hi] = av[lo:hi] @ wv[e].t()
        return float((y * c.double()).sum())

    da = api.ragged_gemm(c, w, off, transpose=True, out_dtype=F32).double()
    dw = api.ragged_wgrad(c, a, off).double()
    for seed in range(3):
        u, v = rnd(50 + seed, 65, 48).double(), rnd(60 + seed, 3, 56, 48).double()
        fa = (loss(a.double() + 0.5 * u, w.double()) - loss(a.double() - 0.5 * u, w.double()))
        fw = (loss(a.double(), w.double() + 0.5 * v) - loss(a.double(), w.double() - 0.5 * v))
        # bounds: f32 sums of 56 (65) products, weighted by |u| (|v|)
        ba = float((sum_bound(57, (c.double().abs() @ torch.ones(56, 48, dtype=torch.float64, device=cuda)) * w.double().abs().max()) * u.abs()).sum())
        bw = float((sum_bound(66, 65 * c.double().abs().max() * a.double().abs().max()) * v.abs()).sum())
        assert abs(float((da * u).sum()) - fa) <= ba + 1e-6
        assert abs(float((dw * v).sum()) - fw) <= bw + 1e-6


def test_bounded_wait_expiry_reports_timeout(cuda):
    """The pair's epilogues wait for a signal that never comes: the bound ends
    them, the status says so, nothing is written, and the next call is right."""
    from quantization_nvfp4_quantize_b200 import _lib
    lib = _lib.load()
    a, w, off = rnd(70, 100, 128), rnd(71, 1, 200, 128), offsets_of([100], cuda)
    out = torch.full((100, 200), 3.0, device=cuda)
    status = torch.zeros(1, dtype=I32, device=cuda)
    p = api._p
    st = lib.nvfp4_debug_ragged_wait_expiry(p(a), 128, 100, p(w), 200, 128, p(off), p(out), 200, p(status), 20_000_000,
                                            api._stream(cuda))
    assert st == 0
    torch.cuda.synchronize()
    assert api.read_status(status) == 5 and bool((out == 3).all())
    got = api.ragged_gemm(a, w, off, out_dtype=F32)
    y, s = ref_rows(a, w, off, False, torch.zeros(100, 200, device=cuda))
    check(got, y, sum_bound(128, s) + rounding(F32, y))


@pytest.mark.parametrize("counts,N,K", [([64], 8, 8), ([1, 64, 0, 130], 264, 72), ([300, 1, 700], 520, 328),
                                        ([2000, 0, 3, 64], 136, 256)], ids=str)
def test_rows_of_no_kept_row_add_nothing(cuda, counts, N, K):
    """Rows whose index lies outside the kept tensor, with Inf and NaN in g:
    alone in a stage, whole stages of them, a segment without any other, the
    last rows of a segment."""
    E, M, T = len(counts), sum(counts) + 5, 40
    off = offsets_of(counts, cuda, start=2)
    a8 = api.act8_quantize(rnd(81, T, -(-K // 8) * 8)[:, :K])
    gen = torch.Generator().manual_seed(82)
    g = rnd(83, M, N, scale=0.1)
    for pick in ("few", "stage", "segment", "ends", "all"):
        rows = torch.randint(0, T, (M,), generator=gen).to(I32).to(cuda)
        gone = torch.zeros(M, dtype=torch.bool, device=cuda)
        if pick == "few":
            gone = (torch.rand(M, generator=gen) < 0.02).to(cuda)
            gone[2 + counts[0] // 2] = True
        elif pick == "stage":
            gone[2:66] = True
            gone[-70:-6] = True
        elif pick == "segment":
            gone[int(off[-2]):int(off[-1])] = True
        elif pick == "ends":
            gone[(off[1:].long() - 1).clamp_min(0)] = True
            gone[off[:-1].long()] = True
        else:
            gone[:] = True
        rows[gone] = torch.where(torch.arange(int(gone.sum()), device=cuda) % 2 == 0, -1, T).to(I32)
        bad = g.clone()
        bad[gone] = float("nan")
        bad[gone.nonzero()[::3, 0]] = float("inf")
        full = torch.zeros(M, K, dtype=torch.float64, device=cuda)
        full[~gone] = kept_values(a8)[rows[~gone].long()]
        y, s = ref_wgrad(torch.where(gone[:, None], torch.zeros_like(g), g), full, off)
        got = api.ragged_wgrad(bad, a8, off, a_rows=rows)
        check(got, y, sum_bound(max(counts) + 1, s) + rounding(F32, y), pick)


def test_rows_of_no_kept_row_in_split_segments(cuda):
    """The same where rows are split over the SMs, and added to an old value."""
    M, T, N, K = 6000, 50, 72, 96
    off = torch.tensor([10, 2500, 5990], dtype=I32, device=cuda)
    assert api._lib.load().moe_ragged_wgrad_workspace_size(M, N, K, 2, 1) > M * K * 2
    a8 = api.act8_quantize(rnd(84, T, K))
    gen = torch.Generator().manual_seed(85)
    rows = torch.randint(-3, T + 3, (M,), generator=gen).to(I32).to(cuda)
    gone = (rows < 0) | (rows >= T)
    g = rnd(86, M, N, scale=0.1)
    full = torch.zeros(M, K, dtype=torch.float64, device=cuda)
    full[~gone] = kept_values(a8)[rows[~gone].long()]
    g[gone] = 0
    y, s = ref_wgrad(g, full, off)
    g[gone] = float("nan")
    old = rnd(87, 2, N, K).float()
    got = api.ragged_wgrad(g, a8, off, a_rows=rows, out=old.clone(), accumulate=True)
    z = y + old.double()
    check(got, z, sum_bound(3500, s) + ULP_ADD * (y.abs() + old.double().abs()) + rounding(F32, z))


def test_kept_tensor_without_rows(cuda):
    """No row of g names a kept row: zeros, or the old value, even of NaN."""
    off = offsets_of([20, 0, 100], cuda, start=1)
    a8 = api.Act8.empty(0, 72, cuda)
    g = torch.full((125, 24), float("nan"), dtype=BF16, device=cuda)
    rows = torch.full((125,), -1, dtype=I32, device=cuda)
    rows[50:] = 0
    got = api.ragged_wgrad(g, a8, off, a_rows=rows)
    assert tuple(got.shape) == (3, 24, 72) and not bool(got.any())
    old = rnd(88, 3, 24, 72).float()
    assert torch.equal(api.ragged_wgrad(g, a8, off, a_rows=rows, out=old.clone(), accumulate=True), old)
    none = torch.zeros(4, dtype=I32, device=cuda)
    assert not bool(api.ragged_wgrad(g[:0], a8, none, a_rows=rows[:0]).any())
    assert not bool(api.ragged_wgrad(g[:0], a8, none).any())


def test_long_segment_under_a_short_wait_limit(cuda):
    """The bound of a wait is on a stage that makes no progress, not on the time
    to a far one: a segment of 2^25 + 5 rows (about 0.1 s) whose last, ragged
    stage another warp waits for from the start, with every wait bounded at 5
    ms.  Ones and small whole numbers: the sums are exact."""
    from quantization_nvfp4_quantize_b200 import _lib
    E, N, K, M = 75, 8, 8, 2 ** 25 + 5                             # enough experts for no row splits
    off = torch.full((E + 1,), M, dtype=I32, device=cuda)
    off[0] = 0
    g = torch.zeros(M, N, dtype=BF16, device=cuda)
    g[::64] = 1
    a = torch.ones(M, K, dtype=BF16, device=cuda)
    a[-1] = 2
    g[-1] = 1
    out = torch.full((E, N, K), 7.0, device=cuda)
    status = torch.zeros(1, dtype=I32, device=cuda)
    assert api._lib.load().moe_ragged_wgrad_workspace_size(M, N, K, E, 0) == 0
    p = api._p
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    assert _lib.load().nvfp4_debug_ragged_wgrad_wait_limit(p(g), N, M, p(a), K, N, K, E, p(off), p(out), p(status),
                                                           5_000_000, api._stream(cuda)) == 0
    end.record()
    torch.cuda.synchronize()
    assert api.read_status(status) == 0
    want = float(g[:, 0].float().double().sum()) + 1               # the last row counts twice
    assert bool((out[0] == want).all()) and not bool(out[1:].any())
    assert start.elapsed_time(end) > 40                            # the case does what its name says


def whole(seed, most, *shape):
    """Whole numbers in [-most, most]: bf16 holds them, and every product and sum
    of the tests below is exact in f32, in any order."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=gen, device="cuda").to(BF16)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("counts", COUNTS + [[1000, 511, 0, 513, 1]], ids=str)
def test_products_of_whole_numbers(cuda, counts, transpose):
    E, M, N, K = len(counts), sum(counts) + 9, 328, 520
    off = offsets_of(counts, cuda, start=3)
    w, a = whole(101, 3, E, N, K), whole(102, 4, M, N if transpose else K)
    for dtype in (F32, BF16):
        fill = torch.full((M, K if transpose else N), 7.0, dtype=dtype, device=cuda)
        y, _ = ref_rows(a, w, off, transpose, fill)
        assert torch.equal(api.ragged_gemm(a, w, off, transpose=transpose, out=fill), y.to(F32).to(dtype))


def whole_gradients(g, a, off, av=None, **kw):
    y, _ = ref_wgrad(g, a if av is None else av, off)
    old = whole(103, 100, *y.shape).float()
    for dtype in (F32, BF16):
        assert torch.equal(api.ragged_wgrad(g, a, off, out_dtype=dtype, **kw), y.to(F32).to(dtype))
        z = (y + old.double()).to(F32).to(dtype)
        assert torch.equal(api.ragged_wgrad(g, a, off, out=old.to(dtype, copy=True), accumulate=True, **kw), z)


@pytest.mark.parametrize("counts", COUNTS + [[1000, 511, 0, 513, 1], [4001, 64, 2500]], ids=str)
@pytest.mark.parametrize("N,K", [(8, 8), (264, 72), (520, 328)])
def test_weight_gradient_of_whole_numbers(cuda, counts, N, K):
    """One lost, doubled or foreign row shows."""
    M = sum(counts) + 9
    g, a = whole(104, 2, M, N), whole(105, 3, M, K)
    g[:2], a[:2], g[-7:], a[-7:] = float("nan"), float("inf"), float("nan"), float("inf")
    whole_gradients(g, a, offsets_of(counts, cuda, start=2))


@pytest.mark.parametrize("E,M,N,K", [(1, 20000, 64, 96), (3, 9001, 256, 264), (2, 5000, 300, 40), (1, 600, 8, 8),
                                     (4, 30011, 8, 520)])
def test_split_rows_of_whole_numbers(cuda, E, M, N, K):
    assert api._lib.load().moe_ragged_wgrad_workspace_size(M, N, K, E, 0) > 0
    cuts = sorted([5] + [int(M * f) for f in (0.13, 0.52, 0.521)][: E - 1] + [M - 3])
    off = torch.tensor(cuts, dtype=I32, device=cuda)
    whole_gradients(whole(106, 2, M, -(-N // 8) * 8)[:, :N], whole(107, 3, M, K), off)


@pytest.mark.parametrize("counts", COUNTS[1:] + [[4001, 64, 2500]], ids=str)
@pytest.mark.parametrize("N,K", [(8, 8), (264, 333), (520, 528)])
def test_kept_rows_of_whole_numbers(cuda, counts, N, K):
    E, M, T = len(counts), sum(counts) + 4, 50
    x = torch.zeros(T, -(-K // 8) * 8, dtype=BF16, device=cuda)[:, :K]
    x.copy_(whole(108, 3, T, K))
    a8 = api.act8_quantize(x)
    assert torch.equal(kept_values(a8), x.double())                # 3 significant bits at most
    rows = torch.randint(-2, T + 2, (M,), generator=torch.Generator().manual_seed(109)).to(I32).to(cuda)
    ok = (rows >= 0) & (rows < T)
    av = torch.where(ok[:, None], x.double()[rows.clamp(0, T - 1).long()], 0.0)
    whole_gradients(whole(110, 2, M, N), a8, offsets_of(counts, cuda, start=1), av, a_rows=rows)


def test_whole_numbers_behind_long_offsets(cuda):
    """Rows whose element offsets pass 2^31, split over the SMs: exact."""
    M, N, K = 1_100_000, 64, 2048
    off = torch.tensor([M - 300, M - 100, M], dtype=I32, device=cuda)
    assert api._lib.load().moe_ragged_wgrad_workspace_size(M, N, K, 2, 0) > 0
    a = torch.full((M, K), 3.0, dtype=BF16, device=cuda)
    g = torch.full((M, N), 2.0, dtype=BF16, device=cuda)
    a[-300:], g[-300:] = whole(111, 3, 300, K), whole(112, 2, 300, N)
    y, _ = ref_wgrad(g[-300:], a[-300:], offsets_of([200, 100], cuda))
    assert torch.equal(api.ragged_wgrad(g, a, off).double(), y)
    w = whole(113, 3, 2, N, K)
    y, _ = ref_rows(a[-300:], w, offsets_of([200, 100], cuda), False, torch.zeros(300, N, device=cuda))
    assert torch.equal(api.ragged_gemm(a, w, off, out_dtype=F32)[-300:].double(), y)


def test_weight_gradient_long_sums(cuda):
    """131072 terms of one sign: at most 512 rows are summed on the tensor core.
    32 MMAs of 16 exact products and the sum so far: 17 terms cut to the
    largest's 24 bits each; then 256 additions in f32 (2^-24 each).  (One sum
    over as many terms on the tensor core was seen to be off by more.)"""
    E, N, K, M = 75, 16, 64, 131072                                # enough experts for no row splits
    off = torch.full((E + 1,), M, dtype=I32, device=cuda)
    off[0] = 0
    g, a = rnd(114, M, N).abs(), rnd(115, M, K).abs()
    assert api._lib.load().moe_ragged_wgrad_workspace_size(M, N, K, E, 0) == 0
    bar = (32 * 17 + 256 + 1) * 2.0 ** -24
    want = g.double().t() @ a.double()
    got = api.ragged_wgrad(g, a, off)[0].double()
    assert float(((got - want) / want).abs().max()) <= bar
    # with the rows split over the SMs the parts are added in f32 as well
    got = api.ragged_wgrad(g, a, off[[0, E]])[0].double()
    assert float(((got - want) / want).abs().max()) <= bar + 64 * 2.0 ** -24


def test_rows_of_no_kept_row_with_either_workspace(cuda):
    """The C call with and without room for the expanding launch's word gives
    the same bits, with and without such rows, from any alignment of the index."""
    import ctypes

    from quantization_nvfp4_quantize_b200 import _lib
    lib, p = _lib.load(), api._p
    M, T, N, K = 3001, 77, 264, 136
    a8 = api.act8_quantize(rnd(120, T, K))
    off = offsets_of([1000, 0, 1990], cuda, start=4)
    for gone in ([], [2999], [5, 6, 1700], list(range(0, 3001, 3))):
        for at in range(4):
            rows = torch.zeros(M + 4, dtype=I32, device=cuda)[at:at + M]
            rows.copy_(torch.randint(0, T, (M,), generator=torch.Generator().manual_seed(121)))
            g = rnd(122, M, N, scale=0.1)
            rows[gone] = -1
            g[gone] = float("nan")
            want = api.ragged_wgrad(g, a8, off, a_rows=rows)
            assert bool(torch.isfinite(want).all())
            sizes = [lib.moe_ragged_wgrad_workspace_size(M, N, K, 3, k) for k in (1, 2)]
            assert 0 < sizes[1] - sizes[0] <= 4096
            for size in sizes:
                ws = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device=cuda)
                out = torch.empty(3, N, K, device=cuda)
                assert lib.moe_ragged_wgrad(p(g), N, M, p(a8.codes), a8.codes.stride(0), p(a8.scales), a8.scales.stride(0),
                                            p(rows), T, N, K, 3, p(off), p(out), 1, 0, p(ws), ctypes.c_size_t(size), None,
                                            api._stream(cuda)) == 0
                assert torch.equal(out, want) and bool((ws[size:] == 0xFF).all())
