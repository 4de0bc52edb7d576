"""Products of a few tokens with NVFP4 weights against 64-bit products of the
dequantized weights.  Bound: products e2m1 * sf * x are exact in f32 (at most 6
+ 8 significant bits), K additions and the final scalings err by at most 2^-23
of sum |products| each."""
import numpy as np
import pytest
import torch

import oracle
from ops_util import BF16, F32, F64, I32, check, rounding, sum_bound
from quantization_nvfp4_quantize_b200 import api

pytestmark = pytest.mark.gpu


def rnd(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF16)


def weights(seed, E, N, K):
    """NVFP4 weights from the library's quantizer and their values (64 bits)
    through the oracle's scale layout."""
    w = rnd(seed, E, N, K, scale=0.02)
    w[:, 0] *= 30.0                                        # rows with other block scales
    _, s, codes, sf = api.qdq_weights(w, want_qdq=False, want_packed=True)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=F64, device=w.device)
    c = codes.view(E, N, K // 2)
    v = torch.stack([grid[(c & 15).int()], grid[(c >> 4).int()]], -1).view(E, N, K)
    per = sf.numel() // E
    scale = torch.stack([torch.from_numpy(oracle.unswizzle_scales(sf.view(-1)[e * per:(e + 1) * per].cpu().numpy(), N, K).copy())
                         for e in range(E)]).to(w.device).view(torch.float8_e4m3fn).double()
    return codes, sf, s, v * scale.repeat_interleave(16, 2) * s.double()[:, None, None]


def bound(K, x, w):
    return sum_bound(K + 8, torch.bmm(w.abs(), x.abs()[:, :, None])[:, :, 0])


def check_swiglu(h, y, b):
    """h against the SwiGLU of y = [gate | up], known to b."""
    n = y.shape[1] // 2
    a, u, ba, bu = y[:, :n], y[:, n:], b[:, :n], b[:, n:]
    sig = torch.sigmoid(a)
    want = a * sig * u
    # d silu / da <= 1.1; f32 sigmoid as in the SwiGLU tests
    lim = 1.1 * ba * (u.abs() + bu) + (a * sig).abs() * bu + (16 + a.abs()) * 2.0 ** -23 * want.abs()
    check(h, want, 1.01 * lim + rounding(BF16, want.abs() + lim))


@pytest.mark.parametrize("T,E,kr", [(1, 8, 2), (1, 5, 1), (3, 16, 8), (9, 4, 3)])
@pytest.mark.parametrize("N,K", [(16, 64), (130, 128), (256, 192), (1536, 2048), (34, 704)])
def test_store_and_swiglu(cuda, T, E, kr, N, K):
    codes, sf, s, w = weights(N + K, E, N, K)
    x = rnd(2, T, K)
    idx = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:kr] for t in range(T)]).to(I32).to(cuda)
    flat = idx.view(-1).long()
    xr = x.double().repeat_interleave(kr, 0)
    y = torch.bmm(w[flat], xr[:, :, None])[:, :, 0]
    b = bound(K, xr, w[flat])
    got = api.nvfp4_gemv(x, codes, sf, s, N, K, expert_idx=idx)
    check(got, y, b + rounding(F32, y))
    h = api.nvfp4_gemv(x, codes, sf, s, N, K, expert_idx=idx, epilogue=api.EPI_SWIGLU_BF16)
    check_swiglu(h, y, b)


@pytest.mark.parametrize("T,E,kr", [(1, 8, 8), (2, 5, 1), (16, 32, 8), (5, 4, 3)])
@pytest.mark.parametrize("N,K", [(8, 64), (130, 192), (2048, 768)])
@pytest.mark.parametrize("gated", [False, True])
def test_combine(cuda, T, E, kr, N, K, gated):
    codes, sf, s, w = weights(N + K + 1, E, N, K)
    x = rnd(3, T * kr, K)
    idx = torch.randint(0, E, (T, kr), generator=torch.Generator().manual_seed(4)).to(I32).to(cuda)   # repeats allowed
    gate = torch.rand(T, kr, generator=torch.Generator().manual_seed(5)).to(cuda) if gated else None
    flat = idx.view(-1).long()
    c = torch.ones(T * kr, dtype=F64, device=cuda) if gate is None else gate.double().view(-1)
    y = torch.bmm(w[flat], x.double()[:, :, None])[:, :, 0] * c[:, None]
    b = bound(K + kr, x.double(), w[flat]) * c[:, None]
    got = api.nvfp4_gemv(x, codes, sf, s, N, K, expert_idx=idx, epilogue=api.EPI_COMBINE_F32, gate=gate)
    want = y.view(T, kr, N).sum(1)
    check(got, want, b.view(T, kr, N).sum(1) + rounding(F32, want))
    assert torch.equal(got, api.nvfp4_gemv(x, codes, sf, s, N, K, expert_idx=idx, epilogue=api.EPI_COMBINE_F32, gate=gate))


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 33])
@pytest.mark.parametrize("N,K", [(1, 64), (48, 320), (640, 1024)])
def test_dense(cuda, T, N, K):
    codes, sf, s, w = weights(N + K + 2, 1, N, K)
    x = rnd(6, T, K)
    y = x.double() @ w[0].t()
    got = api.nvfp4_gemv(x, codes, sf, s, N, K)
    check(got, y, sum_bound(K + 8, x.double().abs() @ w[0].abs().t()) + rounding(F32, y))
    if N % 2 == 0:
        h = api.nvfp4_gemv(x, codes, sf, s, N, K, epilogue=api.EPI_SWIGLU_BF16)
        b = sum_bound(K + 8, x.double().abs() @ w[0].abs().t())
        check_swiglu(h, y, b)
        idx = torch.zeros(T, 1, dtype=I32, device=cuda)
        check_swiglu(api.nvfp4_gemv(x, codes, sf, s, N, K, expert_idx=idx, epilogue=api.EPI_SWIGLU_BF16), y, b)
    c = api.nvfp4_gemv(x, codes, sf, s, N, K, epilogue=api.EPI_COMBINE_F32)
    check(c, y, sum_bound(K + 8, x.double().abs() @ w[0].abs().t()) + rounding(F32, y))


def test_many_tokens_share_experts(cuda):
    """More pairs than one launch lists, more tokens per expert than one pass."""
    T, E, kr, N, K = 300, 5, 4, 48, 192
    codes, sf, s, w = weights(20, E, N, K)
    x = rnd(21, T, K)
    idx = torch.randint(-1, E, (T, kr), generator=torch.Generator().manual_seed(22)).to(I32).to(cuda)
    flat = idx.view(-1).long()
    live = (flat >= 0).double()[:, None]
    wf = w[flat.clamp_min(0)]
    xr = x.double().repeat_interleave(kr, 0)
    y = torch.bmm(wf, xr[:, :, None])[:, :, 0] * live
    check(api.nvfp4_gemv(x, codes, sf, s, N, K, expert_idx=idx), y, bound(K, xr, wf) * live + rounding(F32, y))
    xc = rnd(23, T * kr, K)
    y = torch.bmm(wf, xc.double()[:, :, None])[:, :, 0] * live
    got = api.nvfp4_gemv(xc, codes, sf, s, N, K, expert_idx=idx, epilogue=api.EPI_COMBINE_F32)
    want = y.view(T, kr, N).sum(1)
    check(got, want, (bound(K + kr, xc.double(), wf) * live).view(T, kr, N).sum(1) + rounding(F32, want))


def test_every_code_and_scale_decodes_exactly(cuda):
    """One-hot x: every E2M1 code under every E4M3 scale, exact."""
    N, K = 128, 64
    codes = torch.zeros(1, N, K // 2, dtype=torch.uint8, device=cuda)
    for c in range(16):
        codes[0, :, c // 2] |= c << (4 * (c & 1))                  # element c of block 0 holds code c
    rows = torch.arange(N, device=cuda)
    sfm = np.zeros((N, K // 16), np.uint8)
    sfm[:, 0] = np.minimum(np.arange(N), 126)
    sf = torch.from_numpy(oracle.swizzle_scales(sfm)).to(cuda).view(1, -1)
    s = torch.ones(1, device=cuda)
    x = torch.zeros(16, K, dtype=BF16, device=cuda)
    x[torch.arange(16), torch.arange(16)] = 1.0
    got = api.nvfp4_gemv(x, codes, sf, s, N, K)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=F64, device=cuda)
    scale = rows.clamp_max(126).to(torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(got.double(), grid[:, None] * scale[None, :])


def test_bad_expert_gives_zeros_and_rows_keep_apart(cuda):
    E, N, K = 3, 96, 128
    codes, sf, s, w = weights(9, E, N, K)
    x = rnd(10, 2, K)
    idx = torch.tensor([[0, -1], [3, 2]], dtype=I32, device=cuda)
    got = api.nvfp4_gemv(x, codes, sf, s, N, K, expert_idx=idx)
    assert not bool(got[1].any()) and not bool(got[2].any()) and bool(got[0].any()) and bool(got[3].any())
    xc = rnd(11, 4, K)
    xc[1:3] = float("nan")                                          # rows of no expert
    y = api.nvfp4_gemv(xc, codes, sf, s, N, K, expert_idx=idx, epilogue=api.EPI_COMBINE_F32)
    assert bool(torch.isfinite(y).all())
    x[0, 5] = float("inf")
    got = api.nvfp4_gemv(x, codes, sf, s, N, K, expert_idx=torch.tensor([[0], [0]], dtype=I32, device=cuda))
    assert bool(torch.isfinite(got[1]).all())
    dense = api.nvfp4_gemv(x, codes[:1], sf.view(E, -1)[:1], s[:1], N, K)
    assert bool(torch.isfinite(dense[1]).all())


def test_strides_and_surroundings(cuda):
    E, N, K = 2, 50, 64
    codes, sf, s, w = weights(12, E, N, K)
    x = rnd(13, 3, 2 * K)[:, 8:8 + K]
    idx = torch.tensor([[0, 1], [1, 0], [1, 1]], dtype=I32, device=cuda)
    buf = torch.full((6, N + 5), 4.0, device=cuda)
    api.nvfp4_gemv(x, codes, sf, s, N, K, expert_idx=idx, out=buf[:, 2:2 + N])
    assert torch.equal(buf[:, 2:2 + N], api.nvfp4_gemv(x.contiguous(), codes, sf, s, N, K, expert_idx=idx))
    assert bool((buf[:, :2] == 4).all()) and bool((buf[:, 2 + N:] == 4).all())


@pytest.mark.parametrize("K", [64, 192, 704, 1024])
def test_rows_on_16_and_32_bytes(cuda, K):
    """Rows of x that start on 16 bytes only are loaded in smaller pieces: the
    same bits."""
    E, N, T, kr = 6, 160, 11, 3
    codes, sf, s, w = weights(20, E, N, K)
    idx = torch.randint(0, E, (T, kr), dtype=I32, device=cuda)
    gate = torch.rand(T, kr, device=cuda)
    for form, rows, g in ((api.EPI_STORE_F32, T, None), (api.EPI_SWIGLU_BF16, T, None),
                          (api.EPI_COMBINE_F32, T * kr, gate), (api.EPI_COMBINE_F32, kr, gate[:1])):
        i = idx[:g.shape[0]] if g is not None else idx
        x = rnd(21, rows, 2 * K)[:, :K].contiguous()
        wide = torch.full((rows, K + 24), float("nan"), dtype=x.dtype, device=cuda)
        wide[:, 8:8 + K] = x
        a = api.nvfp4_gemv(x, codes, sf, s, N, K, expert_idx=i, epilogue=form, gate=g)
        assert torch.equal(a, api.nvfp4_gemv(wide[:, 8:8 + K], codes, sf, s, N, K, expert_idx=i, epilogue=form, gate=g))


def test_long_sums(cuda):
    """Sums of 8192 terms of one sign.  A chunk of 128 columns is 8 MMAs of 16
    exact products and the sum so far: 17 terms cut to the largest's 24 bits,
    8 * 17 * 2^-24 in all; 64 chunks and 4 warps are added in f32 (2^-24 each),
    and the scale of the sum is rounded twice."""
    N, K = 32, 8192
    codes, sf, s, w = weights(22, 1, N, K)
    codes = codes & 0x77
    x = rnd(23, 3, 2 * K)[:, :K].abs().contiguous()
    got = api.nvfp4_gemv(x, codes, sf, s, N, K)
    want = x.double() @ w.abs()[0].t()
    assert float(((got.double() - want).abs() / want).max()) <= (8 * 17 + 64 + 4 + 2) * 2.0 ** -24


@pytest.mark.parametrize("T,E,kr", [(2, 128, 8), (3, 128, 8), (4, 128, 8), (3, 128, 11)])
def test_combine_of_a_few_tokens(cuda, T, E, kr):
    """Two to four tokens on both sides of the form's border (T * k_r = E / 4):
    every token has its own x, gates and output row."""
    N, K = 97, 192
    codes, sf, s, w = weights(30, E, N, K)
    x = rnd(31, T * kr, K)
    idx = torch.randint(0, E, (T, kr), generator=torch.Generator().manual_seed(32)).to(I32).to(cuda)
    gate = torch.rand(T, kr, generator=torch.Generator().manual_seed(33)).to(cuda)
    flat = idx.view(-1).long()
    y = torch.bmm(w[flat], x.double()[:, :, None])[:, :, 0] * gate.double().view(-1, 1)
    b = bound(K + kr, x.double(), w[flat]) * gate.double().view(-1, 1)
    buf = torch.full((T, N + 6), 4.0, device=cuda)
    api.nvfp4_gemv(x, codes, sf, s, N, K, expert_idx=idx, epilogue=api.EPI_COMBINE_F32, gate=gate, out=buf[:, 1:1 + N])
    want = y.view(T, kr, N).sum(1)
    check(buf[:, 1:1 + N], want, b.view(T, kr, N).sum(1) + rounding(F32, want))
    assert bool((buf[:, :1] == 4).all()) and bool((buf[:, 1 + N:] == 4).all())


@pytest.mark.parametrize("T,E,kr", [(1, 8, 4), (2, 128, 8), (4, 128, 8), (2, 8, 4), (3, 128, 11), (300, 8, 4)])
def test_combine_skips_experts_that_do_not_exist(cuda, T, E, kr):
    """Such a slot adds nothing, whatever its gate and its row of x hold, in
    every form."""
    N, K = 40, 64
    codes, sf, s, _ = weights(34, E, N, K)
    x = rnd(35, T * kr, K)
    idx = torch.randint(0, E, (T, kr), generator=torch.Generator().manual_seed(36)).to(I32).to(cuda)
    gate = torch.rand(T, kr, generator=torch.Generator().manual_seed(37)).to(cuda)
    gone = torch.rand(T, kr, generator=torch.Generator().manual_seed(38)).to(cuda) < 0.3
    gone[0, 1], gone[-1, 0] = True, True
    run = lambda: api.nvfp4_gemv(x, codes, sf, s, N, K, expert_idx=idx, epilogue=api.EPI_COMBINE_F32, gate=gate)
    gate[gone] = 0.0
    want = run()
    idx[gone] = torch.where(torch.arange(int(gone.sum()), device=cuda) % 2 == 0, -1, E).to(I32)
    gate[gone] = float("nan")
    gate[0, 1] = float("inf")
    x[gone.view(-1)] = float("nan")
    got = run()
    assert bool(torch.isfinite(got).all())
    assert torch.equal(got, want)        # the sums' order goes by the slots, missing ones included


@pytest.mark.parametrize("T,E,kr", [(1, 8, 8), (2, 128, 8), (3, 16, 5), (16, 32, 8), (300, 5, 4)])
@pytest.mark.parametrize("N,K", [(8, 64), (130, 192), (96, 704), (258, 2048)])
def test_whole_numbers(cuda, T, E, kr, N, K):
    """Block and tensor scales of 1, whole x, gates that are powers of two: every
    sum is exact, so one lost or doubled column, token or slot shows."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(40)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=gen, dtype=torch.uint8, device=cuda)
    sf = torch.full((E, -(-N // 128) * 128 * (K // 16)), 0x38, dtype=torch.uint8, device=cuda)     # E4M3 1.0
    s = torch.ones(E, device=cuda)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=F64, device=cuda)
    w = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], -1).view(E, N, K)
    idx = torch.randint(-1, E + 1, (T, kr), generator=gen, device=cuda).to(I32)
    flat = idx.view(-1).long()
    live = ((flat >= 0) & (flat < E)).double()[:, None]
    wf = w[flat.clamp(0, E - 1)]
    x = torch.randint(-4, 5, (T, K), generator=gen, device=cuda).to(BF16)
    y = torch.bmm(wf, x.double().repeat_interleave(kr, 0)[:, :, None])[:, :, 0] * live
    assert torch.equal(api.nvfp4_gemv(x, codes, sf, s, N, K, expert_idx=idx).double(), y)
    xc = torch.randint(-4, 5, (T * kr, K), generator=gen, device=cuda).to(BF16)
    gate = torch.exp2(torch.randint(-2, 3, (T, kr), generator=gen, device=cuda).float())
    y = torch.bmm(wf, xc.double()[:, :, None])[:, :, 0] * live * gate.double().view(-1, 1)
    got = api.nvfp4_gemv(xc, codes, sf, s, N, K, expert_idx=idx, epilogue=api.EPI_COMBINE_F32, gate=gate)
    assert torch.equal(got.double(), y.view(T, kr, N).sum(1))
