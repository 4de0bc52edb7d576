"""Activations kept in 8 bits, the SwiGLU around them, the combine of routed
rows and the router's gradient against their definitions in 64 bits."""
import pytest
import torch

from ops_util import BF16, F32, F64, I32, check, keep, kept_values, rounding
from quantization_nvfp4_quantize_b200 import api

pytestmark = pytest.mark.gpu


def rnd(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF16)


def padded(x, extra=0):
    """x on a row stride that is a multiple of 8 elements."""
    ld = -(-x.shape[1] // 8) * 8 + extra
    buf = torch.zeros(x.shape[0], ld, dtype=BF16, device=x.device)
    buf[:, : x.shape[1]] = x
    return buf[:, : x.shape[1]]


@pytest.mark.parametrize("M,K", [(1, 1), (3, 31), (5, 32), (7, 33), (64, 127), (33, 128), (200, 257), (17, 4096),
                                 (5000, 72), (1, 8192)])
def test_quantize_matches_definition(cuda, M, K):
    x = rnd(1, M, K).float()
    x *= torch.exp2(torch.randint(-140, 118, (M, 1), generator=torch.Generator().manual_seed(2)).float()).to(cuda)
    x[:, : K // 3] *= 0.01
    x = padded(x.to(BF16), 8 if M % 2 else 0)
    v, s = keep(x)
    q = api.act8_quantize(x)
    assert torch.equal(q.scales, s)
    assert torch.equal(kept_values(q), v)
    back = api.act8_dequantize(q)
    assert torch.equal(back.double(), v)                       # exact in bf16


def test_quantize_every_bf16_value(cuda):
    """Each finite bf16 value alone in its group, and against a group maximum
    that puts it anywhere in E4M3's range."""
    bits = torch.arange(65536, dtype=torch.int32, device=cuda).to(torch.int16)
    vals = bits.view(BF16)
    vals = vals[torch.isfinite(vals) & (vals.abs() < 2.0 ** 127)]
    x = torch.zeros(vals.numel(), 64, dtype=BF16, device=cuda)
    x[:, 5] = vals
    x[:, 40] = vals
    x[:, 41] = (vals.float() * 300.0).clamp(-2.0 ** 126, 2.0 ** 126).to(BF16)
    v, s = keep(x)
    q = api.act8_quantize(x)
    assert torch.equal(q.scales, s) and torch.equal(kept_values(q), v)
    assert torch.equal(torch.signbit(q.codes.view(torch.float8_e4m3fn).float()), torch.signbit(x.float()))


def test_infinities_and_nan_mark_their_group(cuda):
    x = rnd(3, 6, 200)
    x[1, 40], x[2, 199], x[3, 0] = float("inf"), float("-inf"), float("nan")
    v, s = keep(x)
    q = api.act8_quantize(x)
    assert torch.equal(q.scales, s)
    got = kept_values(q)
    assert torch.equal(torch.isnan(got), torch.isnan(v)) and torch.equal(got.nan_to_num(0.5), v.nan_to_num(0.5))
    assert torch.equal(torch.isnan(api.act8_dequantize(q).double()), torch.isnan(v))


def test_strided_output_keeps_its_surroundings(cuda):
    x = rnd(4, 20, 100)
    x = padded(x)
    codes = torch.full((20, 160), 9, dtype=torch.uint8, device=cuda)
    scales = torch.full((20, 12), 9, dtype=torch.uint8, device=cuda)
    q = api.act8_quantize(x, out=api.Act8(codes[:, :100], scales[:, :4]))
    assert torch.equal(kept_values(q), keep(x)[0])
    assert bool((codes[:, 100:] == 9).all()) and bool((scales[:, 4:] == 9).all())
    out = torch.full((20, 120), 3.0, dtype=BF16, device=cuda)
    api.act8_dequantize(q, out=out[:, :100])
    assert bool((out[:, 100:] == 3).all()) and torch.equal(out[:, :100].double(), keep(x)[0])


# sigmoid in f32: the exponential, the sum and the quotient err by a few units
# in the last place each, and the rounding of exp's argument by |a| 2^-24; the
# chains below have at most 8 more f32 operations.
def chain(a):
    return (16 + a.abs()) * 2.0 ** -23


@pytest.mark.parametrize("M,I", [(1, 32), (3, 96), (61, 768), (500, 64), (7, 1536), (2000, 32)])
def test_swiglu_with_kept_inputs(cuda, M, I):
    y = rnd(5, M, 2 * I, scale=3.0)
    y[0, 0], y[0, 1], y[0, 2] = -200.0, 200.0, 0.0
    h, q = api.swiglu_act8(y)
    v, s = keep(y)
    assert torch.equal(q.scales, s) and torch.equal(kept_values(q), v)
    a, b = y[:, :I].double(), y[:, I:].double()
    want = a * torch.sigmoid(a) * b
    check(h, want, rounding(BF16, want) + chain(a) * want.abs() * 1.01 + 1e-37 * (a * b).abs())


def ref_backward(q, dh, w):
    v = kept_values(q)
    i = v.shape[1] // 2
    a, b, u = v[:, :i], v[:, i:], dh.double()
    s = torch.sigmoid(a)
    h = a * s * b
    w = torch.ones(v.shape[0], dtype=F64, device=v.device) if w is None else w.double()
    d = w[:, None] * u
    t = a * (1 - s)
    return dict(a=a, da=d * b * s * (1 + t), da_abs=(d * b * s).abs() * (1 + t.abs()), db=d * a * s, gh=w[:, None] * h,
                dg=(u * h).sum(1), dg_abs=(u * h).abs().sum(1))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,I", [(1, 32), (3, 96), (16, 256), (61, 768), (1000, 288), (9, 4096)])
def test_swiglu_backward(cuda, M, I, gated):
    q = api.act8_quantize(rnd(6, M, 2 * I, scale=3.0))
    dh = rnd(7, M, I, scale=0.1)
    w = torch.rand(M, generator=torch.Generator().manual_seed(8)).to(cuda) if gated else None
    dy, gh, dg = api.swiglu_act8_backward(q, dh, row_gate=w)
    r = ref_backward(q, dh, w)
    c = chain(r["a"]) * 1.01
    check(dy[:, :I], r["da"], rounding(BF16, r["da"]) + 2 * c * r["da_abs"], "dgate input")
    check(dy[:, I:], r["db"], rounding(BF16, r["db"]) + c * r["db"].abs(), "dup input")
    check(gh, r["gh"], rounding(BF16, r["gh"]) + c * r["gh"].abs(), "weighted h")
    check(dg, r["dg"], (I + 32) * 2.0 ** -24 * r["dg_abs"] + float(c.max()) * r["dg_abs"], "router weight")
    again = api.swiglu_act8_backward(q, dh, row_gate=w)
    assert torch.equal(again[2], dg)


def test_swiglu_backward_matches_differences(cuda):
    """Against central differences of the 64-bit SwiGLU at the kept inputs."""
    M, I = 5, 64
    q = api.act8_quantize(rnd(9, M, 2 * I))
    dh = rnd(10, M, I)
    w = torch.rand(M, generator=torch.Generator().manual_seed(11)).to(cuda)
    v, u, wd = kept_values(q), dh.double(), w.double()[:, None]

    def loss(y, g):
        a, b = y[:, :I], y[:, I:]
        return (g * u * a * torch.sigmoid(a) * b).sum()

    dy, _, dg = api.swiglu_act8_backward(q, dh, row_gate=w)
    eps = 1e-5
    for seed in range(3):
        d = rnd(12 + seed, M, 2 * I).double()
        num = float((loss(v + eps * d, wd) - loss(v - eps * d, wd)) / (2 * eps))
        # half a bf16 step per element; the difference itself errs by O(eps^2)
        tol = float((rounding(BF16, dy.double()) * 1.02 * d.abs()).sum()) + 1e-5
        assert abs(float((dy.double() * d).sum()) - num) <= tol
    assert abs(float(dg.double().sum()) - float(loss(v, torch.ones_like(wd)))) <= 1e-5 * float((u * v[:, :I] * v[:, I:]).abs().sum())


def test_swiglu_backward_optional_outputs_and_strides(cuda):
    M, I = 40, 96
    q = api.act8_quantize(rnd(13, M, 2 * I))
    dh = rnd(14, M, 128)[:, :I]
    buf = torch.full((M, 2 * I + 16), 2.0, dtype=BF16, device=cuda)
    dy, gh, dg = api.swiglu_act8_backward(q, dh, dy=buf[:, : 2 * I])
    ref = api.swiglu_act8_backward(q, dh.contiguous())
    assert torch.equal(dy, ref[0]) and torch.equal(gh, ref[1]) and torch.equal(dg, ref[2])
    assert bool((buf[:, 2 * I:] == 2).all())


@pytest.mark.parametrize("T,kr,H", [(1, 1, 8), (5, 3, 264), (300, 8, 2048), (2, 32, 4104)])
@pytest.mark.parametrize("gated", [False, True])
def test_combine_rows(cuda, T, kr, H, gated):
    M = T * kr + 3
    rows = rnd(15, M, H)
    dst = torch.randint(0, M, (T, kr), generator=torch.Generator().manual_seed(16)).to(I32).to(cuda)
    dst[0, 0] = -1
    dst[-1, -1] = M
    gate = torch.rand(T, kr, generator=torch.Generator().manual_seed(17)).to(cuda) if gated else None
    got = api.combine_rows(rows, dst, gate=gate)
    ok = ((dst >= 0) & (dst < M)).double()
    w = ok if gate is None else ok * gate.double()
    part = rows.double()[dst.clamp(0, M - 1).long()] * w[:, :, None]
    check(got, part.sum(1), (kr + 1) * 2.0 ** -23 * part.abs().sum(1))


@pytest.mark.parametrize("T,E,kr", [(1, 1, 1), (7, 5, 3), (100, 256, 8), (33, 40, 8)])
def test_route_backward(cuda, T, E, kr):
    """Against autograd of the 64-bit softmax over the selected logits."""
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(18)).to(cuda)
    r = api.route(logits, kr, seg_align=1)
    dg = torch.randn(T * kr, generator=torch.Generator().manual_seed(19)).to(cuda)
    got = api.route_backward(r.topk_idx, r.topk_gate, r.dst_row, dg, E)
    x = logits.double().requires_grad_()
    gates = torch.softmax(x.gather(1, r.topk_idx.long()), 1)
    (gates * dg.double()[r.dst_row.long()]).sum().backward()
    # gates: 2e-6 relative (routing parity); then kr products and sums
    d = dg.double()[r.dst_row.long()].abs()
    lim = torch.zeros(T, E, dtype=F64, device=cuda).scatter_add_(
        1, r.topk_idx.long(), gates.detach() * (d + (gates.detach() * d).sum(1, keepdim=True)))
    check(got, x.grad, (6e-6 + (kr + 4) * 2.0 ** -23) * lim)


def test_unpadded_routing(cuda):
    """seg_align 1: segments without padding, the layout of the ragged products."""
    T, E, kr = 333, 24, 3
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(20)).to(cuda)
    r, p = api.route(logits, kr, seg_align=1), api.route(logits, kr, seg_align=128)
    assert r.m_pad_max == T * kr and int(r.offsets[-1]) == T * kr
    assert torch.equal(r.topk_idx, p.topk_idx) and torch.equal(r.topk_gate, p.topk_gate)
    counts = torch.bincount(r.topk_idx.view(-1).long(), minlength=E)
    assert torch.equal(r.offsets[1:].long(), torch.cumsum(counts, 0))
    tok = r.row_token[r.dst_row.long()]
    assert torch.equal(tok, torch.arange(T, device=cuda, dtype=I32)[:, None].expand(T, kr))
    assert torch.equal(r.row_gate[r.dst_row.long()], r.topk_gate)
