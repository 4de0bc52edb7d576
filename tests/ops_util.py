"""Plain 64-bit forms and error bounds for the experts' training and decode
operators (test infrastructure)."""
import torch

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32

# Sums on the tensor cores: bf16 x bf16 products are exact in f32; every one of
# the at most n additions errs by at most one unit in the last place (2^-23,
# truncation counted) of a partial sum that is at most sum |products|.
ULP32 = 2.0 ** -23


def sum_bound(n, abs_sum):
    return n * ULP32 * abs_sum


def rounding(dtype, y):
    """Half a step of `dtype` at y."""
    return torch.finfo(dtype).eps / 2 * y.abs() + torch.finfo(dtype).smallest_normal


def check(got, want, bound, what=""):
    """|got - want| <= bound elementwise, non-finite places equal."""
    got = got.double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin), f"{what}: non-finite values differ"
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN places differ"
    err = torch.where(fin, (got - want).abs() - bound, torch.zeros_like(want))
    worst = float(err.max()) if err.numel() else 0.0
    assert worst <= 0, f"{what}: over the bound by {worst}"


def offsets_of(counts, dev, start=0):
    off = [start]
    for c in counts:
        off.append(off[-1] + c)
    return torch.tensor(off, dtype=I32, device=dev)


def e4m3(v):
    """Nearest E4M3 value (ties to even) of |v| <= 448, in 64 bits."""
    _, ex = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (ex - 1).clamp_min(-6) - 3)
    return torch.round(v / step) * step


def keep(x):
    """Definition of the 8-bit activations in 64 bits: (values, scale bytes
    with the padded row)."""
    m, k = x.shape
    pad = -(-k // 128) * 128
    g = torch.zeros(m, pad, dtype=F64, device=x.device)
    g[:, :k] = x.double()
    g = g.view(m, pad // 32, 32)
    bad = ~torch.isfinite(g).all(2)
    top = torch.where(bad[:, :, None], torch.zeros_like(g), g).abs().amax(2)
    p = torch.full_like(top, -120.0)
    for q in range(-120, 121):                      # smallest p with top <= 448 * 2^p
        p = torch.where(top > 448.0 * 2.0 ** (q - 1), torch.full_like(p, float(q)), p)
    p = torch.where(top == 0, torch.zeros_like(p), p)
    s = torch.exp2(p)[:, :, None]
    v = torch.where(bad[:, :, None], torch.full_like(g, float("nan")), e4m3(torch.where(bad[:, :, None], 0.0 * s, g) / s) * s)
    byte = torch.where(bad, torch.full_like(p, 255.0), p + 127)
    return v.view(m, pad)[:, :k], byte.to(torch.uint8)


def kept_values(a):
    """Act8 -> its values in 64 bits."""
    m, k = a.codes.shape
    c = a.codes.contiguous().view(torch.float8_e4m3fn).double()
    s = a.scales[:, : -(-k // 32)].double()
    f = torch.where(s == 255, torch.full_like(s, float("nan")), torch.exp2(s - 127))
    return c * f.repeat_interleave(32, 1)[:, :k]
