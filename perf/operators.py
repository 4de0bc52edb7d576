"""Operators of the experts' training and decode paths, as workloads.

Five operators around the expert FFN:

  gemm, dgrad    products grouped by expert over ragged row segments: the
                 forward out[r] = a[r] W_e^T and the input gradient
                 out[r] = g[r] W_e
  wgrad          the weight gradient dW_e = sum_r g[r]^T a[r] of the same
                 products, with a in bf16 or kept in 8 bits (and then named by
                 a row index, so that one kept token row serves all its copies)
  keep           activations kept in 8 bits for the backward pass (E4M3 values
                 with one power-of-two scale per 32 columns of a row), alone or
                 together with the SwiGLU whose inputs they are
  swiglu_bwd     the SwiGLU's backward pass from its inputs kept in 8 bits
  matvec         few-token products with NVFP4 weights (E2M1 codes, E4M3 block
                 scales, one f32 scale per tensor), per token and chosen expert

`own` selects what `run` calls: the plain form in elementary torch operations,
or the library.
"""
import math

import torch

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
GROUP = 32                      # columns that share one scale of a kept activation


# --------------------------------------------------------------------- cases

def listed():
    return [
        # a short batch through eight small experts: launch latency; a few rows
        # per expert, one expert empty, rows of the buffer behind the last segment
        dict(name="gemm_short", op="gemm", experts=8, rows=37, n=512, k=512, spare=11, skew=1.0),
        # the trainer's gate/up product: 4096 tokens, top-8 of 128 experts
        dict(name="gemm_gate_up", op="gemm", experts=128, rows=32768, n=1536, k=2048, spare=0, skew=0.3),
        # the input gradient of the down product at the large layer's sizes per expert
        dict(name="dgrad_down", op="dgrad", experts=32, rows=32768, n=4096, k=1536, spare=0, skew=0.5),
        # odd segment lengths and widths off the tile, bf16 result
        dict(name="wgrad_odd", op="wgrad", experts=5, rows=1003, n=520, k=264, kept=False, f32=False, skew=1.0, fan=1),
        # weight gradient of the down product, f32 (the optimizer's type)
        dict(name="wgrad_down", op="wgrad", experts=32, rows=32768, n=4096, k=1536, kept=False, f32=True, skew=0.5,
             fan=1),
        # weight gradient of gate/up from the tokens kept in 8 bits, top-8
        dict(name="wgrad_gate_up_kept", op="wgrad", experts=128, rows=32768, n=1536, k=2048, kept=True, f32=True,
             skew=0.3, fan=8),
        # the large layer's input kept for the backward pass
        dict(name="keep_x", op="keep", rows=16384, width=4096, swiglu=False),
        # SwiGLU of a short batch with its inputs kept
        dict(name="keep_swiglu_short", op="keep", rows=61, width=1536, swiglu=True),
        # SwiGLU backward of a short batch
        dict(name="swiglu_bwd_short", op="swiglu_bwd", rows=16, width=512, gated=True),
        # SwiGLU backward of the trainer's layer
        dict(name="swiglu_bwd", op="swiglu_bwd", rows=32768, width=1536, gated=True),
        # decode of one token: gate/up of its eight experts with SwiGLU
        dict(name="matvec_gate_up", op="matvec", form="swiglu", tokens=1, experts=128, topk=8, n=1536, k=2048),
        # decode of sixteen tokens: down products combined with the router's weights
        dict(name="matvec_down", op="matvec", form="combine", tokens=16, experts=128, topk=8, n=4096, k=1536),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "dgrad", "wgrad", "wgrad", "keep", "swiglu_bwd", "matvec", "matvec"])
    if op in ("gemm", "dgrad", "wgrad"):
        while True:
            c = dict(op=op, experts=_log(rng, 1, 128), rows=_log(rng, 1, 32768), n=8 * _log(rng, 4, 512),
                     k=8 * _log(rng, 4, 256), skew=rng.choice([0.0, 0.3, 1.0]))
            if op == "gemm":
                c["n"] -= rng.choice([0, 0, 1, 3])          # the output's width is free
            # no more work than the largest listed cases
            if 2.0 * c["rows"] * c["n"] * c["k"] <= 4e11 and c["experts"] * c["n"] * c["k"] <= 4e8:
                break
        if op == "wgrad":
            c["kept"] = rng.random() < 0.5
            c["fan"] = rng.choice([1, 2, 8]) if c["kept"] else 1
            c["f32"] = rng.random() < 0.7
        else:
            c["spare"] = rng.choice([0, 0, 5, 200])
        return c
    if op == "keep":
        swiglu = rng.random() < 0.5
        w = GROUP * 2 * _log(rng, 1, 64) if swiglu else _log(rng, 8, 4096)
        return dict(op=op, rows=_log(rng, 1, 16384), width=w, swiglu=swiglu)
    if op == "swiglu_bwd":
        return dict(op=op, rows=_log(rng, 1, 32768), width=GROUP * 2 * _log(rng, 1, 24), gated=rng.random() < 0.7)
    form = rng.choice(["store", "swiglu", "combine", "dense"])
    e = 1 if form == "dense" else _log(rng, 8, 128)
    return dict(op="matvec", form=form, tokens=_log(rng, 1, 16), experts=e, topk=1 if form == "dense" else rng.randint(1, 8),
                n=8 * _log(rng, 4, 512), k=64 * _log(rng, 1, 24))


# -------------------------------------------------------------------- inputs

def _gen(seed, i):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1000003 + i * 7919) & 0x7FFFFFFF)
    return g


def _segments(c, seed):
    """Ragged segment bounds (int32 [E+1]) of `rows` rows over the experts:
    a router's counts, the second expert left empty where there are several."""
    g = torch.Generator()
    g.manual_seed(seed * 31 + 5)
    e = c["experts"]
    p = torch.softmax(c["skew"] * torch.randn(e, generator=g, dtype=F64), 0)
    if e > 2:
        p[1] = 0.0
    counts = torch.bincount(torch.multinomial(p, c["rows"], replacement=True, generator=g), minlength=e)
    off = torch.zeros(e + 1, dtype=torch.int64)
    off[1:] = torch.cumsum(counts, 0)
    return off, int(counts.max())


def _activations(rows, width, g):
    """N(0,1) with one channel in a hundred scaled up: the outlier channels of
    hidden activations."""
    x = torch.randn(rows, width, generator=g, device="cuda")
    scale = torch.exp(2.0 + 0.5 * torch.randn(width, generator=g, device="cuda"))
    pick = torch.rand(width, generator=g, device="cuda") < 0.01
    return (x * torch.where(pick, scale, torch.ones_like(scale))).to(BF16)


def _keep_plain(x):
    """x (any float type) -> (E4M3 values, scale bytes): per 32 columns of a
    row the smallest power of two 2^p, p >= -120, with max|x| <= 448 2^p; the
    byte is p + 127 (127 for a group of zeros; the scale rows are padded to
    whole 128 columns with 127)."""
    m, k = x.shape
    kp = -(-k // 128) * 128
    v = torch.nn.functional.pad(x.to(F32), (0, kp - k)).view(m, kp // GROUP, GROUP)
    amax = v.abs().amax(2)
    mant, ex = torch.frexp(amax)                     # amax = mant 2^ex, mant in [0.5, 1)
    p = (ex - 9 + (mant > 0.875).to(ex.dtype)).clamp_min(-120)
    p = torch.where(amax == 0, torch.zeros_like(p), p)
    q = torch.ldexp(v, -p[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(m, kp)[:, :k].contiguous(), (p + 127).to(torch.uint8)


def _kept_values(codes, scales, dtype):
    m, k = codes.shape
    s = torch.ldexp(torch.ones((), dtype=dtype, device=codes.device), scales.to(I32) - 127)
    return codes.view(torch.float8_e4m3fn).to(dtype) * s.repeat_interleave(GROUP, 1)[:, :k]


def _codes_buffer(q):
    """E4M3 values as the kept codes: uint8 rows on a 16-byte stride."""
    m, k = q.shape
    buf = torch.zeros(m, -(-k // 16) * 16, dtype=torch.uint8, device=q.device)
    buf[:, :k] = q.view(torch.uint8)
    return buf[:, :k]


def _nvfp4_weights(e, n, k, g):
    """E NVFP4 tensors of N(0, 0.02) weights: codes uint8 [E, N, K/2], block
    scales in the tensor-core layout [E, ...], tensor scales f32 [E]."""
    npad = -(-n // 128) * 128
    codes = torch.empty(e, n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(e, npad * (k // 16), dtype=torch.uint8, device="cuda")
    s_t = torch.empty(e, dtype=F32, device="cuda")
    at = _scale_at(n, k, "cuda")
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    step = max(1, int(6e7 // (n * k)))
    for i in range(0, e, step):
        w = torch.randn(min(step, e - i), n, k, generator=g, device="cuda") * 0.02
        st = w.abs().amax((1, 2)) / 2688.0
        b = w.view(w.shape[0], n, k // 16, 16)
        sf = (b.abs().amax(3) / 6.0 / st[:, None, None]).to(torch.float8_e4m3fn)
        d = (sf.float() * st[:, None, None]).clamp_min(1e-30)
        v = b / d[..., None]
        q = (torch.bucketize(v.abs(), edges) + 8 * (v < 0)).to(torch.uint8).view(w.shape[0], n, k // 2, 2)
        codes[i:i + step] = q[..., 0] | (q[..., 1] << 4)
        scales[i:i + step].scatter_(1, at.view(1, -1).expand(w.shape[0], -1),
                                    sf.view(torch.uint8).reshape(w.shape[0], -1))
        s_t[i:i + step] = st
    return codes, scales, s_t


def _scale_at(n, k, device):
    """Byte offset of the scale of (row, 16-column block) inside one tensor's
    scale buffer: 512-byte atoms of 128 rows x 4 blocks."""
    r = torch.arange(n, device=device)[:, None]
    c = torch.arange(k // 16, device=device)[None, :]
    return ((r // 128) * (k // 64) + c // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + c % 4


def prepare(case, seed):
    c, op = case, case["op"]
    g = _gen(seed, 1)
    s = dict(case=c)
    if op in ("gemm", "dgrad", "wgrad"):
        off, longest = _segments(c, seed)
        s["offsets"], s["longest"] = off.to(I32).cuda(), longest
        rows, n, k, e = c["rows"] + c.get("spare", 0), c["n"], c["k"], c["experts"]
        if op == "wgrad":
            s["g"] = torch.randn(rows, n, generator=g, device="cuda").mul_(0.02).to(BF16)
            if c["kept"]:
                tokens = -(-rows // c["fan"])
                q, s["scales"] = _keep_plain(_activations(tokens, k, g))
                s["codes"] = _codes_buffer(q)
                # a token's copies lie in the segments of its experts
                s["a_rows"] = (torch.randperm(rows, generator=g, device="cuda") % tokens).to(I32)
            else:
                s["a"] = _activations(rows, k, g)
            s["out"] = torch.empty(e, n, k, dtype=F32 if c["f32"] else BF16, device="cuda")
        else:
            s["w"] = torch.empty(e, n, k, dtype=BF16, device="cuda")
            for i in range(e):
                s["w"][i] = torch.randn(n, k, generator=g, device="cuda") * 0.02
            s["a"] = _activations(rows, k, g) if op == "gemm" else \
                torch.randn(rows, n, generator=g, device="cuda").mul_(0.02).to(BF16)
            # the caller's buffer: rows behind the last segment keep what they hold
            s["out"] = torch.full((rows, n if op == "gemm" else k), 3.0, dtype=BF16, device="cuda")
    elif op == "keep":
        x = _activations(c["rows"], c["width"], g)
        if c["width"] % 8:                       # rows on a 16-byte stride
            buf = torch.zeros(c["rows"], -(-c["width"] // 8) * 8, dtype=BF16, device="cuda")
            buf[:, :c["width"]] = x
            x = buf[:, :c["width"]]
        s["x"] = x
    elif op == "swiglu_bwd":
        q, s["scales"] = _keep_plain(torch.randn(c["rows"], c["width"], generator=g, device="cuda") * 2)
        s["codes"] = _codes_buffer(q)
        s["dh"] = torch.randn(c["rows"], c["width"] // 2, generator=g, device="cuda").mul_(0.05).to(BF16)
        s["gate"] = torch.rand(c["rows"], generator=g, device="cuda") if c["gated"] else None
    else:
        t, e, kr, n, k = c["tokens"], c["experts"], c["topk"], c["n"], c["k"]
        s["codes"], s["scales"], s["s_t"] = _nvfp4_weights(e, n, k, g)
        s["x"] = _activations(t * kr if c["form"] == "combine" else t, k, g)
        logits = torch.randn(t, e, generator=g, device="cuda")
        top = torch.topk(logits, kr, dim=1)
        s["idx"] = None if c["form"] == "dense" else top.indices.to(I32)
        s["gate"] = torch.softmax(top.values, 1)
    return s


# ------------------------------------------------------------------ plain form

def _grouped(s, rows):
    """Row numbers [E, longest] of each expert's segment, and which exist."""
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(max(1, s["longest"]), device=off.device)
    return at.clamp_max(rows - 1), at < off[1:, None]


def _plain_rows(s, transposed):
    a, w, off = s["a"], s["w"].to(F32), s["offsets"].long()
    at, _ = _grouped(s, a.shape[0])
    y = torch.bmm(a[at].to(F32), w if transposed else w.transpose(1, 2))
    r = torch.arange(a.shape[0], device=a.device)
    e = (torch.searchsorted(off, r, right=True) - 1).clamp(0, w.shape[0] - 1)
    p = (r - off[e]).clamp_max(y.shape[1] - 1)
    return torch.where((r < off[-1])[:, None], y[e, p].to(BF16), s["out"])


def _plain_wgrad(s):
    c = s["case"]
    at, there = _grouped(s, s["g"].shape[0])
    if c["kept"]:
        a = _kept_values(s["codes"], s["scales"], F32)[s["a_rows"].long()[at]]
    else:
        a = s["a"][at].to(F32)
    zero = torch.zeros((), device=a.device)
    a = torch.where(there[:, :, None], a, zero)
    g = torch.where(there[:, :, None], s["g"][at].to(F32), zero)
    return torch.bmm(g.transpose(1, 2), a).to(s["out"].dtype)


def _plain_keep(s):
    x = s["x"]
    q, scales = _keep_plain(x)
    if not s["case"]["swiglu"]:
        return {"values": q, "exponent": scales}
    i = x.shape[1] // 2
    a, b = x[:, :i].to(F32), x[:, i:].to(F32)
    return {"values": q, "exponent": scales, "h": (a * torch.sigmoid(a) * b).to(BF16)}


def _swiglu_bwd(a, b, dh, gate, out):
    sig = torch.sigmoid(a)
    h = a * sig * b
    d = dh * gate[:, None]
    da = d * b * sig * (1 + a * (1 - sig))
    db = d * a * sig
    return {"dy": torch.cat([da, db], 1).to(out), "gh": (h * gate[:, None]).to(out), "dgate": (dh * h).sum(1)}


def _plain_swiglu_bwd(s):
    v = _kept_values(s["codes"], s["scales"], F32)
    i = v.shape[1] // 2
    gate = torch.ones(v.shape[0], device=v.device) if s["gate"] is None else s["gate"]
    return _swiglu_bwd(v[:, :i], v[:, i:], s["dh"].to(F32), gate, BF16)


def _weight_values(codes, scales, n, k, dtype):
    """[P, N, K/2] codes and [P, ...] scale buffers -> e2m1 * sf, [P, N, K]."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=dtype, device=codes.device)
    grid = torch.cat([grid, -grid])
    v = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], -1).view(codes.shape[0], n, k // 16, 16)
    sf = scales[:, _scale_at(n, k, codes.device)].view(torch.float8_e4m3fn).to(dtype)
    return (v * sf[..., None]).view(codes.shape[0], n, k)


def _matvec(s, dtype):
    c = s["case"]
    t, kr, n, k, form = c["tokens"], c["topk"], c["n"], c["k"], c["form"]
    x = s["x"].to(dtype)
    if form == "dense":
        w = _weight_values(s["codes"], s["scales"], n, k, dtype)[0]
        return (x @ w.t()) * s["s_t"].to(dtype)
    idx = s["idx"].long().view(-1)
    w = _weight_values(s["codes"][idx], s["scales"][idx], n, k, dtype)
    rows = x if form == "combine" else x.repeat_interleave(kr, 0)
    y = torch.bmm(w, rows[:, :, None])[:, :, 0] * s["s_t"].to(dtype)[idx][:, None]
    if form == "combine":
        return (y.view(t, kr, n) * s["gate"].to(dtype)[:, :, None]).sum(1)
    if form == "swiglu":
        a, b = y[:, :n // 2], y[:, n // 2:]
        return a * torch.sigmoid(a) * b
    return y


def _plain_matvec(s):
    y = _matvec(s, F32)
    return y.to(BF16) if s["case"]["form"] == "swiglu" else y


# ------------------------------------------------------------------------ run

def _own_run(s, op, c):
    from quantization_nvfp4_quantize_b200 import api as lib
    if op in ("gemm", "dgrad"):
        return lib.ragged_gemm(s["a"], s["w"], s["offsets"], transpose=op == "dgrad", out=s["out"])
    if op == "wgrad":
        if c["kept"]:
            return lib.ragged_wgrad(s["g"], lib.Act8(s["codes"], s["scales"]), s["offsets"], a_rows=s["a_rows"],
                                    out=s["out"])
        return lib.ragged_wgrad(s["g"], s["a"], s["offsets"], out=s["out"])
    if op == "keep":
        if c["swiglu"]:
            h, q = lib.swiglu_act8(s["x"])
            return {"values": q.codes.view(torch.float8_e4m3fn), "exponent": q.scales, "h": h}
        q = lib.act8_quantize(s["x"])
        return {"values": q.codes.view(torch.float8_e4m3fn), "exponent": q.scales}
    if op == "swiglu_bwd":
        dy, gh, dgate = lib.swiglu_act8_backward(lib.Act8(s["codes"], s["scales"]), s["dh"], row_gate=s["gate"])
        return {"dy": dy, "gh": gh, "dgate": dgate}
    epilogue = {"store": lib.EPI_STORE_F32, "dense": lib.EPI_STORE_F32, "swiglu": lib.EPI_SWIGLU_BF16,
                "combine": lib.EPI_COMBINE_F32}[c["form"]]
    return lib.nvfp4_gemv(s["x"], s["codes"], s["scales"], s["s_t"], c["n"], c["k"], expert_idx=s["idx"],
                          epilogue=epilogue, gate=s["gate"] if c["form"] == "combine" else None)


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        return _own_run(state, op, c)
    if op in ("gemm", "dgrad"):
        return _plain_rows(state, op == "dgrad")
    if op == "wgrad":
        return _plain_wgrad(state)
    if op == "keep":
        return _plain_keep(state)
    if op == "swiglu_bwd":
        return _plain_swiglu_bwd(state)
    return _plain_matvec(state)


# ----------------------------------------------------------------------- work

def work(case):
    c, op = case, case["op"]
    if op in ("gemm", "dgrad", "wgrad"):
        e, m, n, k = c["experts"], c["rows"], c["n"], c["k"]
        used = min(e, m)                                     # experts with rows, at most
        flops = 2.0 * m * n * k
        if op == "wgrad":
            a = -(-m // c["fan"]) * k * (1 + 1 / GROUP) + 4.0 * m if c["kept"] else 2.0 * m * k
            return {"bytes": 2.0 * m * n + a + (4.0 if c["f32"] else 2.0) * e * n * k, "flops": flops}
        return {"bytes": 2.0 * m * (n + k) + 2.0 * used * n * k, "flops": flops}
    if op == "keep":
        m, k = c["rows"], c["width"]
        return {"bytes": m * k * (3.0 + 1 / GROUP) + (m * k if c["swiglu"] else 0.0),
                "flops": m * k * (4.0 if c["swiglu"] else 2.0)}
    if op == "swiglu_bwd":
        m, k = c["rows"], c["width"]
        return {"bytes": m * k * (1 + 1 / GROUP + 1.0 + 2.0 + 1.0) + 8.0 * m, "flops": 10.0 * m * k}
    t, e, kr, n, k = c["tokens"], c["experts"], c["topk"], c["n"], c["k"]
    used = e * (1 - (1 - kr / e) ** t) if e > 1 else 1       # distinct experts, expected
    rows_in = t * kr if c["form"] == "combine" else t
    out = {"store": 4.0 * t * kr * n, "dense": 4.0 * t * n, "swiglu": 1.0 * t * kr * n, "combine": 4.0 * t * n}[c["form"]]
    return {"bytes": used * n * k * 0.5625 + 2.0 * rows_in * k + out, "flops": 2.0 * t * kr * n * k}


# ---------------------------------------------------------------------- exact

def _e4m3(v):
    """Nearest E4M3 value (ties to even) of |v| <= 448, in 64 bits."""
    _, ex = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (ex - 1).clamp_min(-6) - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op in ("gemm", "dgrad", "wgrad"):
        off = s["offsets"].tolist()
        e = c["experts"]
        if op == "wgrad":
            out = torch.zeros(e, c["n"], c["k"], dtype=F64, device="cuda")
            for i in range(e):
                lo, hi = off[i], off[i + 1]
                if c["kept"]:
                    r = s["a_rows"][lo:hi].long()
                    a = _kept_values(s["codes"][r], s["scales"][r], F64)
                else:
                    a = s["a"][lo:hi].double()
                out[i] = s["g"][lo:hi].double().t() @ a
            return out
        out = s["out"].double()
        for i in range(e):
            w = s["w"][i].double()
            out[off[i]:off[i + 1]] = s["a"][off[i]:off[i + 1]].double() @ (w if op == "dgrad" else w.t())
        return out
    if op == "keep":
        x = s["x"].double()
        m, k = x.shape
        pad = -(-k // 128) * 128
        groups = torch.zeros(m, pad, dtype=F64, device="cuda")
        groups[:, :k] = x
        groups = groups.view(m, -1, GROUP)
        top = groups.abs().amax(2)
        p = torch.ceil(torch.log2(top.clamp_min(1e-300) / 448.0)).clamp_min(-120)
        p = p - ((top <= 448.0 * torch.exp2(p - 1)) & (p > -120)).double()      # log2 next to a power of two
        p = p + (top > 448.0 * torch.exp2(p)).double()
        p = torch.where(top == 0, torch.zeros_like(p), p)
        v = _e4m3(groups / torch.exp2(p)[:, :, None]).view(m, pad)[:, :k]
        r = {"values": v, "exponent": (p + 127).to(torch.uint8)}
        if c["swiglu"]:
            a, b = x[:, :k // 2], x[:, k // 2:]
            r["h"] = a / (1 + torch.exp(-a)) * b
        return r
    if op == "swiglu_bwd":
        v = _kept_values(s["codes"], s["scales"], F64)
        i = c["width"] // 2
        gate = torch.ones(c["rows"], device="cuda") if s["gate"] is None else s["gate"]
        return _swiglu_bwd(v[:, :i], v[:, i:], s["dh"].double(), gate.double(), F64)
    return _matvec(s, F64)
