"""The training pair (forward_train, backward) and the decode step of the
layers: the new operators run together, against the same chain in 64 bits with
the chain's own rounding points (bf16 rows, 8-bit kept values).  Bar: relative
Frobenius 2e-3, the framework's layer bar; an f32 sum that lands on the other
side of a bf16 rounding moves an element by 2^-8, and does so for about 1 in
10^3 of them (f32 error 2^-20 against the 2^-8 step), so such flips stay two
orders below the bar."""
import pytest
import torch

import oracle
from gpu_util import rel_fro
from ops_util import BF16, F64, keep
from quantization_nvfp4_quantize_b200.moe import DenseLayerW4A4, MoELayerW4A4, MoELayerW4A16

pytestmark = pytest.mark.gpu

TOL = 2e-3


def rnd(seed, *shape, scale=1.0, dtype=BF16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def layer(cls, T, E, H, I, kr, *args, seed=1):
    w13, w2 = rnd(seed, E, 2 * I, H, scale=0.05), rnd(seed + 1, E, H, I, scale=0.05)
    return cls(w13, w2, T, kr, *args), w13, w2


def bf(x):
    return x.to(BF16).double()


def reference(x, logits, wq13, wq2, dy, kr, exact_gates):
    """Dense per-slot chain in 64 bits (no routed layout): every (token, slot)
    row is its own product."""
    T, I = x.shape[0], wq2.shape[2]
    top = torch.topk(logits, kr, dim=1)
    idx, g = top.indices, exact_gates.double()
    w13, w2 = wq13.double()[idx], wq2.double()[idx]                       # [T, kr, 2I, H], [T, kr, H, I]
    xd, dyd = x.double(), dy.double()
    y13 = bf(torch.einsum("tjnh,th->tjn", w13, xd))
    a, b = y13[..., :I], y13[..., I:]
    h = bf(a * torch.sigmoid(a) * b)
    rows = bf(torch.einsum("tjhi,tji->tjh", w2, h))
    y = (rows * g[..., None]).sum(1)
    # backward
    k = keep(y13.reshape(T * kr, -1).to(BF16))[0].view(T, kr, -1)
    a, b = k[..., :I], k[..., I:]
    s = torch.sigmoid(a)
    hk = a * s * b
    u = bf(torch.einsum("tjhi,th->tji", w2, dyd))
    dg = (u * hk).sum(-1)
    gu = g[..., None] * u
    d13 = bf(torch.cat([gu * b * s * (1 + a * (1 - s)), gu * a * s], -1))
    gh = bf(g[..., None] * hk)
    xk = keep(x)[0]
    E = wq13.shape[0]
    dw13 = torch.zeros(wq13.shape, dtype=F64, device=x.device)
    dw2 = torch.zeros(wq2.shape, dtype=F64, device=x.device)
    for e in range(E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        dw13[e] = d13[t, j].t() @ xk[t]
        dw2[e] = dyd[t].t() @ gh[t, j]
    dx = bf(torch.einsum("tjnh,tjn->tjh", w13, d13)).sum(1)
    dl = torch.zeros(logits.shape, dtype=F64, device=x.device)
    dl.scatter_(1, idx, g * (dg - (g * dg).sum(1, keepdim=True)))
    return y, dx, dl, dw13, dw2


@pytest.mark.parametrize("T,E,H,I,kr", [(1, 4, 64, 64, 2), (37, 3, 128, 192, 1), (130, 8, 256, 128, 3),
                                        (300, 16, 512, 256, 8)])
def test_training_step(cuda, T, E, H, I, kr):
    lay, w13, w2 = layer(MoELayerW4A16, T, E, H, I, kr)
    x, logits, dy = rnd(3, T, H), rnd(4, T, E, dtype=torch.float32), rnd(5, T, H, scale=0.1)
    y = lay.forward_train(x, logits)
    g = lay.backward(dy)
    want = reference(x, logits, lay.wq13, lay.wq2, dy, kr, lay.train_routing.topk_gate)
    for name, a, b in zip(("y", "dx", "dlogits", "dw13", "dw2"), (y, g.dx, g.dlogits, g.dw13, g.dw2), want):
        if kr == 1 and name == "dlogits":
            assert float(a.abs().max()) <= 1e-6 * float(g.dx.abs().max() + 1)      # one slot: the gate is constant
            continue
        assert rel_fro(a.double().cpu().numpy(), b.cpu().numpy()) <= TOL, name
    if I % 128 == 0 and H % 256 == 0:      # the inference forward (padded segments) computes the same Y
        assert rel_fro(y.cpu().numpy(), lay.forward(x, logits).double().cpu().numpy()) <= 2 * 2.0 ** -8
    # again: the same bits; then accumulated
    y2 = lay.forward_train(x, logits)
    g2 = lay.backward(dy, dw13=g.dw13.clone(), dw2=g.dw2.clone(), accumulate=True)
    assert torch.equal(y, y2) and torch.equal(g.dx, g2.dx) and torch.equal(g.dlogits, g2.dlogits)
    assert torch.equal(g2.dw13, 2 * g.dw13) and torch.equal(g2.dw2, 2 * g.dw2)


def test_backward_again_and_after_other_calls(cuda):
    """backward reads only what forward_train kept: a second one, and one after
    an inference forward of the same layer, give the same bits."""
    T, E, H, I, kr = 96, 4, 256, 128, 2
    lay, _, _ = layer(MoELayerW4A16, T, E, H, I, kr)
    x, logits, dy = rnd(20, T, H), rnd(21, T, E, dtype=torch.float32), rnd(22, T, H)
    lay.forward_train(x, logits)
    a = lay.backward(dy)
    lay.forward(rnd(23, T, H), rnd(24, T, E, dtype=torch.float32))
    b = lay.backward(dy)
    for n in ("dx", "dlogits", "dw13", "dw2"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n


def test_training_step_captured(cuda):
    T, E, H, I, kr = 64, 8, 128, 64, 2
    lay, w13, w2 = layer(MoELayerW4A16, T, E, H, I, kr)
    x, logits, dy = rnd(6, T, H), rnd(7, T, E, dtype=torch.float32), rnd(8, T, H)
    lay.forward_train(x, logits)
    lay.backward(dy)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lay.forward_train(x, logits)
        g = lay.backward(dy)
    x.copy_(rnd(9, T, H))
    logits.copy_(rnd(10, T, E, dtype=torch.float32))
    dy.copy_(rnd(11, T, H))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, g.dx, g.dlogits, g.dw13, g.dw2)]
    y = lay.forward_train(x, logits)
    g = lay.backward(dy)
    for a, b in zip(got, (y, g.dx, g.dlogits, g.dw13, g.dw2)):
        assert torch.equal(a, b)


def test_training_step_refusals(cuda):
    lay, _, _ = layer(MoELayerW4A16, 8, 4, 64, 64, 2)
    with pytest.raises(RuntimeError, match="no forward_train"):
        lay.backward(rnd(1, 8, 64))
    with pytest.raises(ValueError, match="forward_train"):
        lay.forward_train(rnd(1, 9, 64), rnd(2, 9, 4, dtype=torch.float32))
    lay.forward_train(rnd(1, 8, 64), rnd(2, 8, 4, dtype=torch.float32))
    with pytest.raises(ValueError, match="dy"):
        lay.backward(rnd(1, 8, 64).float())
    with pytest.raises(ValueError, match="accumulate"):
        lay.backward(rnd(1, 8, 64), accumulate=True)


def values(codes, scales, s_t, N, K):
    """NVFP4 weights in 64 bits: e2m1 * sf * s_t, [E, N, K]."""
    E = s_t.numel()
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=F64, device=codes.device)
    c = codes.view(E, N, K // 2)
    v = torch.stack([grid[(c & 15).int()], grid[(c >> 4).int()]], -1).view(E, N, K)
    sf = torch.stack([torch.from_numpy(oracle.unswizzle_scales(b, N, K).copy())
                      for b in scales.view(E, -1).cpu().numpy()]).to(codes.device)
    return v * sf.view(torch.float8_e4m3fn).double().repeat_interleave(16, 2) * s_t.double()[:, None, None]


@pytest.mark.parametrize("t", [0, 1, 3, 16])
@pytest.mark.parametrize("E,H,I,kr", [(8, 256, 256, 2), (32, 1024, 256, 8)])
def test_decode_step(cuda, t, E, H, I, kr):
    """Against the dense per-slot chain on the NVFP4 weights' values (one
    rounding of h to bf16)."""
    lay, w13, w2 = layer(MoELayerW4A4, 64, E, H, I, kr, 0)
    x, logits = rnd(12, t, H), rnd(13, t, E, dtype=torch.float32)
    y = lay.decode(x, logits)
    assert tuple(y.shape) == (t, H)
    if t == 0:
        return
    idx = torch.topk(logits, kr, dim=1)
    g = torch.softmax(idx.values.double(), 1)
    v13, v2 = values(lay.c13, lay.sf13, lay.s13, 2 * I, H), values(lay.c2, lay.sf2, lay.s2, H, I)
    a13 = torch.einsum("tjnh,th->tjn", v13[idx.indices], x.double())
    a, b = a13[..., :I], a13[..., I:]
    h = bf(a * torch.sigmoid(a) * b)
    want = (torch.einsum("tjhi,tji->tjh", v2[idx.indices], h) * g[..., None]).sum(1)
    assert rel_fro(y.double().cpu().numpy(), want.cpu().numpy()) <= TOL


def test_decode_captured_and_two_batches_in_flight(cuda):
    """Graph replays with new inputs, and two batches on two streams."""
    E, H, I, kr = 16, 512, 256, 4
    lay, _, _ = layer(MoELayerW4A4, 64, E, H, I, kr, 0)
    x, logits = rnd(30, 5, H), rnd(31, 5, E, dtype=torch.float32)
    lay.decode(x, logits)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lay.decode(x, logits)
    x.copy_(rnd(32, 5, H))
    logits.copy_(rnd(33, 5, E, dtype=torch.float32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, lay.decode(x, logits))
    xs = [rnd(34 + i, 40, H) for i in range(2)]
    ls = [rnd(36 + i, 40, E, dtype=torch.float32) for i in range(2)]
    want = [lay.decode(a, b) for a, b in zip(xs, ls)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(lay.decode(xs[i], ls[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert torch.equal(g, want[i])


def test_dense_decode(cuda):
    lay = DenseLayerW4A4(rnd(14, 256, 256, scale=0.05), 16, 0)
    x = rnd(15, 5, 256)
    y = lay.decode(x)
    wd = values(lay.c_w, lay.sf_w, lay.s_w, 256, 256)[0]
    assert rel_fro(y.cpu().numpy(), (x.double() @ wd.t()).cpu().numpy()) <= 1e-5


def test_training_step_of_no_tokens(cuda):
    lay, _, _ = layer(MoELayerW4A16, 0, 4, 64, 64, 2)
    y = lay.forward_train(rnd(1, 0, 64), rnd(2, 0, 4, dtype=torch.float32))
    g = lay.backward(rnd(3, 0, 64))
    assert y.shape == g.dx.shape == (0, 64) and g.dlogits.shape == (0, 4)
    assert not bool(g.dw13.any()) and not bool(g.dw2.any())


def test_training_step_strided_and_two_layers_in_flight(cuda):
    """x and dy on a longer row stride give the same bits; so do two layers
    whose steps run on two streams at once."""
    T, E, H, I, kr = 200, 8, 256, 128, 2
    lays = [layer(MoELayerW4A16, T, E, H, I, kr, seed=s)[0] for s in (40, 50)]
    xs, ls, dys = ([rnd(s + i, T, n, dtype=d) for i in range(2)] for s, n, d in
                   ((60, H, BF16), (62, E, torch.float32), (64, H, BF16)))

    def step(i, x, dy):
        y = lays[i].forward_train(x, ls[i])
        g = lays[i].backward(dy)
        return y, g.dx, g.dlogits, g.dw13, g.dw2

    want = [step(i, xs[i], dys[i]) for i in range(2)]
    wide = [torch.full((T, H + 24), float("nan"), dtype=BF16, device=cuda) for _ in range(2)]
    for w, t in zip(wide, (xs[0], dys[0])):
        w[:, 8:8 + H] = t
    for a, b in zip(step(0, wide[0][:, 8:8 + H], wide[1][:, 8:8 + H]), want[0]):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(i, xs[i], dys[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for a, b in zip(r, want[i]):
                assert torch.equal(a, b)


def test_nothing_kept_after_a_failed_forward_or_new_weights(cuda, monkeypatch):
    """backward never mixes a forward's routing with another's rows or weights."""
    lay, w13, w2 = layer(MoELayerW4A16, 8, 4, 64, 64, 2)
    x, logits, dy = rnd(1, 8, 64), rnd(2, 8, 4, dtype=torch.float32), rnd(3, 8, 64)
    lay.forward_train(x, logits)
    want = lay.backward(dy)
    with pytest.raises(ValueError, match="x must be bf16"):
        lay.forward_train(x.float(), logits)
    assert torch.equal(lay.backward(dy).dx, want.dx)

    def fail(*args, **kw):
        raise MemoryError

    from quantization_nvfp4_quantize_b200 import api
    with monkeypatch.context() as m:
        m.setattr(api, "combine_rows", fail)
        with pytest.raises(MemoryError):
            lay.forward_train(rnd(4, 8, 64), logits)
    with pytest.raises(RuntimeError, match="no forward_train"):
        lay.backward(dy)
    lay.forward_train(x, logits)
    assert torch.equal(lay.backward(dy).dx, want.dx)
    lay.set_weights(w13, w2)
    with pytest.raises(RuntimeError, match="no forward_train"):
        lay.backward(dy)


def test_forward_train_after_one_without_memory(cuda, monkeypatch):
    """A first call whose buffers do not fit can be made again."""
    from quantization_nvfp4_quantize_b200 import api
    lay, _, _ = layer(MoELayerW4A16, 8, 4, 64, 64, 2)
    x, logits = rnd(1, 8, 64), rnd(2, 8, 4, dtype=torch.float32)
    real, calls = api.Act8.empty, []

    def second_fails(*a):
        calls.append(a)
        if len(calls) == 2:
            raise torch.OutOfMemoryError("no memory")
        return real(*a)

    with monkeypatch.context() as m:
        m.setattr(api.Act8, "empty", staticmethod(second_fails))
        with pytest.raises(torch.OutOfMemoryError):
            lay.forward_train(x, logits)
    y = lay.forward_train(x, logits)
    assert torch.equal(y, layer(MoELayerW4A16, 8, 4, 64, 64, 2)[0].forward_train(x, logits))
    lay.backward(rnd(3, 8, 64))


def test_backward_follows_a_replayed_forward(cuda):
    """Routing and kept rows change together: backward after the replay of a
    captured forward_train gives that forward's gradients, whatever was called
    in between, and so does a captured backward after an eager forward."""
    T, E, H, I, kr = 64, 8, 128, 64, 2
    lay, _, _ = layer(MoELayerW4A16, T, E, H, I, kr)
    data = [(rnd(60 + i, T, H), rnd(70 + i, T, E, dtype=torch.float32)) for i in range(2)]
    dy = rnd(80, T, H)
    want = []
    for x, logits in data:
        lay.forward_train(x, logits)
        want.append(lay.backward(dy))
    fwd, bwd = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(fwd):
        lay.forward_train(*data[0])
    with torch.cuda.graph(bwd):
        g = lay.backward(dy)

    def same(a, b):
        return all(torch.equal(getattr(a, n), getattr(b, n)) for n in ("dx", "dlogits", "dw13", "dw2"))

    lay.forward_train(*data[1])
    fwd.replay()
    assert same(lay.backward(dy), want[0])
    bwd.replay()
    assert same(g, want[0])
    lay.forward_train(*data[1])
    bwd.replay()
    assert same(g, want[1]) and same(lay.backward(dy), want[1])


def test_status_of_a_step(cuda):
    """A clean step leaves the word at 0; one that a wait marked is reported."""
    from quantization_nvfp4_quantize_b200._lib import Nvfp4Error
    lay, _, _ = layer(MoELayerW4A16, 8, 4, 64, 64, 2)
    x, logits, dy = rnd(1, 8, 64), rnd(2, 8, 4, dtype=torch.float32), rnd(3, 8, 64)
    lay.forward_train(x, logits)
    g = lay.backward(dy)
    lay.check_status()
    assert int(g.status) == 0
    lay.status.fill_(5)
    with pytest.raises(Nvfp4Error, match="TIMEOUT"):
        lay.check_status()
    lay.check_status()
    with pytest.raises(RuntimeError, match="no forward_train"):
        lay.backward(dy)
    lay.forward_train(x, logits)
    assert torch.equal(lay.backward(dy).dx, g.dx)
    lay.check_status()


def test_reused_buffers_are_never_read_stale(cuda):
    """Steps back to back through the same buffers with new data each time:
    every step's results are those of the step alone."""
    T, E, H, I, kr = 48, 8, 128, 64, 2
    lay, _, _ = layer(MoELayerW4A16, T, E, H, I, kr)
    dec, _, _ = layer(MoELayerW4A4, 64, E, 256, 256, kr, 0)
    steps = [(rnd(100 + i, T, H), rnd(200 + i, T, E, dtype=torch.float32), rnd(300 + i, T, H), rnd(400 + i, 6, 256),
              rnd(500 + i, 6, E, dtype=torch.float32)) for i in range(12)]

    def run(x, logits, dy, xd, ld):
        y = lay.forward_train(x, logits)
        g = lay.backward(dy)
        return y, g.dx, g.dlogits, g.dw13, g.dw2, dec.decode(xd, ld)

    want = []
    for s in steps:
        want.append(run(*s))
        torch.cuda.synchronize()
    for _ in range(5):
        got = [run(*s) for s in steps]
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
