"""Refusals of the experts' training and decode operators: argument errors are
returned before anything is enqueued (no GPU needed)."""
import ctypes

import pytest
import torch

from quantization_nvfp4_quantize_b200 import _lib, api

FAKE = ctypes.c_void_p(0x10000)           # never dereferenced: rejected before any launch
ODD = ctypes.c_void_p(0x10008)
INVALID, ALIGN, SHAPE, WORKSPACE = 1, 2, 3, 6


def calls(name, good, bad):
    """Each (index, value, status) of `bad` put into the good arguments alone."""
    fn = getattr(_lib.load(), name)
    for at, value, status in bad:
        args = list(good)
        args[at] = value
        assert fn(*args) == status, (name, at, value)


def test_ragged_gemm():
    #       a     lda  M    w     N    K   E  off  tr  out   ld  f32 stat  stream
    good = [FAKE, 64, 100, FAKE, 128, 64, 4, FAKE, 0, FAKE, 128, 0, None, None]
    calls("moe_ragged_gemm", good, [
        (9, ctypes.c_void_p(0x10001), ALIGN),
        (0, None, INVALID), (3, None, INVALID), (7, None, INVALID), (9, None, INVALID), (2, -1, INVALID),
        (4, -1, INVALID), (6, 0, SHAPE), (6, 257, SHAPE), (2, 1 << 31, SHAPE), (4, 1 << 24, SHAPE), (5, 60, ALIGN),
        (1, 56, ALIGN), (1, 68, ALIGN), (10, 127, ALIGN), (0, ODD, ALIGN), (3, ODD, ALIGN), (5, 0, SHAPE)])
    lib = _lib.load()
    back = [FAKE, 128, 100, FAKE, 128, 64, 4, FAKE, 1, FAKE, 64, 0, None, None]
    calls("moe_ragged_gemm", back, [(1, 120, ALIGN), (10, 63, ALIGN), (4, 0, SHAPE)])
    # nothing to do: no error, no launch
    good[2] = 0
    assert lib.moe_ragged_gemm(*good) == 0
    back[5] = 0
    back[2] = 100
    assert lib.moe_ragged_gemm(*back) == 0


def test_ragged_wait_expiry_arguments():
    #       a     lda  M    w     N    K   off   out   ld   stat  limit    stream
    good = [FAKE, 64, 100, FAKE, 128, 64, FAKE, FAKE, 128, FAKE, 2000000, None]
    calls("nvfp4_debug_ragged_wait_expiry", good, [
        (9, None, INVALID), (10, 999999, INVALID), (10, 1000000001, INVALID), (2, 257, SHAPE), (4, 257, SHAPE),
        (2, 0, SHAPE), (0, None, INVALID)])


def test_ragged_wgrad():
    #       g     ldg  M    a     lda asc   lds rows  T   N    K   E  off   out   f32 acc ws  n  stat  stream
    good = [FAKE, 256, 5000, FAKE, 256, None, 0, None, 0, 256, 256, 128, FAKE, FAKE, 1, 0, None, 0, None, None]
    calls("moe_ragged_wgrad", good, [
        (13, ctypes.c_void_p(0x10002), ALIGN),
        (0, None, INVALID), (3, None, INVALID), (12, None, INVALID), (13, None, INVALID), (2, -1, INVALID),
        (8, -1, INVALID), (11, 0, SHAPE), (11, 257, SHAPE), (2, 1 << 31, SHAPE), (1, 255, ALIGN), (1, 248, ALIGN),
        (4, 248, ALIGN), (4, 260, ALIGN), (0, ODD, ALIGN), (3, ODD, ALIGN), (7, FAKE, INVALID)])
    kept = list(good)
    kept[5], kept[6], kept[8] = FAKE, 8, 5000
    kept[16], kept[17] = FAKE, 1000
    calls("moe_ragged_wgrad", kept, [(6, 4, ALIGN), (6, 9, ALIGN), (4, 264, ALIGN), (8, 4999, INVALID),
                                     (5, ODD, ALIGN), (16, None, WORKSPACE)])
    assert _lib.load().moe_ragged_wgrad_workspace_size(5000, 256, 256, 128, 1) == 5000 * 256 * 2
    # few output tiles: a workspace is required
    lib = _lib.load()
    few = list(good)
    few[11] = 1
    need = lib.moe_ragged_wgrad_workspace_size(5000, 256, 256, 1, 0)
    assert need > 0
    assert lib.moe_ragged_wgrad(*few) == WORKSPACE
    few[16], few[17] = FAKE, need - 1
    assert lib.moe_ragged_wgrad(*few) == WORKSPACE
    assert lib.moe_ragged_wgrad_workspace_size(5000, 4096, 4096, 1, 0) == 0
    assert lib.moe_ragged_wgrad_workspace_size(-1, 64, 64, 1, 0) == 0
    # empty results and empty sums into an accumulator
    none = list(good)
    none[9] = 0
    assert lib.moe_ragged_wgrad(*none) == 0
    none = list(good)
    none[2], none[15] = 0, 1
    assert lib.moe_ragged_wgrad(*none) == 0


def test_act8():
    good = [FAKE, 10, 100, 104, FAKE, 112, FAKE, 4, None]
    calls("act8_quantize", good, [
        (0, None, INVALID), (4, None, INVALID), (6, None, INVALID), (1, -1, INVALID), (2, 1 << 24, SHAPE),
        (3, 96, ALIGN), (3, 101, ALIGN), (5, 96, ALIGN), (5, 104, ALIGN), (7, 3, ALIGN), (7, 6, ALIGN),
        (0, ODD, ALIGN), (4, ODD, ALIGN), (6, ODD, ALIGN)])
    good = [FAKE, 112, FAKE, 4, 10, 100, FAKE, 104, None]
    calls("act8_dequantize", good, [
        (0, None, INVALID), (2, None, INVALID), (6, None, INVALID), (4, -1, INVALID), (1, 96, ALIGN), (3, 3, ALIGN),
        (7, 100, ALIGN), (0, ODD, ALIGN), (6, ODD, ALIGN)])
    good = [FAKE, 10, 96, 192, FAKE, 96, FAKE, 192, FAKE, 8, None]
    calls("moe_swiglu_act8", good, [
        (0, None, INVALID), (4, None, INVALID), (6, None, INVALID), (8, None, INVALID), (2, 80, SHAPE), (1, -1, INVALID),
        (3, 184, ALIGN), (5, 88, ALIGN), (7, 176, ALIGN), (7, 200, ALIGN), (9, 4, ALIGN), (9, 10, ALIGN),
        (0, ODD, ALIGN)])
    good = [FAKE, 192, FAKE, 6, FAKE, 96, None, 10, 96, FAKE, 192, None, 0, None, None]
    calls("moe_swiglu_act8_backward", good, [
        (0, None, INVALID), (2, None, INVALID), (4, None, INVALID), (9, None, INVALID), (8, 48, SHAPE), (1, 176, ALIGN),
        (3, 5, ALIGN), (5, 95, ALIGN), (10, 184, ALIGN), (9, ODD, ALIGN), (11, FAKE, ALIGN)])
    lib = _lib.load()
    assert lib.act8_quantize(None, 0, 64, 64, None, 64, None, 4, None) == 0
    assert lib.moe_swiglu_act8(None, 0, 32, 64, None, 32, None, 64, None, 4, None) == 0


def test_combine_and_route_backward():
    good = [FAKE, 10, 64, 64, FAKE, None, 5, 2, FAKE, 64, None]
    calls("moe_combine_rows", good, [
        (0, None, INVALID), (4, None, INVALID), (8, None, INVALID), (7, 0, INVALID), (7, 33, INVALID), (2, 60, ALIGN),
        (3, 56, ALIGN), (9, 60, ALIGN), (9, 66, ALIGN), (0, ODD, ALIGN), (6, -1, INVALID)])
    good = [FAKE, FAKE, FAKE, FAKE, 10, 5, 8, 2, FAKE, None]
    calls("moe_route_backward", good, [
        (0, None, INVALID), (1, None, INVALID), (2, None, INVALID), (3, None, INVALID), (8, None, INVALID),
        (6, 0, SHAPE), (7, 0, SHAPE), (7, 33, SHAPE), (5, -1, INVALID)])


def test_gemv():
    #       x     T  ldx   codes sc    s_t   N    K    E  idx  kr epi gate  out   ld  ws    n  stream
    good = [FAKE, 2, 128, FAKE, FAKE, FAKE, 256, 128, 8, FAKE, 2, 0, None, FAKE, 256, None, 0, None]
    calls("moe_nvfp4_gemv", good, [
        (13, ctypes.c_void_p(0x10002), ALIGN),
        (0, None, INVALID), (3, None, INVALID), (4, None, INVALID), (5, None, INVALID), (13, None, INVALID),
        (9, None, INVALID), (11, 2, INVALID), (11, 4, INVALID), (1, -1, INVALID), (7, 96, SHAPE), (7, 0, SHAPE),
        (6, 0, SHAPE), (8, 0, SHAPE), (10, 0, SHAPE), (10, 33, SHAPE), (2, 120, ALIGN), (2, 132, ALIGN),
        (14, 255, ALIGN), (0, ODD, ALIGN), (3, ODD, ALIGN), (4, ODD, ALIGN)])
    many = list(good)
    many[1], many[11] = 16, api.EPI_COMBINE_F32            # tokens share experts: a workspace is required
    need = _lib.load().moe_nvfp4_gemv_workspace_size(16, 256, 8, 2, api.EPI_COMBINE_F32)
    assert need == 16 * 2 * 256 * 4 and _lib.load().moe_nvfp4_gemv_workspace_size(1, 256, 8, 2, 3) == 0
    calls("moe_nvfp4_gemv", many, [(15, None, WORKSPACE), (15, ODD, WORKSPACE)])
    many[15], many[16] = FAKE, need - 1
    assert _lib.load().moe_nvfp4_gemv(*many) == WORKSPACE
    odd = list(good)
    odd[6], odd[11] = 257, 1
    assert _lib.load().moe_nvfp4_gemv(*odd) == SHAPE
    good[1] = 0
    assert _lib.load().moe_nvfp4_gemv(*good) == 0


def test_route_accepts_unpadded_segments():
    lib = _lib.load()
    # rejected for its workspace only: seg_align 1 and T * k_r rows are accepted
    assert lib.moe_route(FAKE, 16, 8, 2, FAKE, FAKE, 1, FAKE, FAKE, FAKE, FAKE, 32, None, 0, None) == WORKSPACE
    assert lib.moe_route(FAKE, 16, 8, 2, FAKE, FAKE, 1, FAKE, FAKE, FAKE, FAKE, 31, FAKE, 4096, None) == INVALID
    assert lib.moe_route(FAKE, 16, 8, 2, FAKE, FAKE, 2, FAKE, FAKE, FAKE, FAKE, 64, FAKE, 4096, None) == INVALID


def good_calls():
    """Well-formed operands on the host: refused for their device alone."""
    bf, f32, i32, u8 = (lambda *n: torch.zeros(*n, dtype=torch.bfloat16)), torch.zeros, \
        (lambda *n: torch.zeros(*n, dtype=torch.int32)), (lambda *n: torch.zeros(*n, dtype=torch.uint8))
    a8 = lambda m, k: api.Act8(u8(m, k), u8(m, -(-k // 128) * 4))
    return {
        "ragged_gemm": lambda **k: api.ragged_gemm(**{**dict(a=bf(4, 64), w=bf(2, 16, 64), offsets=i32(3)), **k}),
        "ragged_wgrad": lambda **k: api.ragged_wgrad(**{**dict(g=bf(4, 16), a=bf(4, 64), offsets=i32(3)), **k}),
        "ragged_wgrad kept": lambda **k: api.ragged_wgrad(**{**dict(g=bf(4, 16), a=a8(4, 64), offsets=i32(3)), **k}),
        "act8_quantize": lambda **k: api.act8_quantize(**{**dict(x=bf(4, 64)), **k}),
        "act8_dequantize": lambda **k: api.act8_dequantize(**{**dict(a=a8(4, 64)), **k}),
        "swiglu_act8": lambda **k: api.swiglu_act8(**{**dict(y=bf(4, 64)), **k}),
        "swiglu_act8_backward": lambda **k: api.swiglu_act8_backward(**{**dict(y=a8(4, 64), dh=bf(4, 32)), **k}),
        "combine_rows": lambda **k: api.combine_rows(**{**dict(rows=bf(4, 64), dst_row=i32(2, 2)), **k}),
        "route_backward": lambda **k: api.route_backward(**{**dict(topk_idx=i32(2, 2), topk_gate=f32(2, 2),
                                                                   dst_row=i32(2, 2), dgate_row=f32(4), E=8), **k}),
        "nvfp4_gemv": lambda **k: api.nvfp4_gemv(**{**dict(x=bf(2, 64), codes=u8(3, 32, 32), scales=u8(3, 512), s_t=f32(3),
                                                           N=32, K=64, expert_idx=i32(2, 2)), **k}),
    }


def test_binding_refuses_host_tensors():
    for name, call in good_calls().items():
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()


def test_binding_refuses_operands():
    bf, u8, i32 = (lambda *n: torch.zeros(*n, dtype=torch.bfloat16)), (lambda *n: torch.zeros(*n, dtype=torch.uint8)), \
        (lambda *n: torch.zeros(*n, dtype=torch.int32))
    a8 = api.Act8
    meta = torch.zeros(4, 64, dtype=torch.bfloat16, device="meta")
    bad = [
        ("ragged_gemm", dict(a=torch.zeros(4, 64)), "a: need BFloat16"),
        ("ragged_gemm", dict(a=bf(4, 56)), "a: need"),
        ("ragged_gemm", dict(a=bf(64, 4).t()), "columns must be contiguous"),
        ("ragged_gemm", dict(w=bf(16, 64)), "w must be"),
        ("ragged_gemm", dict(w=bf(2, 64, 16).transpose(1, 2)), "w must be"),
        ("ragged_gemm", dict(offsets=i32(4)), "3 elements"),
        ("ragged_gemm", dict(offsets=torch.zeros(3, dtype=torch.int64)), "offsets: need"),
        ("ragged_gemm", dict(out=bf(4, 17)), "out: need"),
        ("ragged_gemm", dict(out_dtype=torch.float16), "out_dtype"),
        ("ragged_gemm", dict(transpose=True), "a: need"),
        ("ragged_gemm", dict(a=meta), "expected meta"),
        ("ragged_gemm", dict(a=None), "need a tensor"),
        ("ragged_wgrad", dict(a=bf(5, 64)), "a: need"),
        ("ragged_wgrad", dict(g=bf(4)), "must be"),
        ("ragged_wgrad", dict(out=torch.zeros(2, 64, 16)), "out must be"),
        ("ragged_wgrad", dict(accumulate=True), "accumulate needs out"),
        ("ragged_wgrad kept", dict(a=a8(u8(5, 64), u8(5, 4))), "a.codes: need"),
        ("ragged_wgrad kept", dict(a=a8(u8(4, 64), u8(4, 3))), "a.scales: need"),
        ("ragged_wgrad kept", dict(a=a8(u8(4, 64), u8(3, 4))), "a.scales: need"),
        ("ragged_wgrad kept", dict(a_rows=i32(5)), "a_rows: need"),
        ("act8_quantize", dict(x=bf(4)), "must be"),
        ("act8_quantize", dict(x=torch.zeros(4, 64)), "x: need"),
        ("act8_quantize", dict(out=a8(u8(4, 63), u8(4, 4))), "out.codes: need"),
        ("act8_dequantize", dict(out=bf(4, 63)), "out: need"),
        ("swiglu_act8", dict(y=bf(4, 63)), "must be"),
        ("swiglu_act8", dict(h=bf(4, 33), out=a8(u8(4, 64), u8(4, 4))), "h: need"),
        ("swiglu_act8_backward", dict(dh=bf(4, 31)), "y.codes: need"),
        ("swiglu_act8_backward", dict(row_gate=torch.zeros(5)), "row_gate: need"),
        ("combine_rows", dict(dst_row=i32(4)), "must be"),
        ("combine_rows", dict(gate=torch.zeros(3)), "gate: need"),
        ("route_backward", dict(dst_row=i32(3, 2)), "dst_row: need"),
        ("route_backward", dict(E=0), "1 <= E"),
        ("route_backward", dict(out=torch.zeros(2, 7)), "out must be"),
        ("nvfp4_gemv", dict(x=bf(3, 64)), "rows for 2 tokens"),
        ("nvfp4_gemv", dict(codes=u8(3, 32, 31)), "codes must be"),
        ("nvfp4_gemv", dict(scales=u8(3, 511)), "scales must be"),
        ("nvfp4_gemv", dict(gate=torch.zeros(2, 2)), "EPI_COMBINE"),
        ("nvfp4_gemv", dict(expert_idx=i32(4)), "expert_idx must be"),
        ("nvfp4_gemv", dict(N=0), "must be positive"),
    ]
    calls = good_calls()
    for name, change, match in bad:
        with pytest.raises(ValueError, match=match):
            calls[name](**change)
    with pytest.raises(TypeError):
        _lib.binding().combine_rows(None)


def test_missing_binding_fails_loudly(monkeypatch):
    import sys
    monkeypatch.setattr(_lib, "_bound", None)
    monkeypatch.setitem(sys.modules, "quantization_nvfp4_quantize_b200._binding", None)
    import quantization_nvfp4_quantize_b200 as pkg
    monkeypatch.delattr(pkg, "_binding", raising=False)
    with pytest.raises(RuntimeError, match="not built"):
        _lib.binding()


def test_binding_refuses_lengths_and_flags():
    """Scale buffers with room between the experts, empty offset tables, flags
    without a truth value."""
    calls = good_calls()
    u8, i32 = (lambda *n: torch.zeros(*n, dtype=torch.uint8)), (lambda *n: torch.zeros(*n, dtype=torch.int32))
    with pytest.raises(ValueError, match="scales must be"):
        calls["nvfp4_gemv"](scales=u8(3, 512 + 16))
    for n in (0, 1):
        with pytest.raises(ValueError, match="offsets: need"):
            calls["ragged_wgrad"](offsets=i32(n))
    with pytest.raises(RuntimeError, match="ambiguous"):
        calls["ragged_gemm"](transpose=torch.ones(2))
    with pytest.raises(RuntimeError, match="ambiguous"):
        calls["ragged_wgrad"](accumulate=torch.ones(2))


def test_layers_refuse_tensors_elsewhere():
    """The layers' calls pass bare pointers on: a tensor that is not where the
    weights are is refused before any of them."""
    from quantization_nvfp4_quantize_b200.moe import MoELayerW4A4, MoELayerW4A16
    x, logits = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 4)
    t = MoELayerW4A16.__new__(MoELayerW4A16)
    t.T, t.H, t.E, t.k_r, t.I, t.train_routing = 2, 64, 4, 2, 32, object()
    t.wq13 = torch.empty(4, 64, 64, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="forward_train: x is on cpu"):
        t.forward_train(x, logits)
    with pytest.raises(ValueError, match="forward_train: logits is on cpu"):
        t.forward_train(x.to("meta"), logits)
    with pytest.raises(ValueError, match="backward: dy is on cpu"):
        t.backward(x)
    d = MoELayerW4A4.__new__(MoELayerW4A4)
    d.H, d.E, d.c13 = 64, 4, torch.empty(4, 64, 32, dtype=torch.uint8, device="meta")
    with pytest.raises(ValueError, match="decode: x is on cpu"):
        d.decode(x, logits)
    d.c13 = torch.empty(4, 64, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="decode: need x"):
        d.decode(x[:, :32], logits)
    with pytest.raises(ValueError, match="decode: need x"):
        d.decode(x, logits[:1])


def test_route_of_no_tokens_without_padding_needs_no_rows():
    lib = _lib.load()
    # rejected for its workspace only
    assert lib.moe_route(None, 0, 8, 2, None, None, 1, FAKE, None, None, None, 0, None, 0, None) == WORKSPACE
    assert lib.moe_route(None, 0, 8, 2, None, None, 1, None, None, None, None, 0, FAKE, 4096, None) == INVALID
    assert lib.moe_route(None, 0, 8, 2, None, None, 1, FAKE, None, None, None, 8, FAKE, 4096, None) == INVALID


def test_backward_refuses_destinations_before_any_call():
    from quantization_nvfp4_quantize_b200.moe import MoELayerW4A16
    t = MoELayerW4A16.__new__(MoELayerW4A16)
    t.T, t.H, t.E, t.k_r, t.I, t.train_routing = 2, 64, 4, 2, 32, object()
    t.wq13 = torch.empty(4, 64, 64, dtype=torch.bfloat16, device="meta")
    t.wq2 = torch.empty(4, 64, 32, dtype=torch.bfloat16, device="meta")
    dy = torch.empty(2, 64, dtype=torch.bfloat16, device="meta")
    good = torch.empty(4, 64, 32, device="meta")
    for bad, match in ((torch.empty(4, 64, 63, device="meta"), "dw13 must be"),
                       (torch.empty(4, 64, 64, device="meta", dtype=torch.float16), "dw13 must be"),
                       (torch.empty(4, 64, 64, device="meta").transpose(1, 2), "dw13 must be"),
                       (torch.empty(4, 64, 64), "dw13 is on cpu")):
        with pytest.raises(ValueError, match=match):
            t.backward(dy, dw13=bad, dw2=good, accumulate=True)
    with pytest.raises(ValueError, match="columns must be contiguous"):
        t.backward(torch.empty(64, 2, dtype=torch.bfloat16, device="meta").t())
    x, logits = torch.empty(2, 64, device="meta"), torch.empty(2, 4, device="meta")
    with pytest.raises(ValueError, match="x must be bf16"):
        t.forward_train(x, logits)
    assert t.train_routing is not None          # a refused call leaves what was kept


def test_training_buffers_are_made_together(monkeypatch):
    """One that cannot be allocated leaves the layer as it was, and the next
    try makes all of them."""
    from quantization_nvfp4_quantize_b200.moe import MoELayerW4A16
    t = MoELayerW4A16.__new__(MoELayerW4A16)
    t.T, t.H, t.E, t.k_r, t.I = 2, 64, 4, 2, 32
    before = dict(t.__dict__)
    real = api.Act8.empty

    def full(M, K, device):
        if M == 4:                               # the gate/up rows
            raise torch.OutOfMemoryError("no memory")
        return real(M, K, device)

    with monkeypatch.context() as m:
        m.setattr(api.Act8, "empty", staticmethod(full))
        with pytest.raises(torch.OutOfMemoryError):
            t._train_buffers("cpu")
    assert t.__dict__ == before
    t._train_buffers("cpu")
    assert tuple(t.x8.codes.shape) == (2, 64) and tuple(t.y8.codes.shape) == (4, 64) and tuple(t.gh.shape) == (4, 32)


def test_training_pair_reports_waits_that_ran_out(monkeypatch):
    """Every call that can give up waiting gets the layer's status word;
    check_status raises for it once and keeps nothing."""
    import contextlib

    from quantization_nvfp4_quantize_b200 import moe
    bf = dict(dtype=torch.bfloat16)
    t = moe.MoELayerW4A16.__new__(moe.MoELayerW4A16)
    t.T, t.H, t.E, t.k_r, t.I, t.train_routing = 2, 64, 4, 2, 32, None
    t.wq13, t.wq2 = torch.zeros(4, 64, 64, **bf), torch.zeros(4, 64, 32, **bf)
    t.status = torch.zeros(1, dtype=torch.int32)
    seen = []

    def fake(name, result):
        def call(*args, **kw):
            seen.append((name, kw.get("dev_status")))
            return result
        return call

    monkeypatch.setattr(moe, "_current", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(api, "route", lambda logits, k_r, **kw: kw["out"])
    monkeypatch.setattr(api, "read_status", lambda word: int(word))
    for name in ("act8_quantize", "routed_rows_bf16", "swiglu_act8", "swiglu_act8_backward", "combine_rows",
                 "route_backward"):
        monkeypatch.setattr(api, name, lambda *a, **kw: torch.zeros(1))
    for name in ("ragged_gemm", "ragged_wgrad"):
        monkeypatch.setattr(api, name, fake(name, torch.zeros(1)))
    t.forward_train(torch.zeros(2, 64, **bf), torch.zeros(2, 4))
    assert t.backward(torch.zeros(2, 64, **bf)).status is t.status
    assert [n for n, _ in seen] == ["ragged_gemm"] * 3 + ["ragged_wgrad"] * 2 + ["ragged_gemm"]
    assert all(word is t.status for _, word in seen)
    t.check_status()
    t.status.fill_(5)
    with pytest.raises(_lib.Nvfp4Error, match="TIMEOUT"):
        t.check_status()
    t.check_status()                                   # reported once
    with pytest.raises(RuntimeError, match="no forward_train"):
        t.backward(torch.zeros(2, 64, **bf))


def test_overlapped_kernels_read_coherently():
    """A kernel that starts before its predecessor has finished may not load
    what that one writes as read-only data (the non-coherent path)."""
    import glob
    import os
    import re
    csrc = os.path.join(os.path.dirname(_lib.__file__), "csrc")
    files = [f for f in glob.glob(os.path.join(csrc, "*.cu")) if "grid_wait()" in open(f).read()]
    assert {os.path.basename(f) for f in files} >= {"act8.cu", "gemv.cu", "ragged.cu"}
    for f in files:
        code = re.sub(r"//[^\n]*", "", open(f).read())
        found = re.findall(r"const\s+\w+\s*\*\s*__restrict__|__ldg\s*\(|ld\.global\.nc\b[^\"]*", code)
        assert not found, (os.path.basename(f), found)


def test_accumulator_loads_are_tied_to_their_wait():
    """While another TMEM load is under way only the wait's own registers may be
    used: the ragged products name them."""
    import os
    code = open(os.path.join(os.path.dirname(_lib.__file__), "csrc", "ragged.cu")).read()
    assert "tmem_ld_wait(" in code and "tmem_ld_wait()" not in code


def test_logits_are_refused_without_asserts():
    """Logits that a bare pointer would read wrongly: an error of its own, not
    an assert that python -O takes out, and before anything is dropped."""
    from quantization_nvfp4_quantize_b200.moe import MoELayerW4A4, MoELayerW4A16
    good = torch.zeros(2, 4)
    bad = [good.bfloat16(), good.double(), torch.zeros(4, 2).t(), torch.zeros(2, 8)[:, :4]]
    t = MoELayerW4A16.__new__(MoELayerW4A16)
    t.T, t.H, t.E, t.k_r, t.I, t.train_routing = 2, 64, 4, 2, 32, object()
    t.wq13 = torch.empty(4, 64, 64, dtype=torch.bfloat16)
    d = MoELayerW4A4.__new__(MoELayerW4A4)
    d.H, d.E, d.c13 = 64, 4, torch.empty(4, 64, 32, dtype=torch.uint8)
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    for logits in bad:
        with pytest.raises(ValueError, match="route: logits must be contiguous f32"):
            api.route(logits, 2)
        with pytest.raises(ValueError, match="decode: logits must be contiguous f32"):
            d.decode(x, logits)
        with pytest.raises(ValueError, match="logits"):
            t.forward_train(x, logits)
    assert t.train_routing is not None
    with pytest.raises(ValueError, match="route: logits"):
        api.route(torch.zeros(4), 2)
    with pytest.raises(ValueError, match="route: out is for"):
        api.route(good, 2, out=api.empty_routing(3, 2, 4, "cpu"))


def test_ragged_wgrad_wait_limit_arguments():
    #       g     ldg  M    a     lda  N    K   E   off   out   stat  limit    stream
    good = [FAKE, 256, 100, FAKE, 256, 256, 256, 128, FAKE, FAKE, FAKE, 2000000, None]
    calls("nvfp4_debug_ragged_wgrad_wait_limit", good, [
        (10, None, INVALID), (11, 999999, INVALID), (11, 1000000001, INVALID), (0, None, INVALID), (1, 248, ALIGN)])
    # a result that needs a workspace
    calls("nvfp4_debug_ragged_wgrad_wait_limit", [FAKE, 256, 5000, *good[3:7], 1, *good[8:]], [(11, 2000000, WORKSPACE)])


def test_library_is_linked_without_the_binding(monkeypatch, tmp_path):
    """The C library needs neither torch's headers nor g++; a binding that
    cannot be built is reported all the same."""
    import importlib
    build = importlib.import_module("quantization_nvfp4_quantize_b200.build")
    lib = tmp_path / "lib.so"

    def no_binding(force=False):
        raise RuntimeError("no torch headers")

    def link(cmd):
        open(cmd[cmd.index("-o") + 1], "w").write("linked")

    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "build_binding", no_binding)
    monkeypatch.setattr(build, "_compile", lambda src, verbose: src)
    monkeypatch.setattr(build.subprocess, "check_call", link)
    with pytest.raises(RuntimeError, match="no torch headers"):
        build.build()
    assert lib.read_text() == "linked"
