"""The QUADS rollout MoE expert layer on the library's kernels.

One forward = the whole hot path (QUADS pages: gist.science/it sections 1
and 2.2 B; shd-paper.top abstract):

  1. moe_route                 top-k_r routing, expert-grouped padded row layout
  2. nvfp4_quantize(X)         amax -> s_x, codes/scales written to every routed
                               row of each token, channel scores, top-k S_x,
                               RAC residual rho_x for every routed row
  3. gather_weight_channels_cm W13q[:, :, S_x] as bf16 (e2m1 * sf), read from
                               the channel-major weight copy
  4. grouped GEMM (gate/up)    W4A4 + RAC, epilogue SwiGLU -> h bf16 and max |h|
  5. nvfp4_quantize(h)         over the valid routed rows, s_h from the epilogue's
                               max |h| (no amax pass): codes, S_h, rho_h
  6. gather_weight_channels_cm W2q[:, :, S_h]
  7. grouped GEMM (down)       W4A4 + RAC, epilogue router-weighted scatter-add
                               into Y [T x H] fp32

Weights are quantized to NVFP4 once at construction (the rollout engine holds
NVFP4 weights).  All buffers are allocated once; ``forward`` launches only the
library's kernels plus one memset of Y.
"""
from __future__ import annotations

import contextlib
import dataclasses

import torch

from . import api


def rac_channels(percent: float, K: int) -> int:
    """RAC channel count for "the top k% of channels" (gist.science/it 2.2 B,
    e.g. 50%): round(percent / 100 * K)."""
    return int(round(percent / 100.0 * K))


def _same_device(what: str, weight: torch.Tensor, **tensors):
    """The routing calls take bare pointers: every tensor has to be where the
    layer's weights are."""
    for name, t in tensors.items():
        if t.device != weight.device:
            raise ValueError(f"{what}: {name} is on {t.device}, the layer on {weight.device}")


def _current(device):
    """The device whose stream the calls go to, as the current one."""
    return contextlib.nullcontext() if device.index == torch.cuda.current_device() else torch.cuda.device(device)


class MoELayerW4A4:
    """rac_k: RAC channels of the gate/up input X (and of h unless rac_k_h is
    given); see rac_channels for a percentage.  rac_scope "expert" selects the
    channel sets per expert (nvfp4_quantize_experts): X through its complete
    routed copy, h directly; rac_mode must then be "bf16"."""

    def __init__(self, w13: torch.Tensor, w2: torch.Tensor, tokens: int, topk: int, rac_k: int,
                 seg_align: int = 256, rac_k_h: int | None = None, rac_mode: str = "bf16",
                 rac_scope: str = "tensor"):
        assert w13.dtype == torch.bfloat16 and w2.dtype == torch.bfloat16
        E, N13, H = w13.shape
        E2, H2, I = w2.shape
        assert E2 == E and H2 == H and N13 == 2 * I
        dev = w13.device
        self.E, self.H, self.I, self.T, self.k_r = E, H, I, tokens, topk
        assert rac_mode in ("bf16", "nvfp4") and rac_scope in ("tensor", "expert")
        assert rac_scope == "tensor" or (rac_mode == "bf16" and rac_k > 0 and (rac_k_h is None or rac_k_h > 0))
        self.rac_mode = rac_mode            # "nvfp4": second NVFP4 pass over the selected residual channels
        self.rac_scope = rac_scope
        self.rac_k = rac_k
        self.rac_k_h = rac_k if rac_k_h is None else rac_k_h
        self.rac_ld = -(-rac_k // 64) * 64 if rac_k else 0
        self.rac_ld_h = -(-self.rac_k_h // 64) * 64 if self.rac_k_h else 0
        _, self.s13, self.c13, self.sf13 = api.qdq_weights(w13, want_qdq=False, want_packed=True)
        _, self.s2, self.c2, self.sf2 = api.qdq_weights(w2, want_qdq=False, want_packed=True)
        # channel-major copies: the per-step RAC gathers read only the selected channels
        self.c13_cm, self.sf13_cm = api.weights_channel_major(self.c13, self.sf13, 2 * I, H)
        self.c2_cm, self.sf2_cm = api.weights_channel_major(self.c2, self.sf2, H, I)
        self.seg_align = seg_align          # 256: 2-SM GEMM tiles; 128: one SM per tile
        self.m_pad = api.padded_rows_bound(tokens, topk, E, seg_align)
        mp, ld, ldh = self.m_pad, max(self.rac_ld, 1), max(self.rac_ld_h, 1)
        self.xq = api.Quantized(
            codes=torch.empty(mp, H // 2, dtype=torch.uint8, device=dev),
            scales=torch.empty(api.scale_bytes(mp, H), dtype=torch.uint8, device=dev),
            s_t=torch.empty(1, dtype=torch.float32, device=dev),
            score=torch.empty(H, dtype=torch.float64, device=dev),
            sel=torch.empty(max(rac_k, 1), dtype=torch.int32, device=dev),
            r_sel=torch.empty(mp, ld, dtype=torch.bfloat16, device=dev))
        self.hq = api.Quantized(
            codes=torch.empty(mp, I // 2, dtype=torch.uint8, device=dev),
            scales=torch.empty(api.scale_bytes(mp, I), dtype=torch.uint8, device=dev),
            s_t=torch.empty(1, dtype=torch.float32, device=dev),
            score=torch.empty(I, dtype=torch.float64, device=dev),
            sel=torch.empty(max(self.rac_k_h, 1), dtype=torch.int32, device=dev),
            r_sel=torch.empty(mp, ldh, dtype=torch.bfloat16, device=dev))
        self.w_sel13 = torch.empty(E, 2 * I, ld, dtype=torch.bfloat16, device=dev)
        self.w_sel2 = torch.empty(E, H, ldh, dtype=torch.bfloat16, device=dev)
        self.h = torch.empty(mp, I, dtype=torch.bfloat16, device=dev)
        self.y = torch.empty(tokens, H, dtype=torch.float32, device=dev)
        self.h_amax = torch.empty(1, dtype=torch.float32, device=dev)
        lib = api._lib.load()
        self.ws_x = api._ws(lib.nvfp4_quantize_workspace_size(tokens, H), dev)
        self.ws_h = api._ws(lib.nvfp4_quantize_workspace_size(mp, I), dev)
        self.routing = None
        if rac_scope == "expert":
            # per-expert sets: [E x k] selections, the routed copy of X, and
            # workspaces sized for the routed rows
            self.xq.sel = torch.empty(E, rac_k, dtype=torch.int32, device=dev)
            self.hq.sel = torch.empty(E, self.rac_k_h, dtype=torch.int32, device=dev)
            self.xq.score = self.hq.score = None
            self.x_routed = torch.empty(mp, H, dtype=torch.bfloat16, device=dev)
            self.ws_x = api._ws(lib.nvfp4_quantize_experts_workspace_size(mp, H, E, seg_align), dev)
            self.ws_h = api._ws(lib.nvfp4_quantize_experts_workspace_size(mp, I, E, seg_align), dev)

    def forward(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        if self.rac_scope == "expert":
            return self._forward_experts(x, logits)
        E, H, I, k, kh = self.E, self.H, self.I, self.rac_k, self.rac_k_h
        r = api.route(logits, self.k_r, self.m_pad, self.seg_align) if self.routing is None else self._route_into(logits)
        self.routing = r
        nvfp4_rac = self.rac_mode == "nvfp4"          # the second pass writes the RAC operand
        api.quantize(x, rac_k=k, rac_ld=self.rac_ld, dst_rows=r.dst_row, fanout=self.k_r, m_out=self.m_pad,
                     out=self.xq, workspace=self.ws_x, want_residual=not nvfp4_rac)
        if k and self.rac_mode == "nvfp4":
            api.rac_residual_nvfp4(x, self.xq, k, self.rac_ld, dst_rows=r.dst_row, fanout=self.k_r, m_out=self.m_pad)
        if k:
            api.gather_weight_channels_cm(self.c13_cm, self.sf13_cm, 2 * I, H, self.xq.sel, k, self.rac_ld,
                                          out=self.w_sel13)
        api.grouped_gemm(self.xq.codes, self.xq.scales, self.xq.s_t, self.m_pad, self.c13, self.sf13, self.s13,
                         2 * I, H, E, r.offsets, seg_align=self.seg_align, rac_ld=self.rac_ld if k else 0, rho=self.xq.r_sel,
                         w_sel=self.w_sel13, epilogue=api.EPI_SWIGLU_BF16, row_token=r.row_token,
                         row_gate=r.row_gate, out=self.h, amax_out=self.h_amax)
        api.quantize(self.h, rac_k=kh, rac_ld=self.rac_ld_h, m_out=self.m_pad, m_valid=r.offsets[E:],
                     amax=self.h_amax, out=self.hq, workspace=self.ws_h, want_residual=not nvfp4_rac)
        if kh and self.rac_mode == "nvfp4":
            api.rac_residual_nvfp4(self.h, self.hq, kh, self.rac_ld_h, m_out=self.m_pad, m_valid=r.offsets[E:])
        if kh:
            api.gather_weight_channels_cm(self.c2_cm, self.sf2_cm, H, I, self.hq.sel, kh, self.rac_ld_h,
                                          out=self.w_sel2)
        self.y.zero_()
        api.grouped_gemm(self.hq.codes, self.hq.scales, self.hq.s_t, self.m_pad, self.c2, self.sf2, self.s2,
                         H, I, E, r.offsets, seg_align=self.seg_align, rac_ld=self.rac_ld_h if kh else 0,
                         rho=self.hq.r_sel, w_sel=self.w_sel2,
                         epilogue=api.EPI_SCATTER_ADD_F32, row_token=r.row_token, row_gate=r.row_gate, out=self.y)
        return self.y

    def _forward_experts(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        """The layer with one RAC channel set per expert for X and for h."""
        E, H, I, k, kh, sa = self.E, self.H, self.I, self.rac_k, self.rac_k_h, self.seg_align
        r = api.route(logits, self.k_r, self.m_pad, sa) if self.routing is None else self._route_into(logits)
        self.routing = r
        api.routed_rows_bf16(x, r.row_token, self.m_pad, out=self.x_routed)
        api.quantize_experts(self.x_routed, r.offsets, E, sa, rac_k=k, rac_ld=self.rac_ld, out=self.xq,
                             workspace=self.ws_x)
        api.gather_weight_channels_cm_experts(self.c13_cm, self.sf13_cm, 2 * I, H, self.xq.sel, k, self.rac_ld,
                                              out=self.w_sel13)
        api.grouped_gemm(self.xq.codes, self.xq.scales, self.xq.s_t, self.m_pad, self.c13, self.sf13, self.s13,
                         2 * I, H, E, r.offsets, seg_align=sa, rac_ld=self.rac_ld, rho=self.xq.r_sel,
                         w_sel=self.w_sel13, epilogue=api.EPI_SWIGLU_BF16, row_token=r.row_token,
                         row_gate=r.row_gate, out=self.h, amax_out=self.h_amax)
        api.quantize_experts(self.h, r.offsets, E, sa, rac_k=kh, rac_ld=self.rac_ld_h, amax=self.h_amax,
                             out=self.hq, workspace=self.ws_h)
        api.gather_weight_channels_cm_experts(self.c2_cm, self.sf2_cm, H, I, self.hq.sel, kh, self.rac_ld_h,
                                              out=self.w_sel2)
        self.y.zero_()
        api.grouped_gemm(self.hq.codes, self.hq.scales, self.hq.s_t, self.m_pad, self.c2, self.sf2, self.s2,
                         H, I, E, r.offsets, seg_align=sa, rac_ld=self.rac_ld_h, rho=self.hq.r_sel, w_sel=self.w_sel2,
                         epilogue=api.EPI_SCATTER_ADD_F32, row_token=r.row_token, row_gate=r.row_gate, out=self.y)
        return self.y

    def decode(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        """The layer for the few tokens of a decode step (any number of rows,
        not the constructor's): the same NVFP4 weights, activations in BF16
        (W4A16: nothing is quantized or compensated), two matrix-vector
        calls after the routing.  x bf16 [t, H], logits f32 [t, E]; returns
        f32 [t, H], a new tensor.  Bound by the weights of the experts in use;
        for many tokens forward's grouped GEMM is the faster form (top-8 of 128
        experts, H 2048, I 768, replayed graphs: 64 tokens 185 us against 221
        without RAC and 302 with 64 RAC channels, 96 tokens 250 against 222 and
        303, 128 tokens 335 against 223 and 304)."""
        _same_device("decode", self.c13, x=x, logits=logits)
        if tuple(x.shape) != (logits.shape[0], self.H) or tuple(logits.shape) != (logits.shape[0], self.E):
            raise ValueError(f"decode: need x [t, {self.H}] and logits [t, {self.E}], got {tuple(x.shape)} and "
                             f"{tuple(logits.shape)}")
        api.check_logits("decode", logits)
        if logits.shape[0] == 0:
            return torch.empty(0, self.H, dtype=torch.float32, device=x.device)
        with _current(x.device):
            r = api.route(logits, self.k_r, seg_align=1)
            h = api.nvfp4_gemv(x, self.c13, self.sf13, self.s13, 2 * self.I, self.H, expert_idx=r.topk_idx,
                               epilogue=api.EPI_SWIGLU_BF16)
            return api.nvfp4_gemv(h, self.c2, self.sf2, self.s2, self.H, self.I, expert_idx=r.topk_idx,
                                  epilogue=api.EPI_COMBINE_F32, gate=r.topk_gate)

    def _route_into(self, logits):
        lib = api._lib.load()
        r = self.routing
        T, E = logits.shape
        ws = getattr(self, "_ws_route", None)
        if ws is None:
            ws = self._ws_route = api._ws(lib.moe_route_workspace_size(T, E), logits.device)
        api.check(lib.moe_route(api._p(logits), T, E, self.k_r, api._p(r.topk_idx), api._p(r.topk_gate),
                                self.seg_align, api._p(r.offsets), api._p(r.dst_row), api._p(r.row_token), api._p(r.row_gate),
                                r.m_pad_max, api._p(ws), ws.numel(), api._stream(logits.device)))
        return r


@dataclasses.dataclass
class LayerGrads:
    """Gradients of MoELayerW4A16 (f32)."""
    dx: torch.Tensor            # [T, H]
    dlogits: torch.Tensor       # [T, E]
    dw13: torch.Tensor          # [E, 2I, H], of the fake-quantized weights (straight through to the bf16 ones)
    dw2: torch.Tensor           # [E, H, I]
    status: torch.Tensor | None = None   # int32 [1], the layer's status word: see MoELayerW4A16.check_status


class MoELayerW4A16:
    """Trainer-side asymmetric QAT layer (gist.science/it 2.2 A): the expert
    weights are fake-quantized to NVFP4 (nvfp4_qdq_weights: bf16 ->
    NVFP4 with each expert tensor's own scale -> bf16), activations stay
    BF16, and both expert GEMMs run as BF16 grouped GEMMs on the tensor cores:

      1. moe_route               as in MoELayerW4A4
      2. moe_gather_rows_bf16    X rows to their routed rows
      3. BF16 grouped GEMM       X Wq13^T, epilogue SwiGLU -> h bf16
      4. BF16 grouped GEMM       h Wq2^T, epilogue router-weighted scatter-add
                                 into Y [T x H] fp32

    forward_train / backward are the training step's pair: unpadded ragged
    segments, X and the SwiGLU's inputs kept in 8 bits in between, no atomics
    (the same inputs give the same bits).  A bounded wait of their kernels that
    runs out is reported in a status word only: check_status reads it.
    """

    def __init__(self, w13: torch.Tensor, w2: torch.Tensor, tokens: int, topk: int, seg_align: int = 256):
        assert w13.dtype == torch.bfloat16 and w2.dtype == torch.bfloat16
        E, N13, H = w13.shape
        E2, H2, I = w2.shape
        assert E2 == E and H2 == H and N13 == 2 * I
        dev = w13.device
        self.E, self.H, self.I, self.T, self.k_r = E, H, I, tokens, topk
        self.wq13 = torch.empty_like(w13)
        self.wq2 = torch.empty_like(w2)
        self.s13 = torch.empty(E, dtype=torch.float32, device=dev)
        self.s2 = torch.empty(E, dtype=torch.float32, device=dev)
        lib = api._lib.load()
        self.ws_qdq = api._ws(max(lib.nvfp4_qdq_workspace_size(E, 2 * I, H), lib.nvfp4_qdq_workspace_size(E, H, I)), dev)
        self.set_weights(w13, w2)
        self.seg_align = seg_align
        self.m_pad = api.padded_rows_bound(tokens, topk, E, seg_align)
        self.xr = torch.zeros(self.m_pad, H, dtype=torch.bfloat16, device=dev)
        self.h = torch.empty(self.m_pad, I, dtype=torch.bfloat16, device=dev)
        self.y = torch.empty(tokens, H, dtype=torch.float32, device=dev)
        self.routing = None
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def set_weights(self, w13: torch.Tensor, w2: torch.Tensor):
        """Fake-quantize new bf16 weights into the layer (the per-step work of
        QAT, where the weights change every optimizer step).  What forward_train
        kept belongs to the old ones: backward refuses until its next call."""
        self.train_routing = None
        lib = api._lib.load()
        st = api._stream(w13.device)
        for w, wq, s_t in ((w13, self.wq13, self.s13), (w2, self.wq2, self.s2)):
            assert w.shape == wq.shape and w.dtype == torch.bfloat16 and w.is_contiguous()
            G, rows, cols = w.shape
            api.check(lib.nvfp4_qdq_weights(api._p(w), G, rows, cols, api._p(wq), api._p(s_t), None, None,
                                            api._p(self.ws_qdq), self.ws_qdq.numel(), st))

    def forward(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        E, H, I = self.E, self.H, self.I
        r = api.route(logits, self.k_r, self.m_pad, self.seg_align) if self.routing is None else self._route_into(logits)
        self.routing = r
        api.gather_rows_bf16(x, r.dst_row, self.m_pad, out=self.xr)
        api.bf16_grouped_gemm(self.xr, self.m_pad, self.wq13, 2 * I, H, E, r.offsets, seg_align=self.seg_align,
                              epilogue=api.EPI_SWIGLU_BF16, row_token=r.row_token, row_gate=r.row_gate, out=self.h)
        self.y.zero_()
        api.bf16_grouped_gemm(self.h, self.m_pad, self.wq2, H, I, E, r.offsets, seg_align=self.seg_align,
                              epilogue=api.EPI_SCATTER_ADD_F32, row_token=r.row_token, row_gate=r.row_gate,
                              out=self.y)
        return self.y

    def _train_buffers(self, dev):
        """Buffers of the training pair, made at the first forward_train: all of
        them or, where memory runs out, none."""
        m, H, I = self.T * self.k_r, self.H, self.I
        bf = dict(dtype=torch.bfloat16, device=dev)
        made = dict(
            rows_h=torch.empty(m, H, **bf),             # routed X, later routed dY
            rows_y=torch.empty(m, H, **bf),             # down rows, later dX rows
            y13=torch.empty(m, 2 * I, **bf),            # gate/up rows, later their gradient
            h_t=torch.empty(m, I, **bf),                # h, later its gradient
            gh=torch.empty(m, I, **bf),                 # router-weighted h
            dgate=torch.empty(m, dtype=torch.float32, device=dev),
            # kept between forward_train and backward: the routing beside the rows
            # it belongs to, so that a replayed graph's forward writes all of it
            x8=api.Act8.empty(self.T, H, dev),
            y8=api.Act8.empty(m, 2 * I, dev),
            kept_routing=api.empty_routing(self.T, self.k_r, self.E, dev, seg_align=1),
            ws_kept=api._ws(api._lib.load().moe_route_workspace_size(self.T, self.E), dev))
        self.__dict__.update(made)

    def forward_train(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        """The layer with what backward needs kept in 8 bits: X (per token, not
        per routed copy) and the gate/up rows.  Returns Y f32 [T, H], a new
        tensor.  The gate/up rows and every expert's down rows are rounded to
        bf16 before the SwiGLU and the combine, which forward's fused epilogues
        keep in f32, and so are the dX rows in backward; the kept rows are those
        that the SwiGLU saw.  I must be a multiple of 32.  What is kept lives in the layer's
        buffers: a later call, or a replayed graph that holds one, takes its
        place.  After a call that fails on its way nothing is kept; a kernel
        that gave up waiting shows in check_status only."""
        if tuple(x.shape) != (self.T, self.H) or tuple(logits.shape) != (self.T, self.E):
            raise ValueError(f"forward_train: need x [{self.T}, {self.H}] and logits [{self.T}, {self.E}], got "
                             f"{tuple(x.shape)} and {tuple(logits.shape)}")
        if x.dtype != torch.bfloat16 or logits.dtype != torch.float32:
            raise ValueError(f"forward_train: x must be bf16 and logits f32, got {x.dtype} and {logits.dtype}")
        api.check_logits("forward_train", logits)
        _same_device("forward_train", self.wq13, x=x, logits=logits)
        if not hasattr(self, "x8"):
            self._train_buffers(x.device)
        self.train_routing = None
        with _current(x.device):
            r = api.route(logits, self.k_r, out=self.kept_routing, workspace=self.ws_kept)
            api.act8_quantize(x, out=self.x8)
            api.routed_rows_bf16(x, r.row_token, r.m_pad_max, out=self.rows_h)
            api.ragged_gemm(self.rows_h, self.wq13, r.offsets, out=self.y13, dev_status=self.status)
            api.swiglu_act8(self.y13, h=self.h_t, out=self.y8)
            api.ragged_gemm(self.h_t, self.wq2, r.offsets, out=self.rows_y, dev_status=self.status)
            y = api.combine_rows(self.rows_y, r.dst_row, gate=r.topk_gate)
        self.train_routing = r
        return y

    def backward(self, dy: torch.Tensor, *, dw13: torch.Tensor | None = None, dw2: torch.Tensor | None = None,
                 accumulate: bool = False) -> LayerGrads:
        """Gradients of the last forward_train, called or replayed, for dY (bf16
        [T, H]), with its weights (call it before set_weights).  dw13 / dw2: where the weight
        gradients go (f32 or bf16, contiguous); accumulate adds to them.  A
        refused call changes neither; one that fails on its way (no memory for
        a workspace) may have written the first of them, and check_status tells
        whether both are complete."""
        r = self.train_routing
        if r is None:
            raise RuntimeError("backward: no forward_train to differentiate")
        if tuple(dy.shape) != (self.T, self.H) or dy.dtype != torch.bfloat16:
            raise ValueError(f"backward: dy must be bf16 [{self.T}, {self.H}]")
        if accumulate and (dw13 is None or dw2 is None):
            raise ValueError("backward: accumulate needs dw13 and dw2")
        _same_device("backward", self.wq13, dy=dy)
        if dy.stride(1) != 1 and self.H > 1:
            raise ValueError("backward: dy: columns must be contiguous")
        for name, d, w in (("dw13", dw13, self.wq13), ("dw2", dw2, self.wq2)):
            if d is None:
                continue
            _same_device("backward", self.wq13, **{name: d})
            if d.shape != w.shape or d.dtype not in (torch.float32, torch.bfloat16) or not d.is_contiguous():
                raise ValueError(f"backward: {name} must be contiguous f32 or bf16 {list(w.shape)}")
        with _current(dy.device):
            # routed dY; u = dY W2, the gradient of h before the router's weight
            api.routed_rows_bf16(dy, r.row_token, r.m_pad_max, out=self.rows_h)
            api.ragged_gemm(self.rows_h, self.wq2, r.offsets, transpose=True, out=self.h_t, dev_status=self.status)
            api.swiglu_act8_backward(self.y8, self.h_t, row_gate=r.row_gate, dy=self.y13, gh=self.gh, dgate=self.dgate)
            dw2 = api.ragged_wgrad(self.rows_h, self.gh, r.offsets, out=dw2, accumulate=accumulate, dev_status=self.status)
            dw13 = api.ragged_wgrad(self.y13, self.x8, r.offsets, a_rows=r.row_token, out=dw13, accumulate=accumulate,
                                    dev_status=self.status)
            api.ragged_gemm(self.y13, self.wq13, r.offsets, transpose=True, out=self.rows_y, dev_status=self.status)
            dx = api.combine_rows(self.rows_y, r.dst_row)
            dlogits = api.route_backward(r.topk_idx, r.topk_gate, r.dst_row, self.dgate, self.E)
        return LayerGrads(dx, dlogits, dw13, dw2, self.status)

    def check_status(self):
        """Raises Nvfp4Error if a wait ran out in a forward_train or backward
        since the last check: their results, and gradients they were added to,
        are then incomplete, and nothing is kept.  Waits for the current stream;
        call it before an optimizer step uses the gradients."""
        with _current(self.status.device):
            status = api.read_status(self.status)
            if status == 0:
                return
            self.status.zero_()
        self.train_routing = None
        raise api.Nvfp4Error(status, "a kernel of the training pair gave up waiting; drop the step's results and gradients")

    _route_into = MoELayerW4A4._route_into


class MoELayerW8A8:
    """The FP8 rollout the pages compare NVFP4 against (gist.science/it
    sections 1 and 4), on the same expert layer: per-tensor E4M3 weights
    (quantized once) and activations (quantized online, X to its routed rows,
    h with the scale from the gate/up epilogue's max |h|), grouped E4M3 GEMMs
    with the SwiGLU and router-weighted combine epilogues.  No RAC."""

    def __init__(self, w13: torch.Tensor, w2: torch.Tensor, tokens: int, topk: int, seg_align: int = 256):
        E, N13, H = w13.shape
        _, _, I = w2.shape
        dev = w13.device
        self.E, self.H, self.I, self.T, self.k_r, self.seg_align = E, H, I, tokens, topk, seg_align
        self.c13, self.s13 = api.fp8_quantize(w13.contiguous())
        self.c2, self.s2 = api.fp8_quantize(w2.contiguous())
        self.m_pad = api.padded_rows_bound(tokens, topk, E, seg_align)
        self.xc = torch.empty(self.m_pad, H, dtype=torch.uint8, device=dev)
        self.xs = torch.empty(1, dtype=torch.float32, device=dev)
        self.h = torch.empty(self.m_pad, I, dtype=torch.bfloat16, device=dev)
        self.hc = torch.empty(self.m_pad, I, dtype=torch.uint8, device=dev)
        self.hs = torch.empty(1, dtype=torch.float32, device=dev)
        self.h_amax = torch.empty(1, dtype=torch.float32, device=dev)
        self.y = torch.empty(tokens, H, dtype=torch.float32, device=dev)
        self.routing = None

    def forward(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        E, H, I = self.E, self.H, self.I
        r = api.route(logits, self.k_r, self.m_pad, self.seg_align) if self.routing is None else self._route_into(logits)
        self.routing = r
        api.fp8_quantize(x, dst_rows=r.dst_row, fanout=self.k_r, m_out=self.m_pad, codes=self.xc, s_out=self.xs)
        api.w8a8_grouped_gemm(self.xc, self.xs, self.m_pad, self.c13, self.s13, 2 * I, H, E, r.offsets,
                              seg_align=self.seg_align, epilogue=api.EPI_SWIGLU_BF16, row_token=r.row_token,
                              row_gate=r.row_gate, out=self.h, amax_out=self.h_amax)
        api.fp8_quantize(self.h, amax=self.h_amax, codes=self.hc, s_out=self.hs)
        self.y.zero_()
        api.w8a8_grouped_gemm(self.hc, self.hs, self.m_pad, self.c2, self.s2, H, I, E, r.offsets,
                              seg_align=self.seg_align, epilogue=api.EPI_SCATTER_ADD_F32, row_token=r.row_token,
                              row_gate=r.row_gate, out=self.y)
        return self.y

    _route_into = MoELayerW4A4._route_into


class DenseLayerW4A4:
    """Single dense W4A4 + RAC layer: Y = Xq Wq^T + RAC, fp32 out (one expert,
    identity routing)."""

    def __init__(self, w: torch.Tensor, tokens: int, rac_k: int):
        N, K = w.shape
        self.N, self.K, self.T, self.rac_k = N, K, tokens, rac_k
        self.rac_ld = -(-rac_k // 64) * 64 if rac_k else 0
        _, self.s_w, self.c_w, self.sf_w = api.qdq_weights(w.unsqueeze(0).contiguous(), want_qdq=False,
                                                           want_packed=True)
        self.m_pad = api.padded_rows_bound(tokens, 1, 1)
        dev = w.device
        self.out = torch.empty(self.m_pad, N, dtype=torch.float32, device=dev)
        self.w_sel = torch.empty(1, N, max(self.rac_ld, 1), dtype=torch.bfloat16, device=dev)
        self.logits = torch.zeros(tokens, 1, dtype=torch.float32, device=dev)

    def forward(self, x: torch.Tensor):
        r = api.route(self.logits, 1, self.m_pad)
        self.routing = r
        xq = api.quantize(x, rac_k=self.rac_k, rac_ld=self.rac_ld, dst_rows=r.dst_row, fanout=1, m_out=self.m_pad)
        self.xq = xq
        if self.rac_k:
            api.gather_weight_channels(self.c_w, self.sf_w, self.N, self.K, xq.sel, self.rac_k, self.rac_ld,
                                       out=self.w_sel)
        api.grouped_gemm(xq.codes, xq.scales, xq.s_t, self.m_pad, self.c_w, self.sf_w, self.s_w, self.N, self.K, 1,
                         r.offsets, rac_ld=self.rac_ld, rho=xq.r_sel, w_sel=self.w_sel,
                         epilogue=api.EPI_STORE_F32, row_token=r.row_token, row_gate=r.row_gate, out=self.out)
        return self.out[: self.T]

    def decode(self, x: torch.Tensor) -> torch.Tensor:
        """A few rows' product with the same NVFP4 weight, activations in BF16
        (any number of rows); f32 [rows, N], a new tensor."""
        return api.nvfp4_gemv(x, self.c_w, self.sf_w, self.s_w, self.N, self.K)
