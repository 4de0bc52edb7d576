"""Thin PyTorch-facing binding of the C ABI (include/nvfp4_quads.h).

Each function only allocates output buffers with torch (device memory is
PyTorch's), marshals pointers and sizes, and calls the library on the current
CUDA stream; every step of the computation runs in the library's kernels.
There is no CPU or PyTorch fallback.
"""
from __future__ import annotations

import dataclasses
import functools

import torch

from . import _lib
from ._lib import check

U8 = torch.uint8
I32 = torch.int32
F32 = torch.float32
F64 = torch.float64
BF16 = torch.bfloat16

EPI_STORE_F32 = 0
EPI_SWIGLU_BF16 = 1
EPI_SCATTER_ADD_F32 = 2
EPI_COMBINE_F32 = 3          # nvfp4_gemv only


def _p(t):
    return None if t is None else t.data_ptr()


def _stream(device=None):
    if device is not None and torch.device(device).type != "cuda":
        raise ValueError(f"the NVFP4 kernels run on CUDA tensors only (got a tensor on {device}); "
                         "there is no CPU path")
    return torch.cuda.current_stream(device).cuda_stream


def _ws(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(16, int(nbytes)), dtype=U8, device=device)


def scale_bytes(rows: int, K: int) -> int:
    """Bytes of a swizzled scale buffer: rows padded to 128, K/16 scales each."""
    return -(-rows // 128) * 128 * (K // 16)


@dataclasses.dataclass
class Quantized:
    codes: torch.Tensor          # uint8 [M_out, K/2]
    scales: torch.Tensor         # uint8 swizzled
    s_t: torch.Tensor            # float32 [1]
    score: torch.Tensor | None   # float64 [K]
    sel: torch.Tensor | None     # int32 [rac_k]
    r_sel: torch.Tensor | None   # bf16 [M_out, rac_ld]


def quantize(x: torch.Tensor, *, rac_k: int = 0, rac_ld: int | None = None, s_t: torch.Tensor | None = None,
             amax: torch.Tensor | None = None,
             dst_rows: torch.Tensor | None = None, fanout: int = 1, m_out: int | None = None,
             m_valid: torch.Tensor | None = None, want_score: bool = False, out: Quantized | None = None,
             workspace: torch.Tensor | None = None, dev_status: torch.Tensor | None = None,
             want_residual: bool = True) -> Quantized:
    """nvfp4_quantize on a bf16 [M, K] tensor (see the header for semantics).
    want_residual=False selects the RAC channels without writing r_sel."""
    lib = _lib.load()
    assert x.dtype == BF16 and x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    dev = x.device
    if m_out is None:
        m_out = M
    if rac_ld is None:
        rac_ld = -(-rac_k // 64) * 64 if rac_k else 0
    if out is None:
        out = Quantized(
            codes=torch.empty(m_out, K // 2, dtype=U8, device=dev),
            scales=torch.empty(scale_bytes(m_out, K), dtype=U8, device=dev),
            s_t=torch.empty(1, dtype=F32, device=dev),
            score=torch.empty(K, dtype=F64, device=dev) if (want_score or rac_k) else None,
            sel=torch.empty(max(rac_k, 1), dtype=I32, device=dev) if rac_k else None,
            r_sel=torch.empty(m_out, max(rac_ld, 1), dtype=BF16, device=dev) if rac_k else None,
        )
    if workspace is None:
        workspace = _ws(lib.nvfp4_quantize_workspace_size(M, K), dev)
    check(lib.nvfp4_quantize(_p(x), M, K, x.stride(0), _p(m_valid), _p(s_t), _p(amax), _p(out.s_t), _p(dst_rows),
                             fanout, m_out, _p(out.codes), _p(out.scales), _p(out.score), rac_k, rac_ld,
                             _p(out.sel), _p(out.r_sel) if want_residual else None, _p(dev_status), _p(workspace),
                             workspace.numel(), _stream(dev)))
    return out


def quantize_experts(x: torch.Tensor, offsets: torch.Tensor, E: int, seg_align: int, *, rac_k: int,
                     rac_ld: int | None = None, s_t: torch.Tensor | None = None, amax: torch.Tensor | None = None,
                     want_score: bool = False, out: Quantized | None = None, workspace: torch.Tensor | None = None,
                     dev_status: torch.Tensor | None = None) -> Quantized:
    """nvfp4_quantize_experts on expert-grouped routed rows bf16 [M, K]: one
    RAC channel set per expert (sel [E, rac_k], score [E, K])."""
    lib = _lib.load()
    assert x.dtype == BF16 and x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    dev = x.device
    if rac_ld is None:
        rac_ld = -(-rac_k // 64) * 64
    if out is None:
        out = Quantized(
            codes=torch.empty(M, K // 2, dtype=U8, device=dev),
            scales=torch.empty(scale_bytes(M, K), dtype=U8, device=dev),
            s_t=torch.empty(1, dtype=F32, device=dev),
            score=torch.empty(E, K, dtype=F64, device=dev) if want_score else None,
            sel=torch.empty(E, rac_k, dtype=I32, device=dev),
            r_sel=torch.empty(M, rac_ld, dtype=BF16, device=dev),
        )
    if workspace is None:
        workspace = _ws(lib.nvfp4_quantize_experts_workspace_size(M, K, E, seg_align), dev)
    check(lib.nvfp4_quantize_experts(_p(x), M, K, x.stride(0), _p(offsets), E, seg_align, _p(s_t), _p(amax),
                                     _p(out.s_t), _p(out.codes), _p(out.scales), _p(out.score), rac_k, rac_ld,
                                     _p(out.sel), _p(out.r_sel), _p(dev_status), _p(workspace), workspace.numel(),
                                     _stream(dev)))
    return out


def qdq_weights(w: torch.Tensor, *, want_qdq: bool = True, want_packed: bool = False):
    """nvfp4_qdq_weights on bf16 [G, rows, cols] (or [rows, cols]).
    Returns (w_qdq or None, s_t [G], codes or None, scales or None)."""
    lib = _lib.load()
    assert w.dtype == BF16 and w.is_contiguous()
    squeeze = w.dim() == 2
    w3 = w.unsqueeze(0) if squeeze else w
    G, rows, cols = w3.shape
    dev = w.device
    w_qdq = torch.empty_like(w3) if want_qdq else None
    s_t = torch.empty(G, dtype=F32, device=dev)
    codes = torch.empty(G, rows, cols // 2, dtype=U8, device=dev) if want_packed else None
    scales = torch.empty(G, scale_bytes(rows, cols), dtype=U8, device=dev) if want_packed else None
    ws = _ws(lib.nvfp4_qdq_workspace_size(G, rows, cols), dev)
    check(lib.nvfp4_qdq_weights(_p(w3), G, rows, cols, _p(w_qdq), _p(s_t), _p(codes), _p(scales), _p(ws),
                                ws.numel(), _stream(dev)))
    if squeeze and w_qdq is not None:
        w_qdq = w_qdq[0]
    return w_qdq, s_t, codes, scales


@dataclasses.dataclass
class Routing:
    topk_idx: torch.Tensor      # int32 [T, k_r]
    topk_gate: torch.Tensor     # float32 [T, k_r]
    offsets: torch.Tensor       # int32 [E+1]
    dst_row: torch.Tensor       # int32 [T, k_r]
    row_token: torch.Tensor     # int32 [M_pad_max]
    row_gate: torch.Tensor      # float32 [M_pad_max]
    m_pad_max: int
    seg_align: int = 128


def padded_rows_bound(T: int, k_r: int, E: int, seg_align: int = 128) -> int:
    return -(-(T * k_r + E * (seg_align - 1)) // seg_align) * seg_align


def route(logits: torch.Tensor, k_r: int, m_pad_max: int | None = None, seg_align: int = 128) -> Routing:
    lib = _lib.load()
    assert logits.dtype == F32 and logits.is_contiguous()
    T, E = logits.shape
    dev = logits.device
    if m_pad_max is None:
        m_pad_max = padded_rows_bound(T, k_r, E, seg_align)
    r = Routing(torch.empty(T, k_r, dtype=I32, device=dev), torch.empty(T, k_r, dtype=F32, device=dev),
                torch.empty(E + 1, dtype=I32, device=dev), torch.empty(T, k_r, dtype=I32, device=dev),
                torch.empty(m_pad_max, dtype=I32, device=dev), torch.empty(m_pad_max, dtype=F32, device=dev),
                m_pad_max, seg_align)
    ws = _ws(lib.moe_route_workspace_size(T, E), dev)
    check(lib.moe_route(_p(logits), T, E, k_r, _p(r.topk_idx), _p(r.topk_gate), seg_align, _p(r.offsets), _p(r.dst_row),
                        _p(r.row_token), _p(r.row_gate), m_pad_max, _p(ws), ws.numel(), _stream(dev)))
    return r


def gather_weight_channels(codes: torch.Tensor, scales: torch.Tensor, N: int, K: int, sel: torch.Tensor,
                           k: int, ld: int, out: torch.Tensor | None = None) -> torch.Tensor:
    lib = _lib.load()
    E = codes.shape[0]
    if out is None:
        out = torch.empty(E, N, ld, dtype=BF16, device=codes.device)
    check(lib.nvfp4_gather_weight_channels(_p(codes), _p(scales), E, N, K, _p(sel), k, ld, _p(out),
                                           _stream(codes.device)))
    return out


def weights_channel_major(codes: torch.Tensor, scales: torch.Tensor, N: int, K: int):
    """nvfp4_weights_channel_major: (codes_cm [E, K, N/2], scales_cm [E, K/16, N])."""
    lib = _lib.load()
    E = codes.shape[0]
    ccm = torch.empty(E, K, N // 2, dtype=U8, device=codes.device)
    scm = torch.empty(E, K // 16, N, dtype=U8, device=codes.device)
    check(lib.nvfp4_weights_channel_major(_p(codes), _p(scales), E, N, K, _p(ccm), _p(scm), _stream(codes.device)))
    return ccm, scm


def gather_weight_channels_cm(codes_cm: torch.Tensor, scales_cm: torch.Tensor, N: int, K: int, sel: torch.Tensor,
                              k: int, ld: int, out: torch.Tensor | None = None) -> torch.Tensor:
    lib = _lib.load()
    E = codes_cm.shape[0]
    if out is None:
        out = torch.empty(E, N, ld, dtype=BF16, device=codes_cm.device)
    check(lib.nvfp4_gather_weight_channels_cm(_p(codes_cm), _p(scales_cm), E, N, K, _p(sel), k, ld, _p(out),
                                              _stream(codes_cm.device)))
    return out


def gather_weight_channels_cm_experts(codes_cm: torch.Tensor, scales_cm: torch.Tensor, N: int, K: int,
                                      sel: torch.Tensor, k: int, ld: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """nvfp4_gather_weight_channels_cm_experts: expert e gathers sel[e, :k]."""
    lib = _lib.load()
    E = codes_cm.shape[0]
    assert sel.dtype == I32 and sel.numel() >= E * k
    if out is None:
        out = torch.empty(E, N, ld, dtype=BF16, device=codes_cm.device)
    check(lib.nvfp4_gather_weight_channels_cm_experts(_p(codes_cm), _p(scales_cm), E, N, K, _p(sel), k, ld, _p(out),
                                                      _stream(codes_cm.device)))
    return out


def grouped_gemm(a_codes, a_scales, a_s_t, m_pad_max, b_codes, b_scales, b_s_t, N, K, E, offsets, *,
                 seg_align=128, rac_ld=0, rho=None, w_sel=None, epilogue=EPI_STORE_F32, row_token=None, row_gate=None,
                 out=None, ld_out=None, amax_out=None, dev_status=None):
    """moe_w4a4_grouped_gemm_rac (see the header)."""
    lib = _lib.load()
    if ld_out is None:
        ld_out = out.stride(0)
    check(lib.moe_w4a4_grouped_gemm_rac(_p(a_codes), _p(a_scales), _p(a_s_t), m_pad_max, _p(b_codes),
                                        _p(b_scales), _p(b_s_t), N, K, E, _p(offsets), seg_align, rac_ld, _p(rho),
                                        _p(w_sel), epilogue, _p(row_token), _p(row_gate), _p(out), ld_out,
                                        _p(amax_out), _p(dev_status), _stream(out.device)))
    return out


def bf16_grouped_gemm(a, m_pad_max, b, N, K, E, offsets, *, seg_align=128, epilogue=EPI_STORE_F32,
                      row_token=None, row_gate=None, out=None, ld_out=None, amax_out=None, dev_status=None):
    """moe_bf16_grouped_gemm (see the header): bf16 A [m_pad_max x lda] in
    routed order times bf16 B [E x N x K]."""
    lib = _lib.load()
    assert a.dtype == BF16 and b.dtype == BF16 and b.is_contiguous()
    if ld_out is None:
        ld_out = out.stride(0)
    check(lib.moe_bf16_grouped_gemm(_p(a), a.stride(0), m_pad_max, _p(b), N, K, E, _p(offsets), seg_align, epilogue,
                                    _p(row_token), _p(row_gate), _p(out), ld_out, _p(amax_out), _p(dev_status),
                                    _stream(out.device)))
    return out


def gather_rows_bf16(x: torch.Tensor, dst_rows: torch.Tensor, m_out: int, *, out=None):
    """moe_gather_rows_bf16: token rows of x to their routed rows (dst_rows
    int32 [T x fanout]); rows of `out` not named are left as they are."""
    lib = _lib.load()
    assert x.dtype == BF16 and x.dim() == 2 and dst_rows.dtype == I32
    T, K = x.shape
    if out is None:
        out = torch.zeros(m_out, K, dtype=BF16, device=x.device)
    check(lib.moe_gather_rows_bf16(_p(x), T, K, x.stride(0), _p(dst_rows), dst_rows.shape[1], _p(out), out.stride(0),
                                   m_out, _stream(x.device)))
    return out


def routed_rows_bf16(x: torch.Tensor, row_token: torch.Tensor, m_out: int, *, out=None):
    """moe_routed_rows_bf16: out[r] = x[row_token[r]], zero rows for padding."""
    lib = _lib.load()
    assert x.dtype == BF16 and x.dim() == 2 and x.stride(1) == 1
    T, K = x.shape
    if out is None:
        out = torch.empty(m_out, K, dtype=BF16, device=x.device)
    check(lib.moe_routed_rows_bf16(_p(x), T, K, x.stride(0), _p(row_token), _p(out), out.stride(0), m_out,
                                   _stream(x.device)))
    return out


def rac_residual_nvfp4(x: torch.Tensor, q: "Quantized", rac_k: int, rac_ld: int, *, dst_rows=None, fanout=1,
                       m_out=None, m_valid=None, s_r_out=None):
    """nvfp4_rac_residual_nvfp4: replace q.r_sel by the second-pass NVFP4
    residual operand of the channels q.sel (see the header)."""
    lib = _lib.load()
    M, K = x.shape
    if m_out is None:
        m_out = M
    ws = _ws(lib.nvfp4_rac_residual_nvfp4_workspace_size(), x.device)
    check(lib.nvfp4_rac_residual_nvfp4(_p(x), M, K, x.stride(0), _p(m_valid), _p(q.s_t), _p(q.sel), rac_k, rac_ld,
                                       _p(dst_rows), fanout, m_out, _p(q.r_sel), _p(s_r_out), _p(ws), ws.numel(),
                                       _stream(x.device)))
    return q


def fp8_quantize(x: torch.Tensor, *, s: torch.Tensor | None = None, amax: torch.Tensor | None = None,
                 dst_rows: torch.Tensor | None = None, fanout: int = 1, m_out: int | None = None,
                 codes: torch.Tensor | None = None, s_out: torch.Tensor | None = None):
    """fp8_quantize (see the header) on bf16 [M, K] or [G, M, K]: per-tensor
    E4M3 codes (sign in bit 7).  Returns (codes uint8, s float32 [G])."""
    lib = _lib.load()
    assert x.dtype == BF16 and x.stride(-1) == 1
    x3 = x.unsqueeze(0) if x.dim() == 2 else x
    G, M, K = x3.shape
    assert G == 1 or x3.is_contiguous()
    dev = x.device
    if m_out is None:
        m_out = M
    if codes is None:
        codes = torch.empty((G, m_out, K) if x.dim() == 3 else (m_out, K), dtype=U8, device=dev)
    if s_out is None:
        s_out = torch.empty(G, dtype=F32, device=dev)
    ws = _ws(lib.fp8_quantize_workspace_size(G), dev)
    check(lib.fp8_quantize(_p(x3), G, M, K, x3.stride(1), _p(s), _p(amax), _p(s_out), _p(dst_rows), fanout, m_out,
                           _p(codes), _p(ws), ws.numel(), _stream(dev)))
    return codes, s_out


def w8a8_grouped_gemm(a_codes, a_s, m_pad_max, b_codes, b_s, N, K, E, offsets, *, seg_align=128,
                      epilogue=EPI_STORE_F32, row_token=None, row_gate=None, out=None, ld_out=None, amax_out=None,
                      dev_status=None):
    """moe_w8a8_grouped_gemm (see the header): E4M3 A [m_pad_max x K] in
    routed order times E4M3 B [E x N x K] with per-tensor scales."""
    lib = _lib.load()
    if ld_out is None:
        ld_out = out.stride(0)
    check(lib.moe_w8a8_grouped_gemm(_p(a_codes), _p(a_s), m_pad_max, _p(b_codes), _p(b_s), N, K, E, _p(offsets),
                                    seg_align, epilogue, _p(row_token), _p(row_gate), _p(out), ld_out,
                                    _p(amax_out), _p(dev_status), _stream(out.device)))
    return out


@dataclasses.dataclass(slots=True)
class Act8:
    """Activations kept in 8 bits (act8_quantize): value = e4m3(code) *
    2^(scale - 127), one scale per 32 columns of a row."""
    codes: torch.Tensor          # uint8 [M, K], row stride a multiple of 16
    scales: torch.Tensor         # uint8 [M, 4 * ceil(K / 128)]

    def get_device(self) -> int:
        return self.codes.get_device()


# The experts' training and decode operators.  Their short calls last a few
# microseconds on the device, so the checks below are written to cost little.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_empty = torch.empty


def _on_device(fn):
    """Refuse host tensors; run with the first argument's device current (the
    library launches on the current device)."""
    @functools.wraps(fn)
    def call(x, *args, **kwargs):
        i = x.get_device()
        if i < 0:
            raise ValueError("the NVFP4 kernels run on CUDA tensors only (got a tensor on cpu); there is no CPU path")
        if i != _current_device():
            with torch.cuda.device(i):
                return fn(x, *args, **kwargs)
        return fn(x, *args, **kwargs)
    return call


def _matrix(t, name, dtype, rows, cols, index):
    """Row stride of a [rows, cols] tensor (rows None: any) of `dtype` on
    device `index` with contiguous columns; a single row has none: its width
    rounded up to 16."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not dtype or len(shape) != 2 or shape[1] != cols or (rows is not None and shape[0] != rows):
        raise ValueError(f"{name}: need {dtype} [{'rows' if rows is None else rows}, {cols}], got {t.dtype} {tuple(shape)}")
    if stride[1] != 1 and cols > 1:
        raise ValueError(f"{name}: columns must be contiguous")
    if t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{index}")
    return stride[0] if shape[0] > 1 else -(-cols // 16) * 16


def _vector(t, name, dtype, n, index):
    """Address of n contiguous elements."""
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name}: need contiguous {dtype} with {n} elements, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{index}")
    return t.data_ptr()


def _act8(a: Act8, name, rows, cols, index):
    """(row stride of the codes, of the scales)."""
    ldc = _matrix(a.codes, name + ".codes", U8, rows, cols, index)
    s = a.scales
    shape, stride = s.shape, s.stride()
    if s.dtype is not U8 or len(shape) != 2 or shape[0] != a.codes.shape[0] or shape[1] < -(-cols // 128) * 4 \
            or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name}.scales: need uint8 [{a.codes.shape[0]}, {-(-cols // 128) * 4}], got {s.dtype} "
                         f"{tuple(shape)}")
    if s.get_device() != index:
        raise ValueError(f"{name}.scales: on {s.device}, expected cuda:{index}")
    return ldc, stride[0] if shape[0] > 1 else -(-cols // 128) * 4


def _act8_empty(M, K, device):
    ld = -(-K // 16) * 16
    codes = _empty(M, ld, dtype=U8, device=device)
    return Act8(codes if ld == K else codes[:, :K], _empty(M, -(-K // 128) * 4, dtype=U8, device=device))


@_on_device
def ragged_gemm(a: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, *, transpose: bool = False,
                out: torch.Tensor | None = None, out_dtype: torch.dtype = BF16, dev_status=None):
    """moe_ragged_gemm (see the header): row r of expert e (offsets[e] <= r <
    offsets[e+1]) times w[e]^T, or times w[e] with transpose (the input
    gradient).  a bf16 [M, K] (transpose: [M, N]), w bf16 [E, N, K].  Rows
    outside the segments are not written: pass `out` to keep what they hold
    (without it they are uninitialized)."""
    lib = _lib.load()
    i = a.get_device()
    if w.dim() != 3 or w.dtype is not BF16 or not w.is_contiguous() or w.get_device() != i:
        raise ValueError("ragged_gemm: w must be contiguous bf16 [E, N, K] on a's device")
    E, N, K = w.shape
    width = K if transpose else N
    lda = _matrix(a, "ragged_gemm: a", BF16, None, N if transpose else K, i)
    M = a.shape[0]
    if out is None:
        if out_dtype not in (BF16, F32):
            raise ValueError("ragged_gemm: out_dtype must be bfloat16 or float32")
        out = _empty(M, width, dtype=out_dtype, device=a.device)
    f32 = out.dtype is F32
    ldo = _matrix(out, "ragged_gemm: out", F32 if f32 else BF16, M, width, i)
    check(lib.moe_ragged_gemm(a.data_ptr(), lda, M, w.data_ptr(), N, K, E,
                              _vector(offsets, "ragged_gemm: offsets", I32, E + 1, i), transpose, out.data_ptr(), ldo,
                              f32, _p(dev_status), _raw_stream(i)))
    return out


@_on_device
def ragged_wgrad(g: torch.Tensor, a, offsets: torch.Tensor, *, a_rows: torch.Tensor | None = None,
                 out: torch.Tensor | None = None, out_dtype: torch.dtype = F32, accumulate: bool = False,
                 dev_status=None):
    """moe_ragged_wgrad (see the header): dw[e] = sum over the expert's rows of
    g[r]^T a[r].  g bf16 [M, N]; a bf16 [M, K], or an Act8 [T, K] whose row
    a_rows[r] (int32 [M]; without it row r) belongs to row r.  accumulate adds
    to `out`."""
    lib = _lib.load()
    i = g.get_device()
    if g.dim() != 2:
        raise ValueError("ragged_wgrad: g must be bf16 [M, N]")
    M, N = g.shape
    ldg = _matrix(g, "ragged_wgrad: g", BF16, M, N, i)
    E = offsets.numel() - 1
    off = _vector(offsets, "ragged_wgrad: offsets", I32, E + 1, i)
    kept = isinstance(a, Act8)
    if kept:
        T, K = a.codes.shape
        lda, lds = _act8(a, "ragged_wgrad: a", T if a_rows is not None else M, K, i)
        data, scales = a.codes.data_ptr(), a.scales.data_ptr()
    else:
        T, K = M, a.shape[-1]
        lda, lds = _matrix(a, "ragged_wgrad: a", BF16, M, K, i), 0
        data, scales = a.data_ptr(), None
    rows = None if a_rows is None else _vector(a_rows, "ragged_wgrad: a_rows", I32, M, i)
    if out is None:
        if accumulate:
            raise ValueError("ragged_wgrad: accumulate needs out")
        if out_dtype not in (BF16, F32):
            raise ValueError("ragged_wgrad: out_dtype must be bfloat16 or float32")
        out = _empty(E, N, K, dtype=out_dtype, device=g.device)
    elif out.dtype not in (BF16, F32) or out.shape != (E, N, K) or not out.is_contiguous() or out.get_device() != i:
        raise ValueError(f"ragged_wgrad: out must be contiguous bf16 or f32 [{E}, {N}, {K}] on g's device")
    need = lib.moe_ragged_wgrad_workspace_size(M, N, K, E, kept)
    ws = _empty(need, dtype=U8, device=g.device) if need else None
    check(lib.moe_ragged_wgrad(g.data_ptr(), ldg, M, data, lda, scales, lds, rows, T, N, K, E, off, out.data_ptr(),
                               out.dtype is F32, accumulate, _p(ws), need, _p(dev_status), _raw_stream(i)))
    return out


@_on_device
def act8_quantize(x: torch.Tensor, *, out: Act8 | None = None) -> Act8:
    """act8_quantize (see the header): bf16 [M, K] kept in 8 bits."""
    lib = _lib.load()
    i = x.get_device()
    if x.dim() != 2:
        raise ValueError("act8_quantize: x must be bf16 [M, K]")
    M, K = x.shape
    ldx = _matrix(x, "act8_quantize: x", BF16, M, K, i)
    if out is None:
        out = _act8_empty(M, K, x.device)
    ldc, lds = _act8(out, "act8_quantize: out", M, K, i)
    check(lib.act8_quantize(x.data_ptr(), M, K, ldx, out.codes.data_ptr(), ldc, out.scales.data_ptr(), lds,
                            _raw_stream(i)))
    return out


@_on_device
def act8_dequantize(a: Act8, *, out: torch.Tensor | None = None) -> torch.Tensor:
    """act8_dequantize: the kept values as bf16 [M, K] (exact)."""
    lib = _lib.load()
    i = a.get_device()
    M, K = a.codes.shape
    ldc, lds = _act8(a, "act8_dequantize: a", M, K, i)
    if out is None:
        out = _empty(M, -(-K // 8) * 8, dtype=BF16, device=a.codes.device)[:, :K]
    ldx = _matrix(out, "act8_dequantize: out", BF16, M, K, i)
    check(lib.act8_dequantize(a.codes.data_ptr(), ldc, a.scales.data_ptr(), lds, M, K, out.data_ptr(), ldx,
                              _raw_stream(i)))
    return out


@_on_device
def swiglu_act8(y: torch.Tensor, *, h: torch.Tensor | None = None, out: Act8 | None = None):
    """moe_swiglu_act8 (see the header): (h = silu(gate) * up, y kept in 8
    bits) of y = [gate | up], bf16 [M, 2I]."""
    lib = _lib.load()
    i = y.get_device()
    if y.dim() != 2 or y.shape[1] % 2:
        raise ValueError("swiglu_act8: y must be bf16 [M, 2I]")
    M, K = y.shape
    I = K // 2
    ldy = _matrix(y, "swiglu_act8: y", BF16, M, K, i)
    if h is None:
        h = _empty(M, I, dtype=BF16, device=y.device)
    if out is None:
        out = _act8_empty(M, K, y.device)
    ldh = _matrix(h, "swiglu_act8: h", BF16, M, I, i)
    ldc, lds = _act8(out, "swiglu_act8: out", M, K, i)
    check(lib.moe_swiglu_act8(y.data_ptr(), M, I, ldy, h.data_ptr(), ldh, out.codes.data_ptr(), ldc,
                              out.scales.data_ptr(), lds, _raw_stream(i)))
    return h, out


@_on_device
def swiglu_act8_backward(y: Act8, dh: torch.Tensor, *, row_gate: torch.Tensor | None = None,
                         dy: torch.Tensor | None = None, gh: torch.Tensor | None = None,
                         dgate: torch.Tensor | None = None):
    """moe_swiglu_act8_backward (see the header): (dy [M, 2I], gate-weighted h
    [M, I], dgate f32 [M]) from the kept y and the gradient dh bf16 [M, I] of
    the unweighted h."""
    lib = _lib.load()
    i = y.get_device()
    if dh.dim() != 2:
        raise ValueError("swiglu_act8_backward: dh must be bf16 [M, I]")
    M, I = dh.shape
    lddh = _matrix(dh, "swiglu_act8_backward: dh", BF16, M, I, i)
    ldc, lds = _act8(y, "swiglu_act8_backward: y", M, 2 * I, i)
    gate = None if row_gate is None else _vector(row_gate, "swiglu_act8_backward: row_gate", F32, M, i)
    dev = dh.device
    if dy is None:
        dy = _empty(M, 2 * I, dtype=BF16, device=dev)
    if gh is None:
        gh = _empty(M, I, dtype=BF16, device=dev)
    if dgate is None:
        dgate = _empty(M, dtype=F32, device=dev)
    lddy = _matrix(dy, "swiglu_act8_backward: dy", BF16, M, 2 * I, i)
    ldgh = _matrix(gh, "swiglu_act8_backward: gh", BF16, M, I, i)
    check(lib.moe_swiglu_act8_backward(y.codes.data_ptr(), ldc, y.scales.data_ptr(), lds, dh.data_ptr(), lddh, gate, M,
                                       I, dy.data_ptr(), lddy, gh.data_ptr(), ldgh,
                                       _vector(dgate, "swiglu_act8_backward: dgate", F32, M, i), _raw_stream(i)))
    return dy, gh, dgate


@_on_device
def combine_rows(rows: torch.Tensor, dst_row: torch.Tensor, *, gate: torch.Tensor | None = None,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """moe_combine_rows: out[t] = sum_j gate[t, j] rows[dst_row[t, j]] (f32,
    slot order); rows bf16 [M, H], dst_row int32 [T, k_r]."""
    lib = _lib.load()
    i = rows.get_device()
    if rows.dim() != 2 or dst_row.dim() != 2:
        raise ValueError("combine_rows: rows must be bf16 [M, H], dst_row int32 [T, k_r]")
    M, H = rows.shape
    T, kr = dst_row.shape
    ldr = _matrix(rows, "combine_rows: rows", BF16, M, H, i)
    if out is None:
        out = _empty(T, H, dtype=F32, device=rows.device)
    ldo = _matrix(out, "combine_rows: out", F32, T, H, i)
    check(lib.moe_combine_rows(rows.data_ptr(), M, H, ldr, _vector(dst_row, "combine_rows: dst_row", I32, T * kr, i),
                               None if gate is None else _vector(gate, "combine_rows: gate", F32, T * kr, i), T, kr,
                               out.data_ptr(), ldo, _raw_stream(i)))
    return out


@_on_device
def route_backward(topk_idx: torch.Tensor, topk_gate: torch.Tensor, dst_row: torch.Tensor, dgate_row: torch.Tensor,
                   E: int, *, out: torch.Tensor | None = None) -> torch.Tensor:
    """moe_route_backward: the router logits' gradient f32 [T, E] from the
    routed rows' gate gradients dgate_row f32 [M]."""
    lib = _lib.load()
    i = topk_idx.get_device()
    if topk_idx.dim() != 2 or dgate_row.dim() != 1:
        raise ValueError("route_backward: topk_idx must be int32 [T, k_r], dgate_row float32 [M]")
    T, kr = topk_idx.shape
    M = dgate_row.numel()
    if out is None:
        out = _empty(T, E, dtype=F32, device=topk_idx.device)
    elif out.dtype is not F32 or out.shape != (T, E) or not out.is_contiguous() or out.get_device() != i:
        raise ValueError(f"route_backward: out must be contiguous float32 [{T}, {E}]")
    check(lib.moe_route_backward(_vector(topk_idx, "route_backward: topk_idx", I32, T * kr, i),
                                 _vector(topk_gate, "route_backward: topk_gate", F32, T * kr, i),
                                 _vector(dst_row, "route_backward: dst_row", I32, T * kr, i),
                                 _vector(dgate_row, "route_backward: dgate_row", F32, M, i), M, T, E, kr,
                                 out.data_ptr(), _raw_stream(i)))
    return out


@_on_device
def nvfp4_gemv(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, s_t: torch.Tensor, N: int, K: int, *,
               expert_idx: torch.Tensor | None = None, epilogue: int = EPI_STORE_F32,
               gate: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """moe_nvfp4_gemv (see the header): a few tokens' bf16 activations times
    NVFP4 weights (codes uint8 [E, N, K/2], scales, s_t as qdq_weights returns
    them).  expert_idx int32 [T, k_r] names each token's experts; None: one
    dense weight.  x has one row per token (EPI_COMBINE_F32: per token and
    slot, with the router weights `gate` f32 [T, k_r])."""
    lib = _lib.load()
    i = x.get_device()
    ldx = _matrix(x, "nvfp4_gemv: x", BF16, None, K, i)
    rows = x.shape[0]
    E = s_t.numel()
    if codes.dtype is not U8 or not codes.is_contiguous() or codes.numel() * 2 != E * N * K or codes.get_device() != i:
        raise ValueError(f"nvfp4_gemv: codes must be contiguous uint8 [{E}, {N}, {K // 2}] on x's device")
    if scales.dtype is not U8 or not scales.is_contiguous() or scales.numel() < E * scale_bytes(N, K) \
            or scales.get_device() != i:
        raise ValueError(f"nvfp4_gemv: scales must be contiguous uint8 with {E * scale_bytes(N, K)} bytes on x's device")
    combine = epilogue == EPI_COMBINE_F32
    if expert_idx is None:
        T, kr, idx = rows, 1, None
    else:
        if expert_idx.dim() != 2:
            raise ValueError("nvfp4_gemv: expert_idx must be int32 [T, k_r]")
        T, kr = expert_idx.shape
        idx = _vector(expert_idx, "nvfp4_gemv: expert_idx", I32, T * kr, i)
        if rows != (T * kr if combine else T):
            raise ValueError(f"nvfp4_gemv: x has {rows} rows for {T} tokens with {kr} experts each")
    if gate is not None:
        if not combine:
            raise ValueError("nvfp4_gemv: gate goes with EPI_COMBINE_F32")
        gate = _vector(gate, "nvfp4_gemv: gate", F32, T * kr, i)
    swiglu = epilogue == EPI_SWIGLU_BF16
    dtype, width = (BF16, N // 2) if swiglu else (F32, N)
    orows = T if combine else T * kr
    if out is None:
        out = _empty(orows, width, dtype=dtype, device=x.device)
    ldo = _matrix(out, "nvfp4_gemv: out", dtype, orows, width, i)
    need = lib.moe_nvfp4_gemv_workspace_size(T, N, E, kr, epilogue) if combine else 0
    ws = _empty(need, dtype=U8, device=x.device) if need else None
    check(lib.moe_nvfp4_gemv(x.data_ptr(), T, ldx, codes.data_ptr(), scales.data_ptr(),
                             _vector(s_t, "nvfp4_gemv: s_t", F32, E, i), N, K, E, idx, kr, epilogue, gate,
                             out.data_ptr(), ldo, _p(ws), need, _raw_stream(i)))
    return out


def debug_encode(v: torch.Tensor):
    """nvfp4_debug_encode: (E2M1 codes, E4M3 codes) of float32 values."""
    lib = _lib.load()
    assert v.dtype == F32 and v.is_contiguous()
    e2 = torch.empty(v.shape, dtype=U8, device=v.device)
    e4 = torch.empty(v.shape, dtype=U8, device=v.device)
    check(lib.nvfp4_debug_encode(_p(v), v.numel(), _p(e2), _p(e4), _stream(v.device)))
    return e2, e4


def read_status(dev_status: torch.Tensor) -> int:
    lib = _lib.load()
    import ctypes
    out = ctypes.c_int32(0)
    check(lib.nvfp4_read_status(_p(dev_status), ctypes.addressof(out), _stream(dev_status.device)))
    return int(out.value)
