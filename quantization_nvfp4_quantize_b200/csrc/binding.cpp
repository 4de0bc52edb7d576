// binding.cpp -- the compiled half of the Python binding for the experts'
// training and decode operators: checks the tensors, allocates outputs and
// workspaces with torch, and calls the C ABI on the current stream.
//
// Their short calls last a few microseconds on the device; marshalled from
// Python (argument checks, torch.empty, ctypes) a call took 8 to 16 us of host
// time, from here 4 to 6.  It links to no CUDA code: bind() receives the
// addresses of the C entry points from the loader of libnvfp4_quads.so.
//
// Errors: std::invalid_argument becomes ValueError; a status other than 0 goes
// to the loader's check function, which raises.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "../../include/nvfp4_quads.h"

namespace {

using at::ScalarType;
using at::Tensor;

constexpr ScalarType BF16 = at::kBFloat16, F32 = at::kFloat, I32 = at::kInt, U8 = at::kByte;

// C entry points, filled by bind() in this order.
struct Entry {
    const char *name;
    void *fn;
};
Entry entries[] = {{"moe_ragged_gemm", nullptr}, {"moe_ragged_wgrad_workspace_size", nullptr},
                   {"moe_ragged_wgrad", nullptr}, {"act8_quantize", nullptr}, {"act8_dequantize", nullptr},
                   {"moe_swiglu_act8", nullptr}, {"moe_swiglu_act8_backward", nullptr}, {"moe_combine_rows", nullptr},
                   {"moe_route_backward", nullptr}, {"moe_nvfp4_gemv_workspace_size", nullptr},
                   {"moe_nvfp4_gemv", nullptr}};
enum { GEMM, WGRAD_WS, WGRAD, QUANT, DEQUANT, SWIGLU, SWIGLU_BACK, COMBINE, ROUTE_BACK, GEMV_WS, GEMV, COUNT };
PyObject *check_fn = nullptr;

#define ENTRY(which, name) reinterpret_cast<decltype(&::name)>(entries[which].fn)

struct PythonError {};                   // a Python exception is set

[[noreturn]] void refuse(const std::string &what) { throw std::invalid_argument(what); }

std::string shape_of(const Tensor &t)
{
    std::string s = std::string(c10::toString(t.scalar_type())) + " [";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "]";
}

bool none(PyObject *o) { return o == Py_None; }

const Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) refuse(std::string(name) + ": need a tensor");
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject *o)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    return v;
}

bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonError();
    return v == 1;
}

ScalarType dtype(PyObject *o, const char *name)
{
    const ScalarType t = THPDtype_Check(o) ? reinterpret_cast<THPDtype *>(o)->scalar_type : ScalarType::Undefined;
    if (t != BF16 && t != F32) refuse(std::string(name) + " must be bfloat16 or float32");
    return t;
}

// One call: every tensor lives on the first one's device.
struct Call {
    c10::Device dev;
    explicit Call(const Tensor &first) : dev(first.device()) {}

    void same_device(const Tensor &t, const char *name) const
    {
        if (t.device() != dev) refuse(std::string(name) + ": on " + t.device().str() + ", expected " + dev.str());
    }

    // Row stride of a [rows, cols] tensor (rows < 0: any) with contiguous
    // columns; a single row has none: its width rounded up to 16.
    int64_t matrix(const Tensor &t, const char *name, ScalarType type, int64_t rows, int64_t cols) const
    {
        if (t.scalar_type() != type || t.dim() != 2 || t.size(1) != cols || (rows >= 0 && t.size(0) != rows))
            refuse(std::string(name) + ": need " + c10::toString(type) + " [" +
                   (rows < 0 ? std::string("rows") : std::to_string(rows)) + ", " + std::to_string(cols) + "], got " +
                   shape_of(t));
        if (t.stride(1) != 1 && cols > 1) refuse(std::string(name) + ": columns must be contiguous");
        same_device(t, name);
        return t.size(0) > 1 ? t.stride(0) : (cols + 15) / 16 * 16;
    }

    // n contiguous elements.
    template <typename T>
    T *vector(const Tensor &t, const char *name, ScalarType type, int64_t n) const
    {
        if (t.scalar_type() != type || t.numel() != n || !t.is_contiguous())
            refuse(std::string(name) + ": need contiguous " + c10::toString(type) + " with " + std::to_string(n) +
                   " elements, got " + shape_of(t));
        same_device(t, name);
        return static_cast<T *>(t.data_ptr());
    }

    // Row stride of the scales of a kept [rows, cols] tensor.
    int64_t scales(const Tensor &t, const char *name, int64_t rows, int64_t cols) const
    {
        const int64_t need = (cols + 127) / 128 * 4;
        if (t.scalar_type() != U8 || t.dim() != 2 || t.size(0) != rows || t.size(1) < need ||
            (t.stride(1) != 1 && t.size(1) > 1))
            refuse(std::string(name) + ": need Byte [" + std::to_string(rows) + ", " + std::to_string(need) + "], got " +
                   shape_of(t));
        same_device(t, name);
        return rows > 1 ? t.stride(0) : need;
    }

    void on_gpu() const
    {
        if (!dev.is_cuda())
            refuse("the NVFP4 kernels run on CUDA tensors only (got a tensor on " + dev.str() + "); there is no CPU path");
    }

    Tensor empty(at::IntArrayRef size, ScalarType type) const
    {
        return at::detail::empty_cuda(size, type, dev, c10::nullopt);
    }

    // [rows, cols] on a row stride that is a multiple of `unit` elements
    Tensor padded(int64_t rows, int64_t cols, int64_t unit, ScalarType type) const
    {
        const int64_t ld = (cols + unit - 1) / unit * unit;
        Tensor t = empty({rows, ld}, type);
        return ld == cols ? t : t.narrow(1, 0, cols);
    }

    void *stream() const { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }
};

void check(nvfp4_status status)
{
    if (status == NVFP4_OK) return;
    PyObject *r = PyObject_CallFunction(check_fn, "i", (int)status);      // raises
    Py_XDECREF(r);
    throw PythonError();
}

int32_t *status_word(PyObject *o, const Call &c)
{
    return none(o) ? nullptr : c.vector<int32_t>(tensor(o, "dev_status"), "dev_status", I32, tensor(o, "dev_status").numel());
}

// (a, w, offsets, transpose, out, out_dtype, dev_status) -> out
PyObject *ragged_gemm(PyObject *const *v)
{
    const Tensor &a = tensor(v[0], "ragged_gemm: a"), &w = tensor(v[1], "ragged_gemm: w"),
                 &offsets = tensor(v[2], "ragged_gemm: offsets");
    const bool transpose = truth(v[3]);
    const Call c(a);
    if (w.dim() != 3 || w.scalar_type() != BF16 || !w.is_contiguous())
        refuse("ragged_gemm: w must be contiguous bf16 [E, N, K]");
    c.same_device(w, "ragged_gemm: w");
    const int64_t E = w.size(0), N = w.size(1), K = w.size(2), width = transpose ? K : N;
    const int64_t lda = c.matrix(a, "ragged_gemm: a", BF16, -1, transpose ? N : K), M = a.size(0);
    const int32_t *off = c.vector<int32_t>(offsets, "ragged_gemm: offsets", I32, E + 1);
    ScalarType type = dtype(v[5], "ragged_gemm: out_dtype");
    Tensor out;
    if (!none(v[4])) {
        out = tensor(v[4], "ragged_gemm: out");
        type = out.scalar_type() == F32 ? F32 : BF16;
        c.matrix(out, "ragged_gemm: out", type, M, width);
    }
    c.on_gpu();
    const c10::cuda::CUDAGuard guard(c.dev);
    if (none(v[4])) out = c.empty({M, width}, type);
    check(ENTRY(GEMM, moe_ragged_gemm)(a.data_ptr(), lda, M, w.data_ptr(), N, K, (int32_t)E, off, transpose, out.data_ptr(),
                                       c.matrix(out, "ragged_gemm: out", type, M, width), type == F32,
                                       status_word(v[6], c), c.stream()));
    return THPVariable_Wrap(out);
}

// (g, a or codes, scales or None, offsets, a_rows, out, out_dtype, accumulate, dev_status) -> out
PyObject *ragged_wgrad(PyObject *const *v)
{
    const Tensor &g = tensor(v[0], "ragged_wgrad: g"), &a = tensor(v[1], "ragged_wgrad: a"),
                 &offsets = tensor(v[3], "ragged_wgrad: offsets");
    const Call c(g);
    if (g.dim() != 2 || a.dim() != 2) refuse("ragged_wgrad: g and a must be [M, N] and [M, K]");
    const int64_t M = g.size(0), N = g.size(1), K = a.size(1), E = offsets.numel() - 1;
    if (E < 1) refuse("ragged_wgrad: offsets: need Int with E + 1 elements, got " + shape_of(offsets));
    const int64_t ldg = c.matrix(g, "ragged_wgrad: g", BF16, M, N);
    const int32_t *off = c.vector<int32_t>(offsets, "ragged_wgrad: offsets", I32, E + 1);
    const bool kept = !none(v[2]);
    const int32_t *rows = none(v[4]) ? nullptr : c.vector<int32_t>(tensor(v[4], "ragged_wgrad: a_rows"),
                                                                    "ragged_wgrad: a_rows", I32, M);
    int64_t T = M, lda, lds = 0;
    const uint8_t *scales = nullptr;
    if (kept) {
        if (rows) T = a.size(0);
        lda = c.matrix(a, "ragged_wgrad: a.codes", U8, T, K);
        lds = c.scales(tensor(v[2], "ragged_wgrad: a.scales"), "ragged_wgrad: a.scales", T, K);
        scales = static_cast<const uint8_t *>(tensor(v[2], "ragged_wgrad: a.scales").data_ptr());
    } else {
        lda = c.matrix(a, "ragged_wgrad: a", BF16, M, K);
    }
    const bool accumulate = truth(v[7]);
    ScalarType type = dtype(v[6], "ragged_wgrad: out_dtype");
    Tensor out;
    if (!none(v[5])) {
        out = tensor(v[5], "ragged_wgrad: out");
        type = out.scalar_type();
        if ((type != BF16 && type != F32) || out.dim() != 3 || out.size(0) != E || out.size(1) != N || out.size(2) != K ||
            !out.is_contiguous())
            refuse("ragged_wgrad: out must be contiguous bf16 or f32 [" + std::to_string(E) + ", " + std::to_string(N) +
                   ", " + std::to_string(K) + "], got " + shape_of(out));
        c.same_device(out, "ragged_wgrad: out");
    } else if (accumulate) {
        refuse("ragged_wgrad: accumulate needs out");
    }
    c.on_gpu();
    const c10::cuda::CUDAGuard guard(c.dev);
    if (none(v[5])) out = c.empty({E, N, K}, type);
    const size_t need = ENTRY(WGRAD_WS, moe_ragged_wgrad_workspace_size)(M, N, K, (int32_t)E, kept ? rows ? 2 : 1 : 0);
    Tensor ws;
    if (need) ws = c.empty({(int64_t)need}, U8);
    // a kept tensor without rows has no memory, but the library knows kept rows
    // by their scales: any address does, nothing is read through it
    if (kept && T == 0 && need) scales = static_cast<const uint8_t *>(ws.data_ptr());
    check(ENTRY(WGRAD, moe_ragged_wgrad)(g.data_ptr(), ldg, M, a.data_ptr(), lda, scales, lds, rows, T, N, K, (int32_t)E, off,
                                         out.data_ptr(), type == F32, accumulate, need ? ws.data_ptr() : nullptr, need,
                                         status_word(v[8], c), c.stream()));
    return THPVariable_Wrap(out);
}

PyObject *pair(const Tensor &a, const Tensor &b) { return Py_BuildValue("(NN)", THPVariable_Wrap(a), THPVariable_Wrap(b)); }

// (x, codes, scales) -> (codes, scales)
PyObject *act8_quantize(PyObject *const *v)
{
    const Tensor &x = tensor(v[0], "act8_quantize: x");
    const Call c(x);
    if (x.dim() != 2) refuse("act8_quantize: x must be bf16 [M, K]");
    const int64_t M = x.size(0), K = x.size(1), ldx = c.matrix(x, "act8_quantize: x", BF16, M, K);
    Tensor codes, scales;
    if (!none(v[1])) {
        codes = tensor(v[1], "act8_quantize: out.codes");
        scales = tensor(v[2], "act8_quantize: out.scales");
    }
    if (none(v[1])) {
        c.on_gpu();
        codes = c.padded(M, K, 16, U8);
        scales = c.empty({M, (K + 127) / 128 * 4}, U8);
    }
    const int64_t ldc = c.matrix(codes, "act8_quantize: out.codes", U8, M, K);
    const int64_t lds = c.scales(scales, "act8_quantize: out.scales", M, K);
    c.on_gpu();
    const c10::cuda::CUDAGuard guard(c.dev);
    check(ENTRY(QUANT, act8_quantize)(x.data_ptr(), M, K, ldx, (uint8_t *)codes.data_ptr(), ldc, (uint8_t *)scales.data_ptr(),
                                      lds, c.stream()));
    return pair(codes, scales);
}

// (codes, scales, out) -> out
PyObject *act8_dequantize(PyObject *const *v)
{
    const Tensor &codes = tensor(v[0], "act8_dequantize: a.codes"), &scales = tensor(v[1], "act8_dequantize: a.scales");
    const Call c(codes);
    if (codes.dim() != 2) refuse("act8_dequantize: a.codes must be uint8 [M, K]");
    const int64_t M = codes.size(0), K = codes.size(1);
    const int64_t ldc = c.matrix(codes, "act8_dequantize: a.codes", U8, M, K);
    const int64_t lds = c.scales(scales, "act8_dequantize: a.scales", M, K);
    Tensor out;
    if (!none(v[2])) out = tensor(v[2], "act8_dequantize: out");
    else {
        c.on_gpu();
        out = c.padded(M, K, 8, BF16);
    }
    const int64_t ldx = c.matrix(out, "act8_dequantize: out", BF16, M, K);
    c.on_gpu();
    const c10::cuda::CUDAGuard guard(c.dev);
    check(ENTRY(DEQUANT, act8_dequantize)((const uint8_t *)codes.data_ptr(), ldc, (const uint8_t *)scales.data_ptr(), lds, M,
                                          K, out.data_ptr(), ldx, c.stream()));
    return THPVariable_Wrap(out);
}

// (y, h, codes, scales) -> (h, codes, scales)
PyObject *swiglu_act8(PyObject *const *v)
{
    const Tensor &y = tensor(v[0], "swiglu_act8: y");
    const Call c(y);
    if (y.dim() != 2 || y.size(1) % 2) refuse("swiglu_act8: y must be bf16 [M, 2I]");
    const int64_t M = y.size(0), K = y.size(1), I = K / 2;
    const int64_t ldy = c.matrix(y, "swiglu_act8: y", BF16, M, K);
    Tensor h, codes, scales;
    if (!none(v[1])) h = tensor(v[1], "swiglu_act8: h");
    if (!none(v[2])) {
        codes = tensor(v[2], "swiglu_act8: out.codes");
        scales = tensor(v[3], "swiglu_act8: out.scales");
    }
    if (none(v[1]) || none(v[2])) c.on_gpu();
    if (none(v[1])) h = c.empty({M, I}, BF16);
    if (none(v[2])) {
        codes = c.padded(M, K, 16, U8);
        scales = c.empty({M, (K + 127) / 128 * 4}, U8);
    }
    const int64_t ldh = c.matrix(h, "swiglu_act8: h", BF16, M, I);
    const int64_t ldc = c.matrix(codes, "swiglu_act8: out.codes", U8, M, K);
    const int64_t lds = c.scales(scales, "swiglu_act8: out.scales", M, K);
    c.on_gpu();
    const c10::cuda::CUDAGuard guard(c.dev);
    check(ENTRY(SWIGLU, moe_swiglu_act8)(y.data_ptr(), M, I, ldy, h.data_ptr(), ldh, (uint8_t *)codes.data_ptr(), ldc,
                                         (uint8_t *)scales.data_ptr(), lds, c.stream()));
    return Py_BuildValue("(NNN)", THPVariable_Wrap(h), THPVariable_Wrap(codes), THPVariable_Wrap(scales));
}

// (codes, scales, dh, row_gate, dy, gh, dgate) -> (dy, gh, dgate)
PyObject *swiglu_act8_backward(PyObject *const *v)
{
    const Tensor &codes = tensor(v[0], "swiglu_act8_backward: y.codes"), &scales = tensor(v[1], "swiglu_act8_backward: y.scales"),
                 &dh = tensor(v[2], "swiglu_act8_backward: dh");
    const Call c(codes);
    if (dh.dim() != 2) refuse("swiglu_act8_backward: dh must be bf16 [M, I]");
    const int64_t M = dh.size(0), I = dh.size(1);
    const int64_t lddh = c.matrix(dh, "swiglu_act8_backward: dh", BF16, M, I);
    const int64_t ldc = c.matrix(codes, "swiglu_act8_backward: y.codes", U8, M, 2 * I);
    const int64_t lds = c.scales(scales, "swiglu_act8_backward: y.scales", M, 2 * I);
    const float *gate = none(v[3]) ? nullptr : c.vector<float>(tensor(v[3], "swiglu_act8_backward: row_gate"),
                                                                "swiglu_act8_backward: row_gate", F32, M);
    Tensor dy, gh, dgate;
    if (!none(v[4])) dy = tensor(v[4], "swiglu_act8_backward: dy");
    if (!none(v[5])) gh = tensor(v[5], "swiglu_act8_backward: gh");
    if (!none(v[6])) dgate = tensor(v[6], "swiglu_act8_backward: dgate");
    if (none(v[4]) || none(v[5]) || none(v[6])) c.on_gpu();
    if (none(v[4])) dy = c.empty({M, 2 * I}, BF16);
    if (none(v[5])) gh = c.empty({M, I}, BF16);
    if (none(v[6])) dgate = c.empty({M}, F32);
    const int64_t lddy = c.matrix(dy, "swiglu_act8_backward: dy", BF16, M, 2 * I);
    const int64_t ldgh = c.matrix(gh, "swiglu_act8_backward: gh", BF16, M, I);
    float *dg = c.vector<float>(dgate, "swiglu_act8_backward: dgate", F32, M);
    c.on_gpu();
    const c10::cuda::CUDAGuard guard(c.dev);
    check(ENTRY(SWIGLU_BACK, moe_swiglu_act8_backward)((const uint8_t *)codes.data_ptr(), ldc,
                                                       (const uint8_t *)scales.data_ptr(), lds, dh.data_ptr(), lddh, gate, M,
                                                       I, dy.data_ptr(), lddy, gh.data_ptr(), ldgh, dg, c.stream()));
    return Py_BuildValue("(NNN)", THPVariable_Wrap(dy), THPVariable_Wrap(gh), THPVariable_Wrap(dgate));
}

// (rows, dst_row, gate, out) -> out
PyObject *combine_rows(PyObject *const *v)
{
    const Tensor &rows = tensor(v[0], "combine_rows: rows"), &dst = tensor(v[1], "combine_rows: dst_row");
    const Call c(rows);
    if (rows.dim() != 2 || dst.dim() != 2) refuse("combine_rows: rows must be bf16 [M, H], dst_row int32 [T, k_r]");
    const int64_t M = rows.size(0), H = rows.size(1), T = dst.size(0), kr = dst.size(1);
    const int64_t ldr = c.matrix(rows, "combine_rows: rows", BF16, M, H);
    const int32_t *d = c.vector<int32_t>(dst, "combine_rows: dst_row", I32, T * kr);
    const float *gate = none(v[2]) ? nullptr : c.vector<float>(tensor(v[2], "combine_rows: gate"), "combine_rows: gate", F32,
                                                                T * kr);
    Tensor out;
    if (!none(v[3])) out = tensor(v[3], "combine_rows: out");
    else {
        c.on_gpu();
        out = c.empty({T, H}, F32);
    }
    const int64_t ldo = c.matrix(out, "combine_rows: out", F32, T, H);
    c.on_gpu();
    const c10::cuda::CUDAGuard guard(c.dev);
    check(ENTRY(COMBINE, moe_combine_rows)(rows.data_ptr(), M, H, ldr, d, gate, T, (int32_t)kr, (float *)out.data_ptr(), ldo,
                                           c.stream()));
    return THPVariable_Wrap(out);
}

// (topk_idx, topk_gate, dst_row, dgate_row, E, out) -> out
PyObject *route_backward(PyObject *const *v)
{
    const Tensor &idx = tensor(v[0], "route_backward: topk_idx"), &gate = tensor(v[1], "route_backward: topk_gate"),
                 &dst = tensor(v[2], "route_backward: dst_row"), &dgate = tensor(v[3], "route_backward: dgate_row");
    const Call c(idx);
    if (idx.dim() != 2 || dgate.dim() != 1)
        refuse("route_backward: topk_idx must be int32 [T, k_r], dgate_row float32 [M]");
    const int64_t T = idx.size(0), kr = idx.size(1), M = dgate.numel(), E = integer(v[4]);
    const int32_t *i = c.vector<int32_t>(idx, "route_backward: topk_idx", I32, T * kr);
    const float *g = c.vector<float>(gate, "route_backward: topk_gate", F32, T * kr);
    const int32_t *d = c.vector<int32_t>(dst, "route_backward: dst_row", I32, T * kr);
    const float *dg = c.vector<float>(dgate, "route_backward: dgate_row", F32, M);
    if (E < 1 || E > 65536) refuse("route_backward: need 1 <= E <= 65536");
    Tensor out;
    if (!none(v[5])) {
        out = tensor(v[5], "route_backward: out");
        if (out.dim() != 2 || out.size(0) != T || out.size(1) != E) refuse("route_backward: out must be float32 [T, E]");
    } else {
        c.on_gpu();
        out = c.empty({T, E}, F32);
    }
    float *o = c.vector<float>(out, "route_backward: out", F32, T * E);
    c.on_gpu();
    const c10::cuda::CUDAGuard guard(c.dev);
    check(ENTRY(ROUTE_BACK, moe_route_backward)(i, g, d, dg, M, T, (int32_t)E, (int32_t)kr, o, c.stream()));
    return THPVariable_Wrap(out);
}

// (x, codes, scales, s_t, N, K, expert_idx, epilogue, gate, out) -> out
PyObject *nvfp4_gemv(PyObject *const *v)
{
    const Tensor &x = tensor(v[0], "nvfp4_gemv: x"), &codes = tensor(v[1], "nvfp4_gemv: codes"),
                 &scales = tensor(v[2], "nvfp4_gemv: scales"), &s_t = tensor(v[3], "nvfp4_gemv: s_t");
    const int64_t N = integer(v[4]), K = integer(v[5]);
    const int32_t epilogue = (int32_t)integer(v[7]);
    const Call c(x);
    if (N < 1 || K < 1 || N >= (1ll << 31) || K >= (1ll << 31)) refuse("nvfp4_gemv: N and K must be positive");
    const int64_t ldx = c.matrix(x, "nvfp4_gemv: x", BF16, -1, K), rows = x.size(0), E = s_t.numel();
    const float *st = c.vector<float>(s_t, "nvfp4_gemv: s_t", F32, E);
    if (codes.scalar_type() != U8 || !codes.is_contiguous() || codes.numel() * 2 != E * N * K)
        refuse("nvfp4_gemv: codes must be contiguous uint8 [" + std::to_string(E) + ", " + std::to_string(N) + ", " +
               std::to_string(K / 2) + "], got " + shape_of(codes));
    c.same_device(codes, "nvfp4_gemv: codes");
    const int64_t need_scales = E * ((N + 127) / 128 * 128) * (K / 16);
    // one expert's scales follow another's: a longer buffer would be read at the wrong places
    if (scales.scalar_type() != U8 || !scales.is_contiguous() || scales.numel() < need_scales ||
        (E > 1 && scales.numel() != need_scales))
        refuse("nvfp4_gemv: scales must be contiguous uint8 with " + std::to_string(need_scales) + " bytes, got " +
               shape_of(scales));
    c.same_device(scales, "nvfp4_gemv: scales");
    const bool combine = epilogue == MOE_EPI_COMBINE_F32, swiglu = epilogue == MOE_EPI_SWIGLU_BF16;
    int64_t T = rows, kr = 1;
    const int32_t *idx = nullptr;
    if (!none(v[6])) {
        const Tensor &e = tensor(v[6], "nvfp4_gemv: expert_idx");
        if (e.dim() != 2) refuse("nvfp4_gemv: expert_idx must be int32 [T, k_r]");
        T = e.size(0);
        kr = e.size(1);
        idx = c.vector<int32_t>(e, "nvfp4_gemv: expert_idx", I32, T * kr);
        if (rows != (combine ? T * kr : T))
            refuse("nvfp4_gemv: x has " + std::to_string(rows) + " rows for " + std::to_string(T) + " tokens with " +
                   std::to_string(kr) + " experts each");
    }
    const float *gate = nullptr;
    if (!none(v[8])) {
        if (!combine) refuse("nvfp4_gemv: gate goes with EPI_COMBINE_F32");
        gate = c.vector<float>(tensor(v[8], "nvfp4_gemv: gate"), "nvfp4_gemv: gate", F32, T * kr);
    }
    const ScalarType type = swiglu ? BF16 : F32;
    const int64_t width = swiglu ? N / 2 : N, orows = combine ? T : T * kr;
    Tensor out;
    if (!none(v[9])) out = tensor(v[9], "nvfp4_gemv: out");
    else {
        c.on_gpu();
        out = c.empty({orows, width}, type);
    }
    const int64_t ldo = c.matrix(out, "nvfp4_gemv: out", type, orows, width);
    c.on_gpu();
    const c10::cuda::CUDAGuard guard(c.dev);
    const size_t need = combine ? ENTRY(GEMV_WS, moe_nvfp4_gemv_workspace_size)(T, N, (int32_t)E, (int32_t)kr, epilogue) : 0;
    Tensor ws;
    if (need) ws = c.empty({(int64_t)need}, U8);
    // an empty batch has no expert table to point to
    if (T == 0) return THPVariable_Wrap(out);
    check(ENTRY(GEMV, moe_nvfp4_gemv)(x.data_ptr(), T, ldx, (const uint8_t *)codes.data_ptr(),
                                      (const uint8_t *)scales.data_ptr(), st, N, K, (int32_t)E, idx, (int32_t)kr, epilogue,
                                      gate, out.data_ptr(), ldo, need ? ws.data_ptr() : nullptr, need, c.stream()));
    return THPVariable_Wrap(out);
}

// Argument count, exceptions.
template <PyObject *(*FN)(PyObject *const *), Py_ssize_t N>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    if (!check_fn) {
        PyErr_SetString(PyExc_RuntimeError, "the library's entry points are not bound");
        return nullptr;
    }
    try {
        return FN(args);
    } catch (const PythonError &) {
        return nullptr;
    } catch (const std::invalid_argument &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError &e) {
        PyObject *torch = PyImport_ImportModule("torch");
        PyObject *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type) PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// bind(check, {name: address})
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 2 || !PyCallable_Check(args[0]) || !PyDict_Check(args[1])) {
        PyErr_SetString(PyExc_TypeError, "bind(check, {name: address})");
        return nullptr;
    }
    for (Entry &e : entries) {
        PyObject *a = PyDict_GetItemString(args[1], e.name);
        void *p = a ? PyLong_AsVoidPtr(a) : nullptr;
        if (!p) {
            if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "no address for %s", e.name);
            return nullptr;
        }
        e.fn = p;
    }
    Py_INCREF(args[0]);
    Py_XSETREF(check_fn, args[0]);
    Py_RETURN_NONE;
}

#define METHOD(name, count) {#name, (PyCFunction)(void (*)(void))call<name, count>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
    METHOD(ragged_gemm, 7), METHOD(ragged_wgrad, 9), METHOD(act8_quantize, 3), METHOD(act8_dequantize, 3),
    METHOD(swiglu_act8, 4), METHOD(swiglu_act8_backward, 7), METHOD(combine_rows, 4), METHOD(route_backward, 6),
    METHOD(nvfp4_gemv, 10), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
