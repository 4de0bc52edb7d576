// act8.cu -- activations kept in 8 bits for the trainer's backward pass, the
// SwiGLU around them, and the two small operators that close the layer's
// backward pass (combine of routed rows, router gradient).
//
// Format: E4M3 codes, one scale byte s per 32 consecutive columns of a row,
// value = e4m3(code) * 2^(s - 127).  p = s - 127 is the smallest power with
// max|x| <= 448 * 2^p (p >= -120), so no value saturates; a power of two
// costs a floating 8-bit format no precision inside its range and makes every
// kept value exact in bf16 (4 significant bits, smallest step 2^-129), which
// lets the weight gradient feed it to bf16 tensor-core tiles unrounded.  One
// rounding per element: E4M3_rne(x * 2^-p), the product exact.  A group that
// holds an infinity or NaN gets s = 255 and NaN codes: all of it reads as
// NaN, so an overflow of the forward pass reaches the gradients.
//
// Every kernel here streams: one pass over the data, 16-byte loads and stores,
// a resident grid.  The floor is HBM; measured in a loop over inputs larger than
// L2: quantize 16384 x 4096 35 us (5.8 TB/s), expanding it again 36 us (5.7), SwiGLU
// keeping 32768 rows of 2 x 768 columns 36 us (5.6), its backward pass 47 us (5.3),
// the combine of 4096 tokens' 8 rows of 2048 31 us (5.4).  A single launch with a
// cold L2 takes 4 to 6 us more.  What is left is load latency and the encode: half
// of the issue slots and of the ALU pipe.
#include "common.cuh"

#include <algorithm>

namespace nvfp4 {
namespace act8 {

constexpr int THREADS = 256;
constexpr int QUANT_BLOCKS = 6, SWIGLU_BLOCKS = 5, DEQUANT_BLOCKS = 8, BACKWARD_BLOCKS = 4;     // resident per SM

// p + 127 of a group from the largest |x| (bf16 bits); 255 for Inf / NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits)
{
    if (amax_bits >= 0x7F80u) return 255u;
    if (amax_bits == 0u) return 127u;
    // amax = m * 2^e, m in [1, 2): 448 = 1.75 * 2^8, so p = e - 8, one more above 1.75
    const int p = (int)(amax_bits >> 7) - 127 - 8 + ((amax_bits & 0x7Fu) > 0x60u ? 1 : 0);
    return (uint32_t)(max(p, -120) + 127);
}

// 2^(127 - s) and 2^(s - 127) for s in [7, 247]
__device__ __forceinline__ float inv_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }
__device__ __forceinline__ float scale_of(uint32_t s)
{
    return s == 255u ? __uint_as_float(0x7FC00000u) : s == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(s << 23);
}

__device__ __forceinline__ uint32_t absmax2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }

// four floats -> four E4M3 codes (signed, nearest even)
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    return cvt_e4m3x2(a, b) | (cvt_e4m3x2(c, d) << 16);
}

// 16 bf16 (two 16-byte vectors) -> 16 codes, given the group's scale byte
__device__ __forceinline__ uint4 encode16(const uint32_t w[8], uint32_t s)
{
    if (s == 255u) return make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    const float inv = inv_scale(s);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = e4m3x4(__fmul_rn(bf16lo(w[2 * i]), inv), __fmul_rn(bf16hi(w[2 * i]), inv),
                      __fmul_rn(bf16lo(w[2 * i + 1]), inv), __fmul_rn(bf16hi(w[2 * i + 1]), inv));
    return make_uint4(c[0], c[1], c[2], c[3]);
}

// The group maximum: 16 columns per lane, two neighbouring lanes per group.
__device__ __forceinline__ uint32_t group_amax(const uint32_t w[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = absmax2(m, w[i]);
    uint32_t v = max(m & 0xFFFFu, m >> 16);
    return max(v, __shfl_xor_sync(0xffffffffu, v, 1));
}

// 16 columns from column c of a row of K; columns >= K read as 0.  Rows start
// on 16 bytes; the row may end inside the 16 columns.
__device__ __forceinline__ void load16(const __nv_bfloat16 *row, int64_t c, int64_t K, uint32_t w[8])
{
    if (c + 16 <= K) {
        const uint4 a = *reinterpret_cast<const uint4 *>(row + c);
        const uint4 b = *reinterpret_cast<const uint4 *>(row + c + 8);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t lo = 0, hi = 0;
            if (c + 2 * i < K) lo = __bfloat16_as_ushort(row[c + 2 * i]);
            if (c + 2 * i + 1 < K) hi = __bfloat16_as_ushort(row[c + 2 * i + 1]);
            w[i] = lo | (hi << 16);
        }
    }
}

__device__ __forceinline__ void store16(uint8_t *row, int64_t c, int64_t K, uint4 v)
{
    if (c + 16 <= K) {
        *reinterpret_cast<uint4 *>(row + c) = v;
    } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (c + i < K) row[c + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}

// One item = 16 columns; a row has `items` of them (whole 128 columns, so the
// padding of the scale row is written too).  Consecutive lanes take
// consecutive items; the two lanes of a group always sit side by side because
// `items` and the stride are even.
__global__ void __launch_bounds__(THREADS, QUANT_BLOCKS) k_act8_quantize(const __nv_bfloat16 *x, int64_t M, int64_t K,
                                                           int64_t ldx, uint8_t *__restrict__ codes, int64_t ldc,
                                                           uint8_t *__restrict__ scales, int64_t lds, int items)
{
    grid_wait();
    grid_release();
    const int64_t first = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    const int64_t stride = (int64_t)gridDim.x * THREADS;
    int64_t row = first / items;
    int item = (int)(first - row * items);
    const int64_t drow = stride / items;
    const int ditem = (int)(stride - drow * items);
    for (;;) {
        const bool live = row < M;                       // warp-uniform loop: every lane takes part in the shuffle
        if (!__any_sync(0xffffffffu, live)) break;
        const int64_t c = (int64_t)item * 16;
        uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (live) load16(x + row * ldx, c, K, w);
        const uint32_t s = scale_byte(group_amax(w));
        if (live && c < K) store16(codes + row * ldc, c, K, encode16(w, s));
        if (live && (item & 1) == 0) scales[row * lds + (item >> 1)] = (uint8_t)s;
        row += drow;
        item += ditem;
        if (item >= items) { item -= items; ++row; }
    }
}

// four codes -> four values (exact, unscaled)
__device__ __forceinline__ void decode4(uint32_t w, float v[4])
{
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
    const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<__half2 *>(&hi));
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}

// One item = 16 columns, as in the quantizer.  Every kept value is exact in
// bf16.  Row r of the result is kept row src_rows[r] (null: r); an index
// outside [0, T) gives zeros, and `outside` (where given) tells of it.
__global__ void __launch_bounds__(THREADS, DEQUANT_BLOCKS) k_act8_dequantize(const uint8_t *codes, int64_t ldc,
                                                             const uint8_t *scales, int64_t lds,
                                                             const int32_t *src_rows, int64_t T,
                                                             int64_t M, int64_t K, __nv_bfloat16 *__restrict__ x,
                                                             int64_t ldx, int items, uint8_t *__restrict__ outside)
{
    grid_wait();
    grid_release();
    const int64_t first = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    const int64_t stride = (int64_t)gridDim.x * THREADS;
    int64_t row = first / items;
    int item = (int)(first - row * items);
    const int64_t drow = stride / items;
    const int ditem = (int)(stride - drow * items);
    bool met = false;
    while (row < M) {
        const int64_t c = (int64_t)item * 16;
        const int64_t from = src_rows ? (int64_t)src_rows[row] : row;
        float s = 1.0f;
        uint32_t w[4] = {0, 0, 0, 0};
        if (from >= 0 && from < T) {
            s = scale_of(scales[from * lds + (item >> 1)]);
            const uint8_t *src = codes + from * ldc + c;
            if (c + 16 <= K) {
                const uint4 v = *reinterpret_cast<const uint4 *>(src);
                w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + i < K) w[i >> 2] |= (uint32_t)src[i] << (8 * (i & 3));
            }
        } else {
            met = true;
        }
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[4];
            decode4(w[i], v);
            o[2 * i] = pack_bf16(v[0] * s, v[1] * s);
            o[2 * i + 1] = pack_bf16(v[2] * s, v[3] * s);
        }
        __nv_bfloat16 *dst = x + row * ldx + c;
        if (c + 16 <= K) {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(dst + 8) = make_uint4(o[4], o[5], o[6], o[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c + i < K) dst[i] = __ushort_as_bfloat16((unsigned short)(o[i >> 1] >> (16 * (i & 1))));
        }
        row += drow;
        item += ditem;
        if (item >= items) { item -= items; ++row; }
    }
    if (outside) {
        const int any = __syncthreads_or(met);
        if (threadIdx.x == 0) outside[blockIdx.x] = any != 0;
    }
}

// 1 / (1 + 2^(-a log2 e)) of two values; the power may be infinite (the
// quotient is then 0).  Error: the exponent's rounding, |a| 2^-24 relative, and
// a few units in the last place.
__device__ __forceinline__ float2 sigmoid2(float2 a)
{
    const float2 e = __fmul2_rn(a, make_float2(-1.44269504f, -1.44269504f));
    float x, y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(x) : "f"(e.x));
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(e.y));
    const float2 d = __fadd2_rn(make_float2(x, y), make_float2(1.0f, 1.0f));
    asm("rcp.approx.f32 %0, %1;" : "=f"(x) : "f"(d.x));
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(d.y));
    return make_float2(x, y);
}

// h = silu(gate) * up and both inputs kept: one item = 16 columns of gate and
// the same 16 of up.
__global__ void __launch_bounds__(THREADS, SWIGLU_BLOCKS) k_swiglu_act8(const __nv_bfloat16 *y, int64_t M, int64_t I,
                                                         int64_t ldy, __nv_bfloat16 *__restrict__ h, int64_t ldh,
                                                         uint8_t *__restrict__ codes, int64_t ldc,
                                                         uint8_t *__restrict__ scales, int64_t lds, int items,
                                                         int pad_bytes)
{
    grid_wait();
    grid_release();
    const int64_t first = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    const int64_t stride = (int64_t)gridDim.x * THREADS;
    int64_t row = first / items;
    int item = (int)(first - row * items);
    const int64_t drow = stride / items;
    const int ditem = (int)(stride - drow * items);
    for (;;) {
        const bool live = row < M;
        if (!__any_sync(0xffffffffu, live)) break;
        const int64_t c = (int64_t)item * 16;
        uint32_t a[8] = {0, 0, 0, 0, 0, 0, 0, 0}, b[8] = {0, 0, 0, 0, 0, 0, 0, 0}, o[8];
        if (live) {
            load16(y + row * ldy, c, I, a);
            load16(y + row * ldy + I, c, I, b);
        }
        const uint32_t sa = scale_byte(group_amax(a)), sb = scale_byte(group_amax(b));
        if (live) {
            *reinterpret_cast<uint4 *>(codes + row * ldc + c) = encode16(a, sa);
            *reinterpret_cast<uint4 *>(codes + row * ldc + I + c) = encode16(b, sb);
            uint8_t *srow = scales + row * lds;
            if ((item & 1) == 0) {
                srow[item >> 1] = (uint8_t)sa;
                srow[(I >> 5) + (item >> 1)] = (uint8_t)sb;
                if (item == 0)
                    for (int i = 0; i < pad_bytes; ++i) srow[(I >> 4) + i] = 127;      // 2I / 32 groups, then padding
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 av = make_float2(bf16lo(a[i]), bf16hi(a[i]));
                const float2 hv = __fmul2_rn(__fmul2_rn(av, sigmoid2(av)), make_float2(bf16lo(b[i]), bf16hi(b[i])));
                o[i] = pack_bf16(hv.x, hv.y);
            }
            uint4 *dst = reinterpret_cast<uint4 *>(h + row * ldh + c);
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
        row += drow;
        item += ditem;
        if (item >= items) { item -= items; ++row; }
    }
}

// SwiGLU backward from kept inputs a (gate), b (up), s = sigmoid(a):
//   dgate = sum_i dh_i h_i,  h = a s b     (the router weight's gradient)
//   da = w dh b s (1 + a (1 - s)),  db = w dh a s,  gh = w h
// w the row's router weight.  One warp per row, 8 columns per lane and step;
// the row sum is a lane-ordered f32 sum and a fixed shuffle tree, so it does
// not change from run to run.
__global__ void __launch_bounds__(THREADS, BACKWARD_BLOCKS) k_swiglu_act8_backward(
    const uint8_t *codes, int64_t ldc, const uint8_t *scales, int64_t lds,
    const __nv_bfloat16 *dh, int64_t lddh, const float *row_gate, int64_t M, int64_t I,
    __nv_bfloat16 *__restrict__ dy, int64_t lddy, __nv_bfloat16 *__restrict__ gh, int64_t ldgh,
    float *__restrict__ dgate)
{
    grid_wait();
    grid_release();
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (THREADS / 32);
    for (int64_t row = (int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5); row < M; row += warps) {
        const uint8_t *crow = codes + row * ldc;
        const uint8_t *srow = scales + row * lds;
        const float w = row_gate ? row_gate[row] : 1.0f;
        const float2 w2 = make_float2(w, w);
        float2 sum = make_float2(0.0f, 0.0f);
        // unrolled three times 47.1, twice 46.7, four times 46.9, not at all 46.0 us
        // for 32768 rows of I = 768 (1536: 90.8, 91.6, 88.4, 87.7; 256: 19.0, 16.5, 18.3, 17.4)
#pragma unroll 1
        for (int64_t c = lane * 8; c < I; c += 256) {
            const uint2 ca = *reinterpret_cast<const uint2 *>(crow + c);
            const uint2 cb = *reinterpret_cast<const uint2 *>(crow + I + c);
            const uint4 d4 = *reinterpret_cast<const uint4 *>(dh + row * lddh + c);
            const float fa = scale_of(srow[c >> 5]), fb = scale_of(srow[(I + c) >> 5]);
            const uint32_t d[4] = {d4.x, d4.y, d4.z, d4.w};
            float a[8], b[8];
            decode4(ca.x, a);
            decode4(ca.y, a + 4);
            decode4(cb.x, b);
            decode4(cb.y, b + 4);
            uint32_t oa[4], ob[4], oh[4];
            const float2 fa2 = make_float2(fa, fa), fb2 = make_float2(fb, fb), one = make_float2(1.0f, 1.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 av = __fmul2_rn(make_float2(a[2 * i], a[2 * i + 1]), fa2);
                const float2 bv = __fmul2_rn(make_float2(b[2 * i], b[2 * i + 1]), fb2);
                const float2 u = make_float2(bf16lo(d[i]), bf16hi(d[i]));
                const float2 s = sigmoid2(av), as = __fmul2_rn(av, s), h = __fmul2_rn(as, bv), g = __fmul2_rn(w2, u);
                sum = __ffma2_rn(u, h, sum);
                const float2 t = __ffma2_rn(av, __ffma2_rn(s, make_float2(-1.0f, -1.0f), one), one);
                const float2 da = __fmul2_rn(__fmul2_rn(__fmul2_rn(g, bv), s), t);
                const float2 db = __fmul2_rn(g, as), hw = __fmul2_rn(w2, h);
                oa[i] = pack_bf16(da.x, da.y);
                ob[i] = pack_bf16(db.x, db.y);
                oh[i] = pack_bf16(hw.x, hw.y);
            }
            *reinterpret_cast<uint4 *>(dy + row * lddy + c) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
            *reinterpret_cast<uint4 *>(dy + row * lddy + I + c) = make_uint4(ob[0], ob[1], ob[2], ob[3]);
            if (gh) *reinterpret_cast<uint4 *>(gh + row * ldgh + c) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
        }
        float total = sum.x + sum.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        if (dgate && lane == 0) dgate[row] = total;
    }
}

// out[t] = sum_j g[t,j] rows[dst_row[t,j]] in slot order (f32): the routed
// rows of a token brought back together, without atomics.  One thread per 8
// columns of a token.
__global__ void __launch_bounds__(THREADS) k_combine_rows(const __nv_bfloat16 *rows, int64_t M, int64_t H,
                                                          int64_t ldr, const int32_t *dst_row,
                                                          const float *gate, int kr,
                                                          float *__restrict__ out, int64_t ldo)
{
    grid_wait();
    grid_release();
    const int64_t t = blockIdx.x;
    const int64_t c = ((int64_t)blockIdx.y * THREADS + threadIdx.x) * 8;
    if (c >= H) return;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 8
    for (int j = 0; j < kr; ++j) {
        const int32_t r = dst_row[t * kr + j];
        if (r < 0 || r >= M) continue;
        const float g = gate ? gate[t * kr + j] : 1.0f;
        const uint4 v = *reinterpret_cast<const uint4 *>(rows + (int64_t)r * ldr + c);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[2 * i] += g * bf16lo(w[i]);
            acc[2 * i + 1] += g * bf16hi(w[i]);
        }
    }
    float4 *dst = reinterpret_cast<float4 *>(out + t * ldo + c);
    dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
}

// Gradient of gates = softmax over the selected logits: one warp per token.
//   dlogits[t, e] = sum over slots j with idx_j = e of g_j (d_j - sum_i g_i d_i)
__global__ void __launch_bounds__(THREADS) k_route_backward(const int32_t *idx,
                                                            const float *gate,
                                                            const int32_t *dst_row,
                                                            const float *dgate_row, int64_t M, int64_t T,
                                                            int E, int kr, float *__restrict__ dlogits)
{
    grid_wait();
    grid_release();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5);
    if (t >= T) return;
    int e = -1;
    float g = 0.0f, d = 0.0f;
    if (lane < kr) {
        e = idx[t * kr + lane];
        g = gate[t * kr + lane];
        const int32_t r = dst_row[t * kr + lane];
        d = (r >= 0 && r < M) ? dgate_row[r] : 0.0f;
    }
    float s = g * d;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float v = g * (d - s);
    for (int e0 = 0; e0 < E; e0 += 32) {
        float acc = 0.0f;
        for (int j = 0; j < kr; ++j) {
            const int ej = __shfl_sync(0xffffffffu, e, j);
            const float vj = __shfl_sync(0xffffffffu, v, j);
            if (ej == e0 + lane) acc += vj;
        }
        if (e0 + lane < E) dlogits[t * E + e0 + lane] = acc;
    }
}

// Blocks of a streaming kernel over `work` threads: at most the `resident`
// ones per SM that its registers allow, so that no second wave of blocks
// starts when the first has shared out all the work (8 per SM where 6 fit:
// 45 instead of 37 us for 16384 x 4096).
static unsigned stream_blocks(int64_t work, int resident)
{
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>((work + THREADS - 1) / THREADS, (int64_t)num_sms() * resident));
}

}  // namespace act8

nvfp4_status act8_expand(const uint8_t *codes, int64_t ldc, const uint8_t *scales, int64_t lds, const int32_t *rows,
                         int64_t T, int64_t M, int64_t K, void *x, int64_t ldx, uint8_t *outside, int *blocks,
                         cudaStream_t stream)
{
    const int items = (int)((K + 15) / 16);
    const unsigned grid = act8::stream_blocks(M * items, act8::DEQUANT_BLOCKS);
    if (blocks) *blocks = (int)grid;
    launch_overlapped(act8::k_act8_dequantize, grid, act8::THREADS, 0, stream, codes, ldc, scales, lds, rows, T, M, K,
                      reinterpret_cast<__nv_bfloat16 *>(x), ldx, items, outside);
    return check_launch("k_act8_dequantize");
}

int act8_expand_max_blocks() { return num_sms() * act8::DEQUANT_BLOCKS; }

}  // namespace nvfp4

using namespace nvfp4;
using namespace nvfp4::act8;

extern "C" nvfp4_status act8_quantize(const void *x_dev, int64_t M, int64_t K, int64_t ldx, uint8_t *codes_dev,
                                      int64_t ld_codes, uint8_t *scales_dev, int64_t ld_scales, void *stream)
{
    NVFP4_REQUIRE(M >= 0 && K >= 0, NVFP4_ERR_INVALID_ARG, "act8_quantize: negative size");
    if (M == 0 || K == 0) return NVFP4_OK;
    NVFP4_REQUIRE(x_dev && codes_dev && scales_dev, NVFP4_ERR_INVALID_ARG, "act8_quantize: null pointer");
    NVFP4_REQUIRE(M < (1ll << 31) && K < (1ll << 24), NVFP4_ERR_UNSUPPORTED_SHAPE,
                  "act8_quantize: M must be below 2^31 and K below 2^24");
    NVFP4_REQUIRE(ldx >= K && ldx % 8 == 0, NVFP4_ERR_ALIGNMENT, "act8_quantize: ldx must be >= K and a multiple of 8");
    NVFP4_REQUIRE(ld_codes >= K && ld_codes % 16 == 0, NVFP4_ERR_ALIGNMENT,
                  "act8_quantize: ld_codes must be >= K and a multiple of 16");
    NVFP4_REQUIRE(ld_scales >= (K + 127) / 128 * 4 && ld_scales % 4 == 0, NVFP4_ERR_ALIGNMENT,
                  "act8_quantize: ld_scales must be >= 4 * ceil(K / 128) and a multiple of 4");
    NVFP4_REQUIRE(aligned16(x_dev) && aligned16(codes_dev) && aligned16(scales_dev), NVFP4_ERR_ALIGNMENT,
                  "act8_quantize: pointers must be 16-byte aligned");
    const int items = (int)((K + 127) / 128 * 8);
    launch_overlapped(k_act8_quantize, stream_blocks(M * items, QUANT_BLOCKS), THREADS, 0, (cudaStream_t)stream,
                      reinterpret_cast<const __nv_bfloat16 *>(x_dev), M, K, ldx, codes_dev, ld_codes, scales_dev,
                      ld_scales, items);
    return check_launch("k_act8_quantize");
}

extern "C" nvfp4_status act8_dequantize(const uint8_t *codes_dev, int64_t ld_codes, const uint8_t *scales_dev,
                                        int64_t ld_scales, int64_t M, int64_t K, void *x_dev, int64_t ldx,
                                        void *stream)
{
    NVFP4_REQUIRE(M >= 0 && K >= 0, NVFP4_ERR_INVALID_ARG, "act8_dequantize: negative size");
    if (M == 0 || K == 0) return NVFP4_OK;
    NVFP4_REQUIRE(x_dev && codes_dev && scales_dev, NVFP4_ERR_INVALID_ARG, "act8_dequantize: null pointer");
    NVFP4_REQUIRE(M < (1ll << 31) && K < (1ll << 24), NVFP4_ERR_UNSUPPORTED_SHAPE,
                  "act8_dequantize: M must be below 2^31 and K below 2^24");
    NVFP4_REQUIRE(ldx >= K && ldx % 8 == 0, NVFP4_ERR_ALIGNMENT, "act8_dequantize: ldx must be >= K and a multiple of 8");
    NVFP4_REQUIRE(ld_codes >= K && ld_codes % 16 == 0, NVFP4_ERR_ALIGNMENT,
                  "act8_dequantize: ld_codes must be >= K and a multiple of 16");
    NVFP4_REQUIRE(ld_scales >= (K + 31) / 32, NVFP4_ERR_ALIGNMENT, "act8_dequantize: ld_scales must be >= ceil(K / 32)");
    NVFP4_REQUIRE(aligned16(x_dev) && aligned16(codes_dev), NVFP4_ERR_ALIGNMENT,
                  "act8_dequantize: pointers must be 16-byte aligned");
    return act8_expand(codes_dev, ld_codes, scales_dev, ld_scales, nullptr, M, M, K, x_dev, ldx, nullptr, nullptr,
                       (cudaStream_t)stream);
}

extern "C" nvfp4_status moe_swiglu_act8(const void *y_dev, int64_t M, int64_t I, int64_t ldy, void *h_dev, int64_t ldh,
                                        uint8_t *codes_dev, int64_t ld_codes, uint8_t *scales_dev, int64_t ld_scales,
                                        void *stream)
{
    NVFP4_REQUIRE(M >= 0 && I >= 0, NVFP4_ERR_INVALID_ARG, "moe_swiglu_act8: negative size");
    if (M == 0 || I == 0) return NVFP4_OK;
    NVFP4_REQUIRE(y_dev && h_dev && codes_dev && scales_dev, NVFP4_ERR_INVALID_ARG, "moe_swiglu_act8: null pointer");
    NVFP4_REQUIRE(I % 32 == 0 && M < (1ll << 31) && I < (1ll << 23), NVFP4_ERR_UNSUPPORTED_SHAPE,
                  "moe_swiglu_act8: I must be a multiple of 32 below 2^23 and M below 2^31 (I=%lld)", (long long)I);
    NVFP4_REQUIRE(ldy >= 2 * I && ldy % 8 == 0 && ldh >= I && ldh % 8 == 0, NVFP4_ERR_ALIGNMENT,
                  "moe_swiglu_act8: ldy >= 2I and ldh >= I, multiples of 8");
    NVFP4_REQUIRE(ld_codes >= 2 * I && ld_codes % 16 == 0, NVFP4_ERR_ALIGNMENT,
                  "moe_swiglu_act8: ld_codes must be >= 2I and a multiple of 16");
    const int64_t row_bytes = (2 * I + 127) / 128 * 4;
    NVFP4_REQUIRE(ld_scales >= row_bytes && ld_scales % 4 == 0, NVFP4_ERR_ALIGNMENT,
                  "moe_swiglu_act8: ld_scales must be >= 4 * ceil(2I / 128) and a multiple of 4");
    NVFP4_REQUIRE(aligned16(y_dev) && aligned16(h_dev) && aligned16(codes_dev) && aligned16(scales_dev),
                  NVFP4_ERR_ALIGNMENT, "moe_swiglu_act8: pointers must be 16-byte aligned");
    const int items = (int)(I / 16);
    launch_overlapped(k_swiglu_act8, stream_blocks(M * items, SWIGLU_BLOCKS), THREADS, 0, (cudaStream_t)stream,
                      reinterpret_cast<const __nv_bfloat16 *>(y_dev), M, I, ldy, reinterpret_cast<__nv_bfloat16
                      *>(h_dev), ldh, codes_dev, ld_codes, scales_dev, ld_scales, items, (int)(row_bytes - 2 * I /
                      32));
    return check_launch("k_swiglu_act8");
}

extern "C" nvfp4_status moe_swiglu_act8_backward(const uint8_t *codes_dev, int64_t ld_codes, const uint8_t *scales_dev,
                                                 int64_t ld_scales, const void *dh_dev, int64_t lddh,
                                                 const float *row_gate_dev, int64_t M, int64_t I, void *dy_dev,
                                                 int64_t lddy, void *gh_dev, int64_t ldgh, float *dgate_dev,
                                                 void *stream)
{
    NVFP4_REQUIRE(M >= 0 && I >= 0, NVFP4_ERR_INVALID_ARG, "moe_swiglu_act8_backward: negative size");
    if (M == 0) return NVFP4_OK;
    if (I == 0) {
        if (dgate_dev && cudaMemsetAsync(dgate_dev, 0, (size_t)M * sizeof(float), (cudaStream_t)stream) != cudaSuccess)
            return check_launch("moe_swiglu_act8_backward: memset");
        return NVFP4_OK;
    }
    NVFP4_REQUIRE(codes_dev && scales_dev && dh_dev && dy_dev, NVFP4_ERR_INVALID_ARG,
                  "moe_swiglu_act8_backward: null pointer");
    NVFP4_REQUIRE(I % 32 == 0 && M < (1ll << 31) && I < (1ll << 23), NVFP4_ERR_UNSUPPORTED_SHAPE,
                  "moe_swiglu_act8_backward: I must be a multiple of 32 below 2^23 and M below 2^31 (I=%lld)",
                  (long long)I);
    NVFP4_REQUIRE(ld_codes >= 2 * I && ld_codes % 16 == 0 && ld_scales >= 2 * I / 32, NVFP4_ERR_ALIGNMENT,
                  "moe_swiglu_act8_backward: ld_codes >= 2I, a multiple of 16; ld_scales >= 2I / 32");
    NVFP4_REQUIRE(lddh >= I && lddh % 8 == 0 && lddy >= 2 * I && lddy % 8 == 0 &&
                  (!gh_dev || (ldgh >= I && ldgh % 8 == 0)), NVFP4_ERR_ALIGNMENT,
                  "moe_swiglu_act8_backward: lddh >= I, lddy >= 2I, ldgh >= I, multiples of 8");
    NVFP4_REQUIRE(aligned16(codes_dev) && aligned16(dh_dev) && aligned16(dy_dev) && aligned16(gh_dev),
                  NVFP4_ERR_ALIGNMENT, "moe_swiglu_act8_backward: pointers must be 16-byte aligned");
    const unsigned blocks = stream_blocks(M * 32, BACKWARD_BLOCKS);          // a warp per row
    launch_overlapped(k_swiglu_act8_backward, blocks, THREADS, 0, (cudaStream_t)stream, codes_dev, ld_codes,
                      scales_dev, ld_scales, reinterpret_cast<const __nv_bfloat16 *>(dh_dev), lddh, row_gate_dev, M,
                      I, reinterpret_cast<__nv_bfloat16 *>(dy_dev), lddy, reinterpret_cast<__nv_bfloat16 *>(gh_dev),
                      ldgh, dgate_dev);
    return check_launch("k_swiglu_act8_backward");
}

extern "C" nvfp4_status moe_combine_rows(const void *rows_dev, int64_t M, int64_t H, int64_t ld_rows,
                                         const int32_t *dst_row_dev, const float *gate_dev, int64_t T, int32_t k_r,
                                         float *out_dev, int64_t ld_out, void *stream)
{
    NVFP4_REQUIRE(M >= 0 && H >= 0 && T >= 0, NVFP4_ERR_INVALID_ARG, "moe_combine_rows: negative size");
    if (T == 0 || H == 0) return NVFP4_OK;
    NVFP4_REQUIRE((M == 0 || rows_dev) && dst_row_dev && out_dev, NVFP4_ERR_INVALID_ARG,
                  "moe_combine_rows: null pointer");
    NVFP4_REQUIRE(k_r >= 1 && k_r <= 32, NVFP4_ERR_INVALID_ARG, "moe_combine_rows: k_r must be in [1, 32]");
    NVFP4_REQUIRE(M < (1ll << 31) && T < (1ll << 31) && H <= 65535ll * THREADS * 8, NVFP4_ERR_UNSUPPORTED_SHAPE,
                  "moe_combine_rows: too many rows or columns");
    NVFP4_REQUIRE(H % 8 == 0 && ld_rows >= H && ld_rows % 8 == 0 && ld_out >= H && ld_out % 4 == 0, NVFP4_ERR_ALIGNMENT,
                  "moe_combine_rows: H and ld_rows multiples of 8, ld_out a multiple of 4, both >= H");
    NVFP4_REQUIRE(aligned16(rows_dev) && aligned16(out_dev), NVFP4_ERR_ALIGNMENT,
                  "moe_combine_rows: pointers must be 16-byte aligned");
    const dim3 grid((unsigned)T, (unsigned)((H + THREADS * 8 - 1) / (THREADS * 8)));
    launch_overlapped(k_combine_rows, grid, THREADS, 0, (cudaStream_t)stream, reinterpret_cast<const __nv_bfloat16
                      *>(rows_dev), M, H, ld_rows, dst_row_dev, gate_dev, k_r, out_dev, ld_out);
    return check_launch("k_combine_rows");
}

extern "C" nvfp4_status moe_route_backward(const int32_t *topk_idx_dev, const float *topk_gate_dev,
                                           const int32_t *dst_row_dev, const float *dgate_row_dev, int64_t M, int64_t T,
                                           int32_t E, int32_t k_r, float *dlogits_dev, void *stream)
{
    NVFP4_REQUIRE(T >= 0 && M >= 0, NVFP4_ERR_INVALID_ARG, "moe_route_backward: negative size");
    if (T == 0) return NVFP4_OK;
    NVFP4_REQUIRE(topk_idx_dev && topk_gate_dev && dst_row_dev && (M == 0 || dgate_row_dev) && dlogits_dev,
                  NVFP4_ERR_INVALID_ARG, "moe_route_backward: null pointer");
    NVFP4_REQUIRE(E >= 1 && E <= 65536 && k_r >= 1 && k_r <= 32 && T < (1ll << 31), NVFP4_ERR_UNSUPPORTED_SHAPE,
                  "moe_route_backward: need 1 <= E <= 65536, 1 <= k_r <= 32, T < 2^31");
    const unsigned blocks = (unsigned)((T + THREADS / 32 - 1) / (THREADS / 32));
    launch_overlapped(k_route_backward, blocks, THREADS, 0, (cudaStream_t)stream, topk_idx_dev, topk_gate_dev,
                      dst_row_dev, dgate_row_dev, M, T, E, k_r, dlogits_dev);
    return check_launch("k_route_backward");
}
