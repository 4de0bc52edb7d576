// gemv.cu -- products of a few tokens with NVFP4 weights in BF16 activations
// (W4A16): the rollout layer's single-token form.
//
//   y[r, n] = s_t[e] * sum_k e2m1(w_e[n,k]) sf_e[n, k/16] x[r, k]
//
// Bound by HBM: 0.5625 bytes per weight, each read once; a token's rows of x
// stay in L1.  To keep up with HBM (about 41 weights per clock and SM) the
// decode has to cost about two instructions per weight, so the multiply-adds
// go to mma.sync (m16n8k16, BF16, f32 accumulation): 16 weight rows times up
// to 8 tokens per instruction.  A single token uses one of the 8 columns;
// the tensor pipe is idle otherwise.
//
// Decode: a nibble's bits s|ee|m land in a BF16's sign, low exponent and top
// mantissa bits, which reads as e2m1 * 2^-126 (its subnormal included); one
// BF16 multiplication by sf * 2^117 gives e2m1 * sf * 2^-9, exact (at most 6
// significant bits).  2^9 joins the tensor scale at the end.  The only
// roundings of a product are those of the f32 accumulation.
//
// A warp takes 16 weight rows and 128 columns a step: lane (g, t) = (lane / 4,
// lane % 4) loads 32 consecutive weights (16 bytes, two scale blocks) of row g
// and of row g + 8.  MMA k-slots may be matched to columns in any order as
// long as both operands agree, so each lane feeds its own 32 columns and x is
// loaded in the same arrangement.  The 16 rows are 4 rows of each 32-row
// quarter of a 128-row scale atom: their scales are 64 contiguous bytes.
// A block's 8 warps split the columns (or the token's experts); partial sums
// meet in shared memory and are added in warp order.
#include "common.cuh"

#include <algorithm>

namespace nvfp4 {
namespace gemv {

constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr int ROWS = 16;                 // weight rows per warp tile
constexpr int COLS = 8;                  // tokens per MMA

enum Form { STORE = 0, SWIGLU = 1, COMBINE = 2 };

struct Params {
    const __nv_bfloat16 *x;
    int64_t ldx;
    const uint8_t *codes;
    const uint8_t *scales;
    const float *s_t;
    int64_t N, K;
    int E;
    const int32_t *idx;                  // [T x k_r] or null (one dense weight)
    int64_t T;
    int k_r;
    const float *gate;
    void *out;
    int64_t ld_out;
};

struct Step {
    uint4 c[2];                          // codes of rows g, g + 8
    uint32_t s[2];                       // their two scale bytes
    uint4 x[4];
};

__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// E4M3 scale byte -> sf * 2^117 in both halves (exact: the byte's bits read as
// sf * 2^-120).
__device__ __forceinline__ uint32_t scale_operand(uint32_t b)
{
    return bmul2(bmul2(b * 0x00100010u, 0x7B807B80u), 0x7A007A00u);
}

// Eight codes -> four BF16 pairs (element i, element i + 4), unscaled * 2^-126.
__device__ __forceinline__ void decode8(uint32_t w, uint32_t p[4])
{
    constexpr uint32_t SIGN = 0x80008000u, MAG = 0x01C001C0u;
    p[0] = ((w << 12) & SIGN) | ((w << 6) & MAG);
    p[1] = ((w << 8) & SIGN) | ((w << 2) & MAG);
    p[2] = ((w << 4) & SIGN) | ((w >> 2) & MAG);
    p[3] = (w & SIGN) | ((w >> 6) & MAG);
}

__device__ __forceinline__ void mma16816(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weight row of tile-local row rr (0..15): 4 rows of each 32-row quarter.
__device__ __forceinline__ int64_t tile_row(int tile, int rr)
{
    const int g = rr & 7;
    return (int64_t)(tile >> 3) * 128 + 32 * (g & 3) + 4 * (tile & 7) + (g >> 2) + 2 * (rr >> 3);
}

// One expert's weight as a lane sees it.
struct Lane {
    const uint8_t *c[2];                 // codes of its two rows, or null
    const uint8_t *s[2];                 // their scale words in column group 0
    const __nv_bfloat16 *x;              // its token's row, or null
};

__device__ __forceinline__ void load_step(Step &st, const Lane &l, int64_t k0, int64_t K)
{
    const bool in = k0 < K;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        st.c[h] = make_uint4(0, 0, 0, 0);
        st.s[h] = 0;
        if (in && l.c[h]) {
            st.c[h] = __ldg(reinterpret_cast<const uint4 *>(l.c[h] + (k0 >> 1)));
            // scale column k0 / 16: 64-column atoms of 512 bytes, 4 bytes per row
            st.s[h] = __ldg(reinterpret_cast<const uint16_t *>(l.s[h] + (k0 >> 6) * 512 + ((k0 >> 4) & 3)));
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        st.x[i] = make_uint4(0, 0, 0, 0);
        if (in && l.x) st.x[i] = __ldg(reinterpret_cast<const uint4 *>(l.x + k0) + i);
    }
}

__device__ __forceinline__ void compute_step(const Step &st, float (&acc)[2][4])
{
    const uint32_t ca[4] = {st.c[0].x, st.c[0].y, st.c[0].z, st.c[0].w};
    const uint32_t cb[4] = {st.c[1].x, st.c[1].y, st.c[1].z, st.c[1].w};
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
        const uint32_t sa = scale_operand((st.s[0] >> (8 * blk)) & 0xFFu);
        const uint32_t sb = scale_operand((st.s[1] >> (8 * blk)) & 0xFFu);
#pragma unroll
        for (int q = 2 * blk; q < 2 * blk + 2; ++q) {
            uint32_t pa[4], pb[4];
            decode8(ca[q], pa);
            decode8(cb[q], pb);
            // x pairs (i, i + 4)
            const uint4 v = st.x[q];
            const uint32_t x0 = __byte_perm(v.x, v.z, 0x5410), x1 = __byte_perm(v.x, v.z, 0x7632);
            const uint32_t x2 = __byte_perm(v.y, v.w, 0x5410), x3 = __byte_perm(v.y, v.w, 0x7632);
            mma16816(acc[0], bmul2(pa[0], sa), bmul2(pb[0], sb), bmul2(pa[1], sa), bmul2(pb[1], sb), x0, x1);
            mma16816(acc[1], bmul2(pa[2], sa), bmul2(pb[2], sb), bmul2(pa[3], sa), bmul2(pb[3], sb), x2, x3);
        }
    }
}

// Columns [128 ch0, ...) in steps of 128 * stride, the next step's loads in
// flight while one is computed.
__device__ __forceinline__ void dot_range(const Lane &l, int ch0, int stride, int chunks, int64_t K, float (&acc)[2][4])
{
    const int t = threadIdx.x & 3;
    if (ch0 >= chunks) return;
    Step cur, nxt;
    load_step(cur, l, (int64_t)ch0 * 128 + 32 * t, K);
    for (int ch = ch0; ch < chunks; ch += stride) {
        if (ch + stride < chunks) load_step(nxt, l, (int64_t)(ch + stride) * 128 + 32 * t, K);
        compute_step(cur, acc);
        cur = nxt;
    }
}

__device__ __forceinline__ Lane lane_of(const Params &p, int e, int tile, int64_t row_base, int64_t row_end,
                                        const __nv_bfloat16 *x)
{
    const int g = (threadIdx.x & 31) >> 2;
    const int64_t sf_expert = ((p.N + 127) / 128) * 128 * (p.K / 16);
    Lane l;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t r = tile_row(tile, g + 8 * h);
        const int64_t n = row_base + r;
        const bool ok = e >= 0 && n < row_end;
        l.c[h] = ok ? p.codes + ((int64_t)e * p.N + n) * (p.K / 2) : nullptr;
        l.s[h] = ok ? p.scales + (int64_t)e * sf_expert + sf_offset(n, 0, p.K) : nullptr;
    }
    l.x = x;
    return l;
}

__device__ __forceinline__ float silu(float z) { return __fdividef(z, 1.0f + expf(-z)); }

// blockIdx.x: (token, slot) pair / group of 8 tokens (dense) / token
// (COMBINE), fastest, so that blocks that share an expert's rows run together
// and meet in L2; blockIdx.y: tile of 16 rows.
template <int FORM>
__global__ void __launch_bounds__(THREADS, 2) k_nvfp4_gemv(const Params p)
{
    __shared__ float part[WARPS][ROWS][COLS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int tile = blockIdx.y;
    const int chunks = (int)((p.K + 127) / 128);
    const int64_t b = blockIdx.x;
    const bool dense = p.idx == nullptr;
    const int64_t n_rows = FORM == SWIGLU ? p.N / 2 : p.N;       // output rows
    float tot[4] = {0, 0, 0, 0};

    if (FORM == COMBINE) {
        // the token's (expert, chunk) pairs, dealt to the warps in order
        const int units = p.k_r * chunks;
        const int per = (units + WARPS - 1) / WARPS;
        int u = warp * per;
        const int u_end = min(u + per, units);
        while (u < u_end) {
            const int j = u / chunks, ch = u - j * chunks;
            const int ch_end = min(chunks, ch + (u_end - u));
            const int64_t pair = b * p.k_r + j;
            const int e = dense ? 0 : p.idx[pair];
            if (e >= 0 && e < p.E) {
                const Lane l = lane_of(p, e, tile, 0, p.N, g == 0 ? p.x + pair * p.ldx : nullptr);
                float acc[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
                dot_range(l, ch, 1, ch_end, p.K, acc);
                const float coef = p.gate ? p.gate[pair] * p.s_t[e] : p.s_t[e];
#pragma unroll
                for (int i = 0; i < 4; ++i) tot[i] += coef * (acc[0][i] + acc[1][i]);
            }
            u += ch_end - ch;
        }
    } else {
        int64_t tok;
        int e = 0;
        const __nv_bfloat16 *x = nullptr;
        if (dense) {
            tok = b * COLS + g;
            if (tok < p.T) x = p.x + tok * p.ldx;
        } else {
            tok = b / p.k_r;
            e = p.idx[b];
            if (e < 0 || e >= p.E) e = -1;
            if (g == 0) x = p.x + tok * p.ldx;
        }
        const int parts = FORM == SWIGLU ? WARPS / 2 : WARPS;      // warps that share one set of rows
        const int64_t base = FORM == SWIGLU && warp >= parts ? p.N / 2 : 0;
        if (e >= 0) {
            const Lane l = lane_of(p, e, tile, base, base + n_rows, x);
            float acc[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
            dot_range(l, warp % parts, parts, chunks, p.K, acc);
            const float coef = p.s_t[e];
#pragma unroll
            for (int i = 0; i < 4; ++i) tot[i] = coef * (acc[0][i] + acc[1][i]);
        }
    }
    part[warp][g][2 * t] = tot[0];
    part[warp][g][2 * t + 1] = tot[1];
    part[warp][g + 8][2 * t] = tot[2];
    part[warp][g + 8][2 * t + 1] = tot[3];
    __syncthreads();
    // 16 rows x 8 columns; the operands carry 2^-9
    if (threadIdx.x < ROWS * COLS) {
        const int rr = threadIdx.x & 15, col = threadIdx.x >> 4;
        const int64_t n = tile_row(tile, rr);
        const int64_t orow = FORM != COMBINE && dense ? b * COLS + col : b;
        const bool live = n < n_rows && (FORM != COMBINE && dense ? orow < p.T : col == 0);
        if (live) {
            if (FORM == SWIGLU) {
                float a = 0.0f, u = 0.0f;
#pragma unroll
                for (int w = 0; w < WARPS / 2; ++w) {
                    a += part[w][rr][col];
                    u += part[w + WARPS / 2][rr][col];
                }
                a *= 512.0f;
                u *= 512.0f;
                reinterpret_cast<__nv_bfloat16 *>(p.out)[orow * p.ld_out + n] = __float2bfloat16_rn(silu(a) * u);
            } else {
                float y = 0.0f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) y += part[w][rr][col];
                reinterpret_cast<float *>(p.out)[orow * p.ld_out + n] = 512.0f * y;
            }
        }
    }
}

}  // namespace gemv
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status moe_nvfp4_gemv(const void *x_dev, int64_t T, int64_t ldx, const uint8_t *codes_dev,
                                       const uint8_t *scales_dev, const float *s_t_dev, int64_t N, int64_t K,
                                       int32_t E, const int32_t *expert_idx_dev, int32_t k_r, int32_t epilogue,
                                       const float *gate_dev, void *out_dev, int64_t ld_out, void *stream)
{
    using namespace nvfp4::gemv;
    NVFP4_REQUIRE(epilogue == MOE_EPI_STORE_F32 || epilogue == MOE_EPI_SWIGLU_BF16 || epilogue == MOE_EPI_COMBINE_F32,
                  NVFP4_ERR_INVALID_ARG, "moe_nvfp4_gemv: bad epilogue");
    NVFP4_REQUIRE(T >= 0, NVFP4_ERR_INVALID_ARG, "moe_nvfp4_gemv: negative size");
    NVFP4_REQUIRE(E >= 1 && k_r >= 1 && k_r <= 32, NVFP4_ERR_UNSUPPORTED_SHAPE,
                  "moe_nvfp4_gemv: need E >= 1 and 1 <= k_r <= 32");
    NVFP4_REQUIRE(expert_idx_dev || (k_r == 1 && E == 1), NVFP4_ERR_INVALID_ARG,
                  "moe_nvfp4_gemv: without expert_idx there is one weight (E = 1, k_r = 1)");
    NVFP4_REQUIRE(N >= 1 && K >= 64 && K % 64 == 0 && K < (1ll << 31), NVFP4_ERR_UNSUPPORTED_SHAPE,
                  "moe_nvfp4_gemv: N must be positive and K a positive multiple of 64 (N=%lld, K=%lld)", (long long)N,
                  (long long)K);
    NVFP4_REQUIRE(epilogue != MOE_EPI_SWIGLU_BF16 || N % 2 == 0, NVFP4_ERR_UNSUPPORTED_SHAPE,
                  "moe_nvfp4_gemv: SwiGLU needs an even N");
    const int64_t rows = epilogue == MOE_EPI_SWIGLU_BF16 ? N / 2 : N;
    const int64_t tiles = (rows + 127) / 128 * 8;
    NVFP4_REQUIRE(tiles <= 65535 && T * k_r < (1ll << 31), NVFP4_ERR_UNSUPPORTED_SHAPE,
                  "moe_nvfp4_gemv: N or T too large");
    if (T == 0) return NVFP4_OK;
    NVFP4_REQUIRE(x_dev && codes_dev && scales_dev && s_t_dev && out_dev, NVFP4_ERR_INVALID_ARG,
                  "moe_nvfp4_gemv: null pointer");
    NVFP4_REQUIRE(ldx >= K && ldx % 8 == 0 && ld_out >= rows, NVFP4_ERR_ALIGNMENT,
                  "moe_nvfp4_gemv: ldx must be >= K and a multiple of 8, ld_out >= the output width");
    NVFP4_REQUIRE(aligned16(x_dev) && aligned16(codes_dev) && aligned16(scales_dev), NVFP4_ERR_ALIGNMENT,
                  "moe_nvfp4_gemv: pointers must be 16-byte aligned");
    Params p;
    p.x = reinterpret_cast<const __nv_bfloat16 *>(x_dev);
    p.ldx = ldx;
    p.codes = codes_dev;
    p.scales = scales_dev;
    p.s_t = s_t_dev;
    p.N = N;
    p.K = K;
    p.E = E;
    p.idx = expert_idx_dev;
    p.T = T;
    p.k_r = k_r;
    p.gate = gate_dev;
    p.out = out_dev;
    p.ld_out = ld_out;
    const int64_t units = epilogue == MOE_EPI_COMBINE_F32 ? T : expert_idx_dev ? T * k_r : (T + COLS - 1) / COLS;
    const dim3 grid((unsigned)units, (unsigned)tiles);
    cudaStream_t st = (cudaStream_t)stream;
    if (epilogue == MOE_EPI_SWIGLU_BF16) k_nvfp4_gemv<SWIGLU><<<grid, THREADS, 0, st>>>(p);
    else if (epilogue == MOE_EPI_COMBINE_F32) k_nvfp4_gemv<COMBINE><<<grid, THREADS, 0, st>>>(p);
    else k_nvfp4_gemv<STORE><<<grid, THREADS, 0, st>>>(p);
    return check_launch("k_nvfp4_gemv");
}
