// gemv.cu -- products of a few tokens with NVFP4 weights in BF16 activations
// (W4A16): the rollout layer's single-token form.
//
//   y[r, n] = s_t[e] * sum_k e2m1(w_e[n,k]) sf_e[n, k/16] x[r, k]
//
// The floor is HBM (0.5625 bytes per weight, each read once: 41 weights per
// clock and SM); what bounds it is the decode, with the loads behind it.  A
// weight costs 3.8 thread-instructions in all (1.0 mask, 0.6 multiplication, 0.1
// shift, 0.6 scale, 0.13 MMA, the rest copies, x and addresses), the whole issue
// 1.2 times the HBM rate: 82 experts of 4096 x 1536 (16 tokens, top-8 of 128)
// take 94-101 us (by box) against 45 for the bytes, with 62% of the issue slots in use.
// (When it took 99: copies and x without the products 75, products with half
// the decode 86.  Neither alone is the bound, and the registers allow no more
// warps to overlap them.)
// The multiply-adds go to mma.sync (m16n8k16, BF16, f32 accumulation), 16
// weight rows times up to 8 tokens per instruction: the tensor pipe is idle
// otherwise (13% with them), and a second token costs no decode.  Measured
// slower: more warps per SM (spills at 80 registers; 96 registers the same),
// operands prefetched in registers instead of shared slots, a fourth slot (106
// us: less L1 for x), first MMAs without a zeroed accumulator (one token
// gate/up 9.6 instead of 9.3 us).
//
// Decode: a nibble's bits s|ee|m land in a BF16's sign, low exponent and top
// mantissa bits, which reads as e2m1 * 2^-126 (its subnormal included); one
// BF16 multiplication by sf * 2^117 gives e2m1 * sf * 2^-9, exact (at most 6
// significant bits).  2^9 joins the tensor scale at the end.  The only
// roundings of a product are those of the f32 accumulation: the tensor core
// truncates its additions, so a chunk's 8 MMAs start from zero and the chunks
// are added in f32 (16 tokens, down 4096 x 1536: error 4.4e-7 -> 1.0e-7 in
// norm, that of plain f32 sums, for 0.2% of the time).
//
// A warp takes 16 weight rows and 128 columns a step: lane (g, t) = (lane / 4,
// lane % 4) loads 32 consecutive weights (16 bytes, two scale blocks) of row g
// and of row g + 8.  MMA k-slots may be matched to columns in any order as
// long as both operands agree, so each lane feeds its own 32 columns and x is
// loaded in the same arrangement.  The 16 rows are 4 rows of each 32-row
// quarter of a 128-row scale atom: their scales are 64 contiguous bytes.
// Warps that split the columns (or a token's experts) meet in shared memory;
// their sums are added in warp order.
#include "common.cuh"

#include <algorithm>
#include <mutex>

namespace nvfp4 {
namespace gemv {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int COMBINE_WARPS = 8;         // of a one-launch combine block
constexpr int ROWS = 16;                 // weight rows of a set
constexpr int COLS = 8;                  // tokens per MMA

constexpr int BLOCKS = 4;                // resident per SM
constexpr int DEPTH = 3;                 // ring slots per warp: one chunk computed, DEPTH - 1 in flight
constexpr int MAX_PAIRS = 1024;          // (token, slot) pairs per launch

enum Form { STORE = 0, SWIGLU = 1 };

struct Params {
    const __nv_bfloat16 *x;
    int64_t ldx;
    const uint8_t *codes;
    const uint8_t *scales;
    const float *s_t;
    int32_t N, K;
    int E;
    int64_t code_stride, scale_stride;   // bytes of one expert's codes and scales
    const int32_t *idx;                  // experts of the pairs, or null (one dense weight)
    int pairs;                           // (token, slot) pairs (dense: tokens)
    int k_r;
    uint32_t x_mul;                      // row of x = pair * x_mul >> 16 (pair / k_r, or pair)
    const float *gate;
    void *out;
    int64_t ld_out;
    int x_wide;                          // rows of x start on 32 bytes
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
// One multiplication puts a nibble at both places, its sign's (<< 12) and its
// magnitude's (<< 6): 9 operations of the ALU pipe where shifts and masks take
// 15 (16 tokens, down 4096 x 1536: 98.3 -> 95.0 us).
__device__ __forceinline__ void decode8(uint32_t w, uint32_t p[4])
{
    constexpr uint32_t FIELDS = 0x81C081C0u;                     // sign, and exponent with mantissa
    const uint32_t u = w >> 8;
    p[0] = ((w & 0x000F000Fu) * 0x1040u) & FIELDS;
    p[1] = ((w & 0x00F000F0u) * 0x0104u) & FIELDS;
    p[2] = ((u & 0x000F000Fu) * 0x1040u) & FIELDS;
    p[3] = ((u & 0x00F000F0u) * 0x0104u) & FIELDS;
}

__device__ __forceinline__ void mma16816(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weight row of tile-local row rr (0..15): 4 rows of each 32-row quarter.
__device__ __forceinline__ int tile_row(int tile, int rr)
{
    const int g = rr & 7;
    return (tile >> 3) * 128 + 32 * (g & 3) + 4 * (tile & 7) + (g >> 2) + 2 * (rr >> 3);
}

// A lane's pointer into one 16-row set: codes of row g, column 0; row g + 8
// (two weight rows further) lies c2 bytes on.  A row past the end reads an
// existing one; its sums are not stored.
struct Set {
    const uint8_t *c;
    int32_t c2;
};

__device__ __forceinline__ Set set_of(const Params &p, const uint8_t *codes, int tile, int row_base, int rows)
{
    const int r = tile_row(tile, (threadIdx.x & 31) >> 2);
    Set l;
    l.c = codes + (uint64_t)(uint32_t)(row_base + min(r, rows - 1)) * (uint32_t)(p.K >> 1);
    l.c2 = r + 2 < rows ? p.K : 0;
    return l;
}

// Scale word of a set's row rr, columns 0..63 (a row past the end: an existing
// one's).
__device__ __forceinline__ const uint8_t *scales_of(const Params &p, const uint8_t *scales, int tile, int row_base, int rows,
                                                    int rr)
{
    const uint32_t n = (uint32_t)(row_base + min(tile_row(tile, rr), rows - 1));
    return scales + (uint64_t)(n >> 7) * ((uint32_t)p.K * 8u) + (n & 31u) * 16u + ((n >> 5) & 3u) * 4u;
}

// 128 columns of SETS row sets: codes c and scale words s of their rows (set
// k: 2k, 2k + 1), the lane's two scale bytes being byte0 and byte0 + 1 of a
// word; the lane's 32 x as pairs (i, i + 4) in xp.  The sets take turns, so one's
// decode runs under the other's dependent MMAs (one token gate/up 9.55 ->
// 9.27 us).
template <int SETS>
__device__ __forceinline__ void compute_chunk(const uint32_t (&c)[2 * SETS][4], const uint32_t (&s)[2 * SETS],
                                              uint32_t byte0, const uint32_t (&xp)[16], float (&acc)[SETS][4])
{
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
        const uint32_t pick = 0x4440u + byte0 + blk;
        uint32_t sf[2 * SETS];
#pragma unroll
        for (int r = 0; r < 2 * SETS; ++r) sf[r] = scale_operand(__byte_perm(s[r], 0u, pick));
#pragma unroll
        for (int q = 2 * blk; q < 2 * blk + 2; ++q)
#pragma unroll
            for (int k = 0; k < SETS; ++k) {
                uint32_t pa[4], pb[4];
                const uint32_t sa = sf[2 * k], sb = sf[2 * k + 1];
                decode8(c[2 * k][q], pa);
                decode8(c[2 * k + 1][q], pb);
                mma16816(acc[k], bmul2(pa[0], sa), bmul2(pb[0], sb), bmul2(pa[1], sa), bmul2(pb[1], sb), xp[4 * q],
                         xp[4 * q + 1]);
                mma16816(acc[k], bmul2(pa[2], sa), bmul2(pb[2], sb), bmul2(pa[3], sa), bmul2(pb[3], sb), xp[4 * q + 2],
                         xp[4 * q + 3]);
            }
    }
}

// One chunk's operands in flight through shared memory.  A lane reads back the
// codes that it copied itself; the scale words are shared: the warp copies each
// of its rows' two words (64 columns each) once, in an order that puts a lane's
// rows side by side (set k, row g + 8 hi at g * 2 SETS + 2 k + hi).  Each lane
// copying its own (four 4-byte copies a chunk instead of two, half of them
// twice) took 11 us of the 75 that the loads of 16 tokens' down products take
// by themselves.
template <int SETS>
struct Slot {
    uint4 c[2 * SETS][32];               // codes of the lane's rows
    uint32_t s[2][16 * (2 * SETS - 1)];  // scale words per 64 columns (the halves 16 banks apart)
};

// The lane's (half, row) among the scale words of its warp's copy j < SETS.
template <int SETS>
struct ScaleWord {
    int half, pos, k, rr;
    __device__ __forceinline__ ScaleWord(int j, int lane)
    {
        const int i = j * 32 + lane;
        half = i / (16 * SETS);
        pos = i % (16 * SETS);
        k = pos / 2 % SETS;
        rr = pos / (2 * SETS) + 8 * (pos & 1);
    }
};

__device__ __forceinline__ void copy16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

__device__ __forceinline__ void copy4(void *dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

// 16 bytes of x.
__device__ __forceinline__ void load16(const __nv_bfloat16 *src, uint4 &a)
{
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w) : "l"(src));
}

// 32 bytes of x (32-byte aligned).
__device__ __forceinline__ void load32(const __nv_bfloat16 *src, uint4 &a, uint4 &b)
{
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(src));
}

// Chunks of 128 columns ch0, ch0 + stride, ... below `chunks`, of SETS row sets
// against the same x; DEPTH - 1 chunks are in flight while one is computed.
// s: this lane's rows for ScaleWord j.  x: the lane's token row (a column
// without a token may take any row: its sums are not stored).  K is a multiple
// of 64, so half of the last chunk may be missing: its lanes read earlier
// columns again, against zeros of x.
template <int SETS>
__device__ __forceinline__ void dot_range(Slot<SETS> *ring, const Set (&l)[SETS], const uint8_t *const (&s)[SETS],
                                          const __nv_bfloat16 *x, bool x_wide, int ch0, int stride, int chunks, int K,
                                          float (&acc)[SETS][4])
{
    const int lane = threadIdx.x & 31, t = lane & 3;
    if (ch0 >= chunks) return;
    const int n = (chunks - 1 - ch0) / stride + 1;
    const int step = stride * 128;
    int base = ch0 * 128;                                         // of the next chunk to copy
    const int col0 = base + 32 * t;
    const int at = col0 < K ? col0 : col0 - 64;
    const uint8_t *pc[SETS], *ps[SETS];
#pragma unroll
    for (int k = 0; k < SETS; ++k) {
        pc[k] = l[k].c + (at >> 1);
        ps[k] = s[k] + (uint64_t)((base >> 6) + ScaleWord<SETS>(k, lane).half) * 512;
    }
    int issued = 0;
    auto issue = [&]() {
        if (issued < n) {
            Slot<SETS> &slot = ring[issued % DEPTH];
#pragma unroll
            for (int k = 0; k < SETS; ++k) {
                copy16(&slot.c[2 * k][lane], pc[k]);
                copy16(&slot.c[2 * k + 1][lane], pc[k] + l[k].c2);
                const ScaleWord<SETS> w(k, lane);
                copy4(&slot.s[w.half][w.pos], base + 64 * w.half < K ? ps[k] : ps[k] - 512);
            }
            ++issued;
            base += step;
#pragma unroll
            for (int k = 0; k < SETS; ++k) {
                if (base + 32 * t < K) pc[k] += step / 2;
                ps[k] += step * 8;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint4 v[4];
    const __nv_bfloat16 *px = x + at;
    auto load_x = [&]() {
        if (x_wide) {
            load32(px, v[0], v[1]);
            load32(px + 16, v[2], v[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) load16(px + 8 * k, v[k]);
        }
    };
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i) issue();
    load_x();
    int xcol = col0;                                              // of the chunk whose x is in v
    for (int i = 0; i < n; ++i) {
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 2) : "memory");
        __syncwarp();                                             // chunk i has landed, chunk i - 1 has been read, by every lane
        issue();
        uint32_t xp[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            xp[4 * q] = __byte_perm(v[q].x, v[q].z, 0x5410);
            xp[4 * q + 1] = __byte_perm(v[q].x, v[q].z, 0x7632);
            xp[4 * q + 2] = __byte_perm(v[q].y, v[q].w, 0x5410);
            xp[4 * q + 3] = __byte_perm(v[q].y, v[q].w, 0x7632);
        }
        if (i + 1 == n && (K & 64)) {
            // the last chunk may be the half one (uniform branch; full lanes keep theirs)
            const uint32_t keep = xcol < K ? 0xFFFFFFFFu : 0u;
#pragma unroll
            for (int q = 0; q < 16; ++q) xp[q] &= keep;
        }
        if (i + 1 < n) {
            xcol += step;
            if (xcol < K) px += step;
            load_x();
        }
        const Slot<SETS> &slot = ring[i % DEPTH];
        const uint32_t *words = &slot.s[t >> 1][(lane >> 2) * 2 * SETS];
        uint32_t w[2 * SETS];
        if (SETS == 2) {
            const uint4 q = *reinterpret_cast<const uint4 *>(words);
            w[0] = q.x; w[1] = q.y; w[2 * SETS - 2] = q.z; w[2 * SETS - 1] = q.w;
        } else {
            const uint2 q = *reinterpret_cast<const uint2 *>(words);
            w[0] = q.x; w[1] = q.y;
        }
        uint32_t c[2 * SETS][4];
#pragma unroll
        for (int r = 0; r < 2 * SETS; ++r) {
            const uint4 q = slot.c[r][lane];
            c[r][0] = q.x; c[r][1] = q.y; c[r][2] = q.z; c[r][3] = q.w;
        }
        float d[SETS][4] = {};
        compute_chunk<SETS>(c, w, 2 * (t & 1), xp, d);
#pragma unroll
        for (int k = 0; k < SETS; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[k][j] += d[k][j];
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();                                                 // nothing in flight or unread when the ring is reused
}

__device__ __forceinline__ float silu(float z) { return __fdividef(z, 1.0f + expf(-z)); }

// STORE and SWIGLU.  A warp takes two 16-row sets (STORE: 32 output rows;
// SWIGLU: 16 gate rows and their up rows) and one of `splits` interleaved
// parts of the columns; a block's 4 warps are 4 / splits such row pairs.
// blockIdx.x: (token, slot) pair (dense: group of 8 tokens), fastest, so that
// blocks that share an expert's rows run together and meet in L2.  The block
// of the first pair that names an expert serves every pair that does, 8 per
// pass of its weights; the others leave at once.
template <int FORM>
__global__ void __launch_bounds__(THREADS, BLOCKS) k_nvfp4_gemv(const Params p, int splits)
{
    extern __shared__ __align__(16) uint8_t dyn[];
    Slot<2> *ring = reinterpret_cast<Slot<2> *>(dyn) + (threadIdx.x >> 5) * DEPTH;
    __shared__ float part[WARPS][2][ROWS][COLS];
    __shared__ int list[MAX_PAIRS];
    __shared__ int count;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int chunks = (p.K + 127) / 128;
    const int b = (int)blockIdx.x;
    grid_wait();
    grid_release();
    const int per_block = WARPS / splits;                        // row pairs
    const int rp = (int)blockIdx.y * per_block + warp / splits;  // this warp's
    const int split = warp % splits;
    const int n_rows = FORM == SWIGLU ? p.N / 2 : p.N;           // output rows
    const bool dense = p.idx == nullptr;
    int e = 0, members = 1, first = b;
    bool listed = false;
    unsigned set_bits = 0;                                       // up to 32 pairs: the expert's, as bits
    if (dense) {
        first = b * COLS;
        members = min(COLS, p.pairs - first);
    } else if (p.pairs <= 32) {
        const int mine = lane < p.pairs ? p.idx[lane] : -1;
        e = __shfl_sync(0xffffffffu, mine, b);
        if (e < 0 || e >= p.E) {
            e = -1;                                              // no such expert: zeros, for this pair alone
        } else {
            set_bits = __ballot_sync(0xffffffffu, mine == e);
            if (set_bits & ((1u << b) - 1u)) return;
            members = __popc(set_bits);
        }
    } else {
        e = p.idx[b];
        if (e < 0 || e >= p.E) {
            e = -1;
        } else {
            if (warp == 0) {
                int n = 0;
                bool later = false;
                for (int i0 = 0; i0 < p.pairs; i0 += 32) {
                    const int i = i0 + lane;
                    const bool same = i < p.pairs && p.idx[i] == e;
                    const unsigned m = __ballot_sync(0xffffffffu, same);
                    if (same) list[n + __popc(m & ((1u << lane) - 1u))] = i;
                    n += __popc(m);
                    later = later || __any_sync(0xffffffffu, same && i < b);
                }
                if (lane == 0) count = later ? 0 : n;
            }
            __syncthreads();
            members = count;
            listed = true;
            if (members == 0) return;
        }
    }
    // the pair in column `col` (< members) of this block's products
    auto pair_of = [&](int col) {
        if (listed) return list[col];
        if (members > 1 && set_bits) return (int)__fns(set_bits, 0, col + 1);
        return first + col;
    };
    // STORE: the row pair's two sets are neighbouring tiles; SWIGLU: gate and up
    const int tile0 = FORM == SWIGLU ? rp : 2 * rp, tile1 = FORM == SWIGLU ? rp : 2 * rp + 1;
    for (int m0 = 0; m0 < members; m0 += COLS) {
        float acc[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        float coef = 0.0f;
        if (e >= 0) {
            const int pair = pair_of(min(m0 + g, members - 1));
            const uint8_t *codes = p.codes + e * p.code_stride, *scales = p.scales + e * p.scale_stride;
            const int base1 = FORM == SWIGLU ? n_rows : 0;
            const Set l[2] = {set_of(p, codes, tile0, 0, n_rows), set_of(p, codes, tile1, base1, n_rows)};
            const ScaleWord<2> w(0, lane);                       // the same row for both halves
            const uint8_t *row = scales_of(p, scales, w.k ? tile1 : tile0, w.k ? base1 : 0, n_rows, w.rr);
            const uint8_t *const s[2] = {row, row};
            dot_range<2>(ring, l, s, p.x + (int64_t)((uint32_t)pair * p.x_mul >> 16) * p.ldx, p.x_wide, split, splits, chunks,
                         p.K, acc);
            coef = 512.0f * p.s_t[e];                            // the operands carry 2^-9
        }
        if (m0 > 0) __syncthreads();                             // the last pass's sums have been read
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            *reinterpret_cast<float2 *>(&part[warp][i][g][2 * t]) = make_float2(coef * acc[i][0], coef * acc[i][1]);
            *reinterpret_cast<float2 *>(&part[warp][i][g + 8][2 * t]) = make_float2(coef * acc[i][2], coef * acc[i][3]);
        }
        __syncthreads();
        // one thread per row and column; sets and row pairs in turn
        static_assert(THREADS == ROWS * COLS, "one output per thread and set");
        const int rr = threadIdx.x & 15, col = threadIdx.x >> 4;
        if (m0 + col < members) {
            const int64_t orow = pair_of(m0 + col);
            for (int j = 0; j < per_block; ++j) {
                const int orp = (int)blockIdx.y * per_block + j;
                float y[2] = {0.0f, 0.0f};
                for (int w = j * splits; w < (j + 1) * splits; ++w) {
                    y[0] += part[w][0][rr][col];
                    y[1] += part[w][1][rr][col];
                }
                if (FORM == SWIGLU) {
                    const int n = tile_row(orp, rr);
                    if (n < n_rows)
                        reinterpret_cast<__nv_bfloat16 *>(p.out)[orow * p.ld_out + n] = __float2bfloat16_rn(silu(y[0]) * y[1]);
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int n = tile_row(2 * orp + i, rr);
                        if (n < n_rows) reinterpret_cast<float *>(p.out)[orow * p.ld_out + n] = y[i];
                    }
                }
            }
        }
    }
}

// COMBINE: blockIdx.x a token, its (expert, chunk) pairs dealt to the warps in
// order; one launch, nothing shared between tokens.
__global__ void __launch_bounds__(32 * COMBINE_WARPS, 2) k_nvfp4_gemv_combine(const Params p)
{
    extern __shared__ __align__(16) uint8_t dyn[];
    Slot<1> *ring = reinterpret_cast<Slot<1> *>(dyn) + (threadIdx.x >> 5) * DEPTH;
    __shared__ float part[COMBINE_WARPS][ROWS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int tile = blockIdx.y;
    const int chunks = (p.K + 127) / 128;
    const bool dense = p.idx == nullptr;
    grid_wait();
    grid_release();
    float tot[2] = {0, 0};
    const int units = p.k_r * chunks;
    const int per = (units + COMBINE_WARPS - 1) / COMBINE_WARPS;
    int u = warp * per;
    const int u_end = min(u + per, units);
    while (u < u_end) {
        const int j = u / chunks, ch = u - j * chunks;
        const int ch_end = min(chunks, ch + (u_end - u));
        const int64_t pair = (int64_t)blockIdx.x * p.k_r + j;
        const int e = dense ? 0 : p.idx[pair];
        if (e >= 0 && e < p.E) {
            const Set l[1] = {set_of(p, p.codes + e * p.code_stride, tile, 0, p.N)};
            const uint8_t *const s[1] = {scales_of(p, p.scales + e * p.scale_stride, tile, 0, p.N, ScaleWord<1>(0, lane).rr)};
            float acc[1][4] = {{0, 0, 0, 0}};
            dot_range<1>(ring, l, s, p.x + pair * p.ldx, p.x_wide, ch, 1, ch_end, p.K, acc);
            const float coef = 512.0f * (p.gate ? p.gate[pair] * p.s_t[e] : p.s_t[e]);
            tot[0] += coef * acc[0][0];                          // column 0 is lane t = 0's
            tot[1] += coef * acc[0][2];
        }
        u += ch_end - ch;
    }
    if (t == 0) {
        part[warp][g] = tot[0];
        part[warp][g + 8] = tot[1];
    }
    __syncthreads();
    if (threadIdx.x < ROWS) {
        const int n = tile_row(tile, threadIdx.x);
        if (n < p.N) {
            float y = 0.0f;
#pragma unroll
            for (int w = 0; w < COMBINE_WARPS; ++w) y += part[w][threadIdx.x];
            reinterpret_cast<float *>(p.out)[(int64_t)blockIdx.x * p.ld_out + n] = y;
        }
    }
}

// out[t, n] = sum_j gate[t, j] y[t k_r + j, n], in slot order; a slot whose
// expert does not exist takes no part, whatever its gate holds (as in the
// one-launch form).
__global__ void __launch_bounds__(THREADS) k_gemv_combine(const float *y, const float *gate,
                                                          const int32_t *idx, int E, int k_r, int64_t N,
                                                          float *__restrict__ out, int64_t ld_out)
{
    const int64_t n = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    const int64_t t = blockIdx.y;
    grid_wait();
    grid_release();
    if (n >= N) return;
    float s = 0.0f;
    for (int j = 0; j < k_r; ++j) {
        const int64_t pair = t * k_r + j;
        if (idx && (idx[pair] < 0 || idx[pair] >= E)) continue;
        s += (gate ? gate[pair] : 1.0f) * y[pair * N + n];
    }
    out[t * ld_out + n] = s;
}

// Opt the kernel in to its ring's shared memory (once per device).
template <auto KERNEL>
static nvfp4_status allow_ring(size_t bytes)
{
    static std::once_flag once[64];
    static cudaError_t err[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return check_launch("k_nvfp4_gemv: device");
    std::call_once(once[dev], [&] { err[dev] = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes); });
    if (err[dev] != cudaSuccess) return set_error(NVFP4_ERR_CUDA, "k_nvfp4_gemv: smem attribute: %s", cudaGetErrorString(err[dev]));
    return NVFP4_OK;
}

// Column splits of a row pair: the fewest that give every SM two blocks (or one
// chunk of 128 columns per warp).  Measured without splits, for one, two and four
// blocks an SM: dense 4096 x 4096, one row, 19.0, 6.7, 6.7, 6.7 us; top-8 gate/up
// 1536 x 2048 of one token 11.4, 9.6, 9.3, 9.3, of two 16.3, 16.3, 15.1, 13.9, of
// four 25.9, 25.9, 25.9, 21.8; top-8 of 4096 x 1536, one token, 13.4, 13.4, 12.7,
// 13.7.
static int column_splits(int64_t units, int64_t row_pairs, int64_t K)
{
    int s = 1;
    while (s < WARPS && units * row_pairs * s < (int64_t)num_sms() * 2 * WARPS && (int64_t)s * 128 < K) s *= 2;
    return s;
}

// The combine form shares weights between tokens (partial rows in the
// workspace, a second launch) when the tokens name experts more than once.
// Measured in one launch and shared, top-8 of 128 experts, 4096 x 1536: 2 tokens
// 23.3 and 23.9 us, 4 41.9 and 37.6, 5 51.4 and 44.1, 16 145 and 93; 2048 x 768: 2
// tokens 7.3 and 11.2, 4 13.1 and 15.8, 5 17.0 and 16.8, 16 42 and 34.  With few
// experts the second launch shows: top-2 of 8, 2048 x 768, 2 tokens 3.9 and 6.6, 8
// tokens 10.6 and 10.3.
static bool grouped_combine(int64_t T, int32_t E, int32_t k_r) { return T > 1 && T * k_r > E / 4; }

}  // namespace gemv
}  // namespace nvfp4

using namespace nvfp4;

extern "C" size_t moe_nvfp4_gemv_workspace_size(int64_t T, int64_t N, int32_t E, int32_t k_r, int32_t epilogue)
{
    using namespace nvfp4::gemv;
    if (T <= 0 || N <= 0 || E <= 0 || k_r <= 0 || epilogue != MOE_EPI_COMBINE_F32 || !grouped_combine(T, E, k_r)) return 0;
    return (size_t)std::min<int64_t>(T, MAX_PAIRS / k_r) * (size_t)k_r * (size_t)N * 4;
}

extern "C" nvfp4_status moe_nvfp4_gemv(const void *x_dev, int64_t T, int64_t ldx, const uint8_t *codes_dev,
                                       const uint8_t *scales_dev, const float *s_t_dev, int64_t N, int64_t K,
                                       int32_t E, const int32_t *expert_idx_dev, int32_t k_r, int32_t epilogue,
                                       const float *gate_dev, void *out_dev, int64_t ld_out, void *workspace,
                                       size_t workspace_bytes, void *stream)
{
    using namespace nvfp4::gemv;
    NVFP4_REQUIRE(epilogue == MOE_EPI_STORE_F32 || epilogue == MOE_EPI_SWIGLU_BF16 || epilogue == MOE_EPI_COMBINE_F32,
                  NVFP4_ERR_INVALID_ARG, "moe_nvfp4_gemv: bad epilogue");
    NVFP4_REQUIRE(T >= 0, NVFP4_ERR_INVALID_ARG, "moe_nvfp4_gemv: negative size");
    NVFP4_REQUIRE(E >= 1 && k_r >= 1 && k_r <= 32, NVFP4_ERR_UNSUPPORTED_SHAPE,
                  "moe_nvfp4_gemv: need E >= 1 and 1 <= k_r <= 32");
    NVFP4_REQUIRE(expert_idx_dev || (k_r == 1 && E == 1), NVFP4_ERR_INVALID_ARG,
                  "moe_nvfp4_gemv: without expert_idx there is one weight (E = 1, k_r = 1)");
    NVFP4_REQUIRE(N >= 1 && K >= 64 && K % 64 == 0 && K < (1ll << 24), NVFP4_ERR_UNSUPPORTED_SHAPE,
                  "moe_nvfp4_gemv: N must be positive and K a positive multiple of 64 below 2^24 (N=%lld, K=%lld)", (long long)N,
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
    NVFP4_REQUIRE(aligned16(x_dev) && aligned16(codes_dev) && aligned16(scales_dev) &&
                  reinterpret_cast<uintptr_t>(out_dev) % (epilogue == MOE_EPI_SWIGLU_BF16 ? 2 : 4) == 0,
                  NVFP4_ERR_ALIGNMENT,
                  "moe_nvfp4_gemv: x, codes and scales must be 16-byte aligned, out aligned to its elements");
    const size_t need = moe_nvfp4_gemv_workspace_size(T, N, E, k_r, epilogue);
    NVFP4_REQUIRE(need == 0 || (workspace && workspace_bytes >= need && aligned16(workspace)), NVFP4_ERR_WORKSPACE,
                  "moe_nvfp4_gemv: workspace of %zu bytes required", need);
    cudaStream_t st = (cudaStream_t)stream;
    const bool combine = epilogue == MOE_EPI_COMBINE_F32, dense = expert_idx_dev == nullptr;
    // the pair list holds MAX_PAIRS: longer batches run in slices of tokens
    const int64_t slice = MAX_PAIRS / k_r;
    const int64_t x_rows = combine ? k_r : 1;                   // rows of x per token
    for (int64_t t0 = 0; t0 < T; t0 += slice) {
        const int64_t tn = std::min(slice, T - t0);
        Params p;
        p.x = reinterpret_cast<const __nv_bfloat16 *>(x_dev) + t0 * x_rows * ldx;
        p.ldx = ldx;
        p.codes = codes_dev;
        p.scales = scales_dev;
        p.s_t = s_t_dev;
        p.N = (int32_t)N;
        p.K = (int32_t)K;
        p.E = E;
        p.code_stride = N * (K / 2);
        p.scale_stride = sf_bytes(N, K);
        p.idx = dense ? nullptr : expert_idx_dev + t0 * k_r;
        p.pairs = (int)(tn * k_r);
        p.k_r = k_r;
        // pair / k_r for pairs below MAX_PAIRS: exact because 1024 * 32 < 65536
        p.x_mul = combine || k_r == 1 ? 65536u : 65536u / (uint32_t)k_r + 1u;
        p.gate = gate_dev ? gate_dev + t0 * k_r : nullptr;
        p.out = epilogue == MOE_EPI_SWIGLU_BF16
                    ? (void *)(reinterpret_cast<__nv_bfloat16 *>(out_dev) + t0 * k_r * ld_out)
                    : (void *)(reinterpret_cast<float *>(out_dev) + (combine ? t0 : t0 * k_r) * ld_out);
        p.ld_out = ld_out;
        p.x_wide = reinterpret_cast<uintptr_t>(p.x) % 32 == 0 && ldx % 16 == 0;
        const int64_t units = dense ? (tn + COLS - 1) / COLS : tn * k_r;
        const int64_t row_pairs = epilogue == MOE_EPI_SWIGLU_BF16 ? tiles : tiles / 2;
        const int splits = column_splits(units, row_pairs, K);
        const dim3 per_pair((unsigned)units, (unsigned)((row_pairs * splits + WARPS - 1) / WARPS));
        constexpr size_t RING1 = sizeof(Slot<1>) * DEPTH * COMBINE_WARPS, RING2 = sizeof(Slot<2>) * DEPTH * WARPS;
        nvfp4_status rc = combine && need == 0 ? allow_ring<k_nvfp4_gemv_combine>(RING1)
                          : epilogue == MOE_EPI_SWIGLU_BF16 ? allow_ring<k_nvfp4_gemv<SWIGLU>>(RING2)
                                                            : allow_ring<k_nvfp4_gemv<STORE>>(RING2);
        if (rc != NVFP4_OK) return rc;
        if (combine && need == 0) {
            launch_overlapped(k_nvfp4_gemv_combine, dim3((unsigned)tn, (unsigned)tiles), 32 * COMBINE_WARPS, RING1, st, p);
        } else if (combine) {
            float *out = reinterpret_cast<float *>(p.out);
            p.out = workspace;
            p.ld_out = N;
            launch_overlapped(k_nvfp4_gemv<STORE>, per_pair, THREADS, RING2, st, p, splits);
            if (check_launch("k_nvfp4_gemv") != NVFP4_OK) return NVFP4_ERR_CUDA;
            launch_overlapped(k_gemv_combine, dim3((unsigned)((N + THREADS - 1) / THREADS), (unsigned)tn), THREADS, 0, st,
                              reinterpret_cast<const float *>(workspace), p.gate, p.idx, p.E, (int)k_r, N, out, ld_out);
        } else if (epilogue == MOE_EPI_SWIGLU_BF16) {
            launch_overlapped(k_nvfp4_gemv<SWIGLU>, per_pair, THREADS, RING2, st, p, splits);
        } else {
            launch_overlapped(k_nvfp4_gemv<STORE>, per_pair, THREADS, RING2, st, p, splits);
        }
        if (check_launch("k_nvfp4_gemv") != NVFP4_OK) return NVFP4_ERR_CUDA;
    }
    return NVFP4_OK;
}
