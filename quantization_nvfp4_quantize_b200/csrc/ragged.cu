// ragged.cu -- products grouped by expert over ragged row segments, and their
// gradients, on the sm_100a tensor cores (BF16 operands, f32 accumulation).
//
// Expert e owns rows [off[e], off[e+1]) of the routed row order; segments have
// any length, zero included, and are not padded.
//   FWD    out[r, n]  = sum_k a[r, k] w_e[n, k]
//   DGRAD  out[r, k]  = sum_n g[r, n] w_e[n, k]
//   WGRAD  dw_e[n, k] = sum_{r in e} g[r, n] a[r, k]
//   KEPT   WGRAD with a kept in 8 bits (E4M3, one power-of-two scale per 32
//          columns of a row) and named by a row index
//
// Bound by the tensor pipe for segments of a few hundred rows and more, by the
// weights' bytes below that (WGRAD: by the f32 result's bytes).
//
// A cluster of two CTAs computes 256 x 256 tiles with tcgen05 .cta_group::2:
// each CTA stages 128 rows of the M-side operand and 128 of the N-side one,
// 64 deep, 32 KB a stage, in a ring of stages; the even CTA issues the MMAs.
// TMEM holds two 256-column accumulators, so one tile's epilogue runs under
// the next tile's MMAs.
//
// The tensor core takes an operand either way round (instruction descriptor
// bits 15 / 16), so no operand is ever transposed in memory:
//   K-major    the reduction runs along a row: a 128-row x 64-column TMA box;
//   MN-major   the reduction runs down the rows: two 64-column x 64-row boxes.
// FWD is K x K, DGRAD K x MN, WGRAD MN x MN.
//
// Ragged reduction (WGRAD): a segment's last stage also holds rows of the next
// expert, or rows nobody wrote.  Zeroing one operand would not do (0 * NaN), so
// that stage lands on a barrier of its own CTA, warp 3 zeroes the surplus rows
// of both operands in shared memory and only then reports the stage to the
// MMA issuer.  Ragged rows (FWD, DGRAD) need nothing: a surplus row only makes
// an accumulator row that the epilogue does not store.
//
// KEPT: one converter warp per slot of the stage ring: 64 rows x 128 columns of
// codes from global memory to registers (before the slot is free), to BF16
// (exact), to the slot in the MMA's swizzle.  Not more warps than slots: a
// warp further ahead could find its slot two uses behind, where the parity of
// the slot's barrier looks like a free one.  The codes are read at their own size
// and never expanded in global memory.
//
// WGRAD with few output tiles splits every segment's rows over several tiles:
// f32 partial results in the workspace, added in split order by a second
// kernel (no atomics: the result does not change from run to run).
//
// Warps: 0, 2 TMA producers; 1 MMA issuer; 3 the surplus-row fixer; 4..11
// epilogue; 12..17 converters (KEPT).  Every mbarrier wait is bounded (1 s);
// on expiry the kernel records NVFP4_ERR_TIMEOUT, its roles stop, copies in
// flight get 1 ms to land, MMAs are drained and TMEM is freed.
#include "common.cuh"
#include "ptx.cuh"

#include <cuda.h>
#include <algorithm>
#include <mutex>

namespace nvfp4 {
namespace ragged {

constexpr int TILE = 256;                        // both output dimensions of a pair's tile
constexpr int BK = 64;                           // reduction depth of a stage
constexpr int STAGES = 6;
constexpr uint32_t OPER_BYTES = 128 * BK * 2;    // one operand of one CTA: 16 KB
constexpr uint32_t BOX_BYTES = 64 * BK * 2;      // one MN-major box: 8 KB
constexpr uint32_t STAGE_BYTES = 2 * OPER_BYTES;
constexpr uint32_t SMEM = STAGES * STAGE_BYTES + 1024 /*align*/ + 4096 /*barriers, offsets*/;
static_assert(SMEM <= 232448, "shared memory budget");
constexpr int EPI_WARPS = 8, EPI_WARP0 = 4, CONV_WARP0 = 12, CONV_WARPS = STAGES;
constexpr int PROD_A_WARP = 0, MMA_WARP = 1, PROD_B_WARP = 2, FIX_WARP = 3;
constexpr uint32_t TMEM_COLS = 512;
constexpr int MAX_E = 256;
constexpr uint64_t TIMEOUT_NS = 1000000000ull;

enum Mode { FWD = 0, DGRAD = 1, WGRAD = 2, KEPT = 3 };

template <int MODE>
struct Cfg {
    static constexpr bool RAGGED_K = MODE == WGRAD || MODE == KEPT;
    static constexpr bool A_MN = RAGGED_K;                   // M-side operand MN-major
    static constexpr bool B_MN = MODE != FWD;                // N-side operand MN-major
    static constexpr int THREADS = MODE == KEPT ? 384 + 32 * CONV_WARPS : 384;
    // arrivals per stage: both producers; KEPT: the producer's two, one converter warp per CTA
    static constexpr uint32_t FULL_COUNT = MODE == KEPT ? 4 : 2;
};

struct Params {
    int64_t M;                 // rows of the routed order
    int64_t out_m, out_n;      // WGRAD: N x K of one expert's gradient; else out_n = output columns
    int64_t red;               // reduction length (FWD: K, DGRAD: N)
    int E;
    int n_tiles;               // tiles along the N side
    int m_tiles;               // WGRAD: tiles along the M side
    int splits;                // WGRAD: row splits of every segment
    const int32_t *offsets;
    void *out;
    int64_t ld_out;
    int out_f32;
    int accumulate;            // WGRAD: add to out
    int vec_bytes;             // widest store that out's base and rows allow: 32, 16 or 0 (element by element)
    // KEPT
    const uint8_t *codes;
    int64_t ld_codes;
    const uint8_t *scales;
    int64_t ld_scales;
    const int32_t *a_rows;     // or null: row r itself
    int64_t T;                 // kept rows
    int32_t *dev_status;
};

struct Shared {
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t raw[STAGES];      // ragged last stages land here first (own CTA)
    uint64_t tmem_full[2];
    uint64_t tmem_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    int off[MAX_E + 1];        // segment bounds, made monotone and in [0, M]
    int tiles[MAX_E + 1];      // FWD / DGRAD: row tiles before expert e
};

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag, int32_t *dev_status,
                                         bool ignore_abort = false)
{
    uint64_t t0 = 0;
    for (uint32_t i = 0;; ++i) {
        if (ptx::mbar_try_wait_cluster(bar, parity)) return true;
        if ((i & 63u) == 63u) {
            if (!ignore_abort && *abort_flag) return false;
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            else if (now - t0 > TIMEOUT_NS) {
                *abort_flag = 1;
                report_status(dev_status, NVFP4_ERR_TIMEOUT);
                return false;
            }
        }
    }
}

// What a tile covers.
struct Tile {
    int e;
    int64_t m0, m_end;         // M-side start and end (rows, or rows of w for WGRAD)
    int64_t n0;
    int r0, r1;                // WGRAD: its rows
    int stages;                // reduction stages (0: WGRAD of an empty segment)
    int split;
};

template <int MODE>
__device__ __forceinline__ Tile tile_at(const Params &p, const Shared *sh, int64_t t)
{
    Tile w;
    if (Cfg<MODE>::RAGGED_K) {
        const int per = p.m_tiles * p.n_tiles * p.splits;
        w.e = (int)(t / per);
        int rem = (int)(t - (int64_t)w.e * per);
        w.split = rem / (p.m_tiles * p.n_tiles);
        rem -= w.split * (p.m_tiles * p.n_tiles);
        const int mt = rem / p.n_tiles;
        w.m0 = (int64_t)mt * TILE;
        w.m_end = p.out_m;
        w.n0 = (int64_t)(rem - mt * p.n_tiles) * TILE;
        const int lo = sh->off[w.e], hi = sh->off[w.e + 1];
        // whole stages per split, so that only a segment's last stage is ragged
        const int chunk = ((hi - lo + p.splits - 1) / p.splits + BK - 1) / BK * BK;
        const int64_t r0 = (int64_t)lo + (int64_t)w.split * chunk;
        w.r0 = (int)min((int64_t)hi, r0);
        w.r1 = (int)min((int64_t)hi, r0 + chunk);
        w.stages = (w.r1 - w.r0 + BK - 1) / BK;
    } else {
        const int rt = (int)(t / p.n_tiles);
        int lo = 0, hi = p.E;                        // tiles[lo] <= rt < tiles[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sh->tiles[mid] <= rt) lo = mid; else hi = mid;
        }
        w.e = lo;
        w.m0 = (int64_t)sh->off[lo] + (int64_t)(rt - sh->tiles[lo]) * TILE;
        w.m_end = sh->off[lo + 1];
        w.n0 = (t - (int64_t)rt * p.n_tiles) * TILE;
        w.r0 = w.r1 = 0;
        w.split = 0;
        w.stages = (int)((p.red + BK - 1) / BK);
    }
    return w;
}

// E4M3 pair codes -> two BF16 values times a scale pair: the code's exponent
// and mantissa bits read as value * 2^-120 in a BF16, its zero exponent
// (subnormals) included; both multiplications are exact.
__device__ __forceinline__ uint32_t kept_pair(uint32_t t, uint32_t scale2)
{
    const uint32_t v = ((t >> 4) & 0x07F007F0u) | (t & 0x80008000u);
    const uint32_t up = 0x7B807B80u;                 // 2^120
    __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&v), *reinterpret_cast<const __nv_bfloat162 *>(&up));
    r = __hmul2(r, *reinterpret_cast<const __nv_bfloat162 *>(&scale2));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// 2^(s - 127) in both halves; NaN for s = 255.
__device__ __forceinline__ uint32_t kept_scale(uint32_t s)
{
    return s == 255u ? 0x7FC07FC0u : s == 0u ? 0x00400040u : s * 0x00800080u;
}

// 16 codes of which `left` are inside the row.
__device__ __forceinline__ uint4 load_codes(const uint8_t *src, int64_t left)
{
    if (left >= 16) return __ldg(reinterpret_cast<const uint4 *>(src));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (i < left) w[i >> 2] |= (uint32_t)src[i] << (8 * (i & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int MODE>
__global__ void __launch_bounds__(Cfg<MODE>::THREADS, 1)
k_ragged_gemm(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, const Params p)
{
    using C = Cfg<MODE>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *stage_base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Shared *sh = reinterpret_cast<Shared *>(stage_base + STAGES * STAGE_BYTES);
    volatile int *abort_flag = &sh->abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;
    const int unit = (int)(blockIdx.x >> 1), n_units = (int)(gridDim.x >> 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh->full[s]), C::FULL_COUNT);
            ptx::mbar_init(ptx::smem_u32(&sh->empty[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh->raw[s]), MODE == KEPT ? 1 : 2);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_u32(&sh->tmem_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh->tmem_empty[i]), 2 * EPI_WARPS);
        }
        ptx::mbar_init(ptx::smem_u32(&sh->drain), 1);
        sh->abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 0) {
        ptx::tmem_alloc_pair(ptx::smem_u32(&sh->tmem_base), TMEM_COLS);
        ptx::tmem_relinquish_pair();
    }
    if (warp == FIX_WARP) {
        // lane l takes bounds 8l .. 8l + 7: running maximum, clamped to [0, M]
        // (a bad table can then give no row outside the tensors), and the
        // number of row tiles before each expert
        constexpr int PER = MAX_E / 32;
        int v[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane * PER + i;
            const int raw = e <= p.E ? p.offsets[e] : 0;
            v[i] = (int)min(max((int64_t)raw, (int64_t)0), p.M);
            if (i > 0) v[i] = max(v[i], v[i - 1]);
        }
        int last = p.E == MAX_E ? (int)min(max((int64_t)p.offsets[MAX_E], (int64_t)0), p.M) : 0;
        int m = v[PER - 1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, m, o);
            if (lane >= o) m = max(m, u);
        }
        int before = __shfl_up_sync(0xffffffffu, m, 1);
        if (lane == 0) before = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = max(v[i], before);
        last = max(last, __shfl_sync(0xffffffffu, m, 31));
        int nxt = __shfl_down_sync(0xffffffffu, v[0], 1);
        if (lane == 31) nxt = last;
        int cnt[PER], sum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane * PER + i;
            const int len = (i + 1 < PER ? v[i + 1 < PER ? i + 1 : i] : nxt) - v[i];
            cnt[i] = e < p.E ? (len + TILE - 1) / TILE : 0;
            sum += cnt[i];
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        int pre = incl - sum;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane * PER + i;
            if (e <= p.E) { sh->off[e] = v[i]; sh->tiles[e] = pre; }
            pre += cnt[i];
        }
        if (lane == 31 && p.E == MAX_E) { sh->off[MAX_E] = last; sh->tiles[MAX_E] = incl; }
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();                   // barriers of both CTAs initialized before any remote use
    ptx::tc_fence_after();
    const uint32_t tmem = sh->tmem_base;
    const int64_t total = C::RAGGED_K ? (int64_t)p.E * p.m_tiles * p.n_tiles * p.splits
                                      : (int64_t)sh->tiles[p.E] * p.n_tiles;

    if (warp == PROD_A_WARP || (warp == PROD_B_WARP && MODE != KEPT)) {
        if (lane == 0) {
            // ------------------------------------------------- producers
            const bool role_a = warp == PROD_A_WARP;
            const CUtensorMap *tm = role_a ? &tm_a : &tm_b;
            ptx::prefetch_tmap(tm);
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            for (int64_t t = unit; ok && t < total; t += n_units) {
                const Tile w = tile_at<MODE>(p, sh, t);
                // this CTA's 128 of the tile's 256 rows / columns
                const int mn = (int)((role_a ? w.m0 : w.n0) + rank * 128);
                for (int kb = 0; kb < w.stages; ++kb) {
                    if (!wait_bar(ptx::smem_u32(&sh->empty[stage]), phase ^ 1u, abort_flag, p.dev_status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = ptx::smem_u32(stage_base + stage * STAGE_BYTES + (role_a ? 0 : OPER_BYTES));
                    const uint32_t fb = ptx::smem_u32(&sh->full[stage]);
                    if (C::RAGGED_K) {
                        const int row = w.r0 + kb * BK;
                        if (row + BK > w.r1) {
                            // ragged: land in this CTA, the fixer reports it
                            const uint32_t rb = ptx::smem_u32(&sh->raw[stage]);
                            ptx::mbar_arrive_expect_tx(rb, OPER_BYTES);
                            ptx::tma_load_2d(dst, tm, mn, row, rb);
                            ptx::tma_load_2d(dst + BOX_BYTES, tm, mn + 64, row, rb);
                        } else {
                            const uint32_t lfb = ptx::mapa_shared(fb, 0);
                            if (leader) {
                                ptx::mbar_arrive_expect_tx(fb, 2 * OPER_BYTES);
                                if (MODE == KEPT) ptx::mbar_arrive(fb);
                            }
                            ptx::tma_load_2d_pair(dst, tm, mn, row, lfb);
                            ptx::tma_load_2d_pair(dst + BOX_BYTES, tm, mn + 64, row, lfb);
                        }
                    } else {
                        const uint32_t lfb = ptx::mapa_shared(fb, 0);
                        if (leader) ptx::mbar_arrive_expect_tx(fb, 2 * OPER_BYTES);
                        if (role_a) {
                            ptx::tma_load_2d_pair(dst, tm, kb * BK, mn, lfb);
                        } else if (C::B_MN) {
                            ptx::tma_load_3d_pair(dst, tm, mn, kb * BK, w.e, lfb);
                            ptx::tma_load_3d_pair(dst + BOX_BYTES, tm, mn + 64, kb * BK, w.e, lfb);
                        } else {
                            ptx::tma_load_3d_pair(dst, tm, kb * BK, mn, w.e, lfb);
                        }
                    }
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            if (!ok) {
                // copies in flight land before the CTA's memory is released
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 1000000ull) { }
            }
        }
        __syncwarp();
    } else if (warp == MMA_WARP) {
        if (lane == 0 && leader) {
            // ----------------------------------------------- MMA issuer
            const uint32_t idesc = ptx::idesc_bf16(TILE, TILE) | (C::A_MN ? 1u << 15 : 0u) | (C::B_MN ? 1u << 16 : 0u);
            uint32_t stage = 0, phase = 0;
            bool ok = true, issued = false;
            int iter = 0;
            for (int64_t t = unit; ok && t < total; t += n_units) {
                const Tile w = tile_at<MODE>(p, sh, t);
                if (w.stages == 0) continue;
                const int acc = iter & 1;
                if (!wait_bar(ptx::smem_u32(&sh->tmem_empty[acc]), (uint32_t)((iter >> 1) & 1) ^ 1u, abort_flag,
                              p.dev_status)) {
                    ok = false;
                    break;
                }
                ++iter;
                ptx::tc_fence_after();
                const uint32_t d = tmem + (uint32_t)acc * TILE;
                const int64_t len = C::RAGGED_K ? (int64_t)(w.r1 - w.r0) : p.red;
                for (int kb = 0; kb < w.stages; ++kb) {
                    if (!wait_bar(ptx::smem_u32(&sh->full[stage]), phase, abort_flag, p.dev_status)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t sa = ptx::smem_u32(stage_base + stage * STAGE_BYTES), sb = sa + OPER_BYTES;
                    const int64_t left = len - (int64_t)kb * BK;
                    const int steps = left >= BK ? BK / 16 : (int)((left + 15) / 16);
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk) {
                        if (kk < steps) {
                            // K-major: 32 bytes along the row; MN-major: 16 rows of 128 bytes
                            const uint64_t ad = C::A_MN ? ptx::make_sdesc(sa + 2048 * kk, BOX_BYTES, 1024, 2)
                                                        : ptx::make_sdesc(sa + 32 * kk, 16, 1024, 2);
                            const uint64_t bd = C::B_MN ? ptx::make_sdesc(sb + 2048 * kk, BOX_BYTES, 1024, 2)
                                                        : ptx::make_sdesc(sb + 32 * kk, 16, 1024, 2);
                            ptx::mma_bf16_pair(d, ad, bd, idesc, (kb | kk) != 0);
                        }
                    }
                    ptx::tc_commit_pair_mc(ptx::smem_u32(&sh->empty[stage]), 3);
                    issued = true;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
                if (ok) ptx::tc_commit_pair_mc(ptx::smem_u32(&sh->tmem_full[acc]), 3);
            }
            if (!ok && issued) {
                // let every issued MMA finish before TMEM is released
                ptx::tc_commit_pair_mc(ptx::smem_u32(&sh->drain), 1);
                wait_bar(ptx::smem_u32(&sh->drain), 0, abort_flag, p.dev_status, true);
            }
        }
        __syncwarp();
    } else if (warp == FIX_WARP) {
        if (C::RAGGED_K) {
            // --------------------- zero the surplus rows of ragged stages
            uint32_t stage = 0, parity = 0;             // one parity bit per stage's raw barrier
            for (int64_t t = unit; t < total; t += n_units) {
                const Tile w = tile_at<MODE>(p, sh, t);
                if (w.stages == 0) continue;
                const uint32_t s = (stage + (uint32_t)(w.stages - 1)) % STAGES;
                stage = (s + 1) % STAGES;
                const int rows = (w.r1 - w.r0) - (w.stages - 1) * BK;
                if (rows == BK) continue;
                bool ok = true;
                if (lane == 0) ok = wait_bar(ptx::smem_u32(&sh->raw[s]), (parity >> s) & 1u, abort_flag, p.dev_status);
                if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) break;
                __syncwarp();
                parity ^= 1u << s;
                uint8_t *base = stage_base + s * STAGE_BYTES;
                constexpr int BOXES = MODE == KEPT ? 2 : 4;          // the converters zero their own operand
                // 128-byte rows `rows`..63 of each box; the swizzle stays inside a row
                for (int i = lane; i < (BK - rows) * 8; i += 32) {
#pragma unroll
                    for (int b = 0; b < BOXES; ++b)
                        *reinterpret_cast<uint4 *>(base + b * BOX_BYTES + rows * 128 + i * 16) = make_uint4(0, 0, 0, 0);
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_u32(&sh->full[s]), 0));
            }
        }
    } else if (warp >= EPI_WARP0 && warp < EPI_WARP0 + EPI_WARPS) {
        // --------------------------------------------------- epilogue
        const int q = warp & 3, half = (warp - EPI_WARP0) >> 2;
        const int row_in_tile = (int)rank * 128 + q * 32 + lane;
        int iter = 0;
        for (int64_t t = unit; t < total; t += n_units) {
            const Tile w = tile_at<MODE>(p, sh, t);
            const bool empty_sum = w.stages == 0;
            if (empty_sum && p.accumulate) continue;
            const int acc = iter & 1;
            if (!empty_sum) {
                bool ok = true;
                if (lane == 0)
                    ok = wait_bar(ptx::smem_u32(&sh->tmem_full[acc]), (uint32_t)((iter >> 1) & 1), abort_flag,
                                  p.dev_status);
                if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) break;
                __syncwarp();
                ++iter;
                ptx::tc_fence_after();
            }
            const uint32_t src = tmem + (uint32_t)acc * TILE + (uint32_t)half * 128 + ((uint32_t)(q * 32) << 16);
            const int64_t r = w.m0 + row_in_tile;
            const bool live = r < w.m_end;
            const int64_t orow = C::RAGGED_K ? ((int64_t)w.split * p.E + w.e) * p.out_m + r : r;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t v[32];
                __syncwarp();                            // lanes without a row rejoin before the collective load
                if (!empty_sum) {
                    ptx::tmem_ld_32x32b_x32(src + c * 32, v);
                    ptx::tmem_ld_wait();
                    if (c == 3) {
                        // the accumulator is free once both CTAs' warps have read it
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_u32(&sh->tmem_empty[acc]), 0));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0;
                }
                const int64_t col = w.n0 + half * 128 + c * 32;
                if (!live || col >= p.out_n) continue;
                const int64_t left = p.out_n - col;
                if (p.out_f32) {
                    float *dst = reinterpret_cast<float *>(p.out) + orow * p.ld_out + col;
                    if (p.vec_bytes && left >= 32) {
                        if (C::RAGGED_K && p.accumulate) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float4 o = *reinterpret_cast<const float4 *>(dst + 4 * i);
                                v[4 * i] = __float_as_uint(__uint_as_float(v[4 * i]) + o.x);
                                v[4 * i + 1] = __float_as_uint(__uint_as_float(v[4 * i + 1]) + o.y);
                                v[4 * i + 2] = __float_as_uint(__uint_as_float(v[4 * i + 2]) + o.z);
                                v[4 * i + 3] = __float_as_uint(__uint_as_float(v[4 * i + 3]) + o.w);
                            }
                        }
                        if (p.vec_bytes == 32) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) ptx::st_v8(dst + 8 * i, &v[8 * i]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                *reinterpret_cast<uint4 *>(dst + 4 * i) =
                                    make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < left)
                                dst[i] = C::RAGGED_K && p.accumulate ? dst[i] + __uint_as_float(v[i])
                                                                     : __uint_as_float(v[i]);
                    }
                } else {
                    __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(p.out) + orow * p.ld_out + col;
                    if (p.vec_bytes && left >= 32) {
                        uint32_t o[16];
                        if (C::RAGGED_K && p.accumulate) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint4 old = *reinterpret_cast<const uint4 *>(dst + 8 * i);
                                const uint32_t u[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    v[8 * i + 2 * j] = __float_as_uint(__uint_as_float(v[8 * i + 2 * j]) + bf16lo(u[j]));
                                    v[8 * i + 2 * j + 1] =
                                        __float_as_uint(__uint_as_float(v[8 * i + 2 * j + 1]) + bf16hi(u[j]));
                                }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[i] = pack_bf16(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                        if (p.vec_bytes == 32) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) ptx::st_v8(dst + 16 * i, &o[8 * i]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                *reinterpret_cast<uint4 *>(dst + 8 * i) =
                                    make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < left) {
                                float x = __uint_as_float(v[i]);
                                if (C::RAGGED_K && p.accumulate) x += __bfloat162float(dst[i]);
                                dst[i] = __float2bfloat16_rn(x);
                            }
                    }
                }
            }
        }
    } else if (MODE == KEPT && warp >= CONV_WARP0) {
        // -------------------------------------------------- converters
        // Warp w fills slot w: stages w, w + STAGES, ... of this CTA's sequence.  Lane
        // layout of a 16-byte chunk (16 codes): 4 rows x 8 chunks a step, in
        // an order whose shared stores touch every bank once.
        const int cw = warp - CONV_WARP0;
        const int chunk = (lane & 3) + 4 * ((lane >> 3) & 1);
        const int rsub = ((lane >> 2) & 1) + 2 * (lane >> 4);
        const uint32_t box = (uint32_t)(chunk >> 2) * BOX_BYTES;
        const int q0 = 2 * (chunk & 3);
        uint32_t seq = 0, ph = 0;
        bool ok = true;
        for (int64_t t = unit; ok && t < total; t += n_units) {
            const Tile w = tile_at<MODE>(p, sh, t);
            const int64_t col0 = w.n0 + rank * 128, col = col0 + chunk * 16;
            const bool col_ok = col < p.out_n;
            // seq: the slot of the tile's first stage
            for (int kb = (cw + CONV_WARPS - (int)seq) % CONV_WARPS; kb < w.stages; kb += CONV_WARPS) {
                const uint32_t s = (uint32_t)cw;
                uint8_t *dst = stage_base + s * STAGE_BYTES + OPER_BYTES + box;
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf) {
                    // 32 rows: lane l looks row l up, the codes then go 8 chunks a lane
                    const int r = w.r0 + kb * BK + hf * 32 + lane;
                    int64_t src = -1;
                    uint32_t sw = 0;
                    if (r < w.r1) {
                        src = p.a_rows ? (int64_t)p.a_rows[r] : (int64_t)r;
                        if (src >= p.T) src = -1;
                    }
                    if (src >= 0 && col0 < p.out_n)
                        sw = __ldg(reinterpret_cast<const uint32_t *>(p.scales + src * p.ld_scales + (col0 >> 5)));
                    uint4 code[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int rr = i * 4 + rsub;
                        const int64_t sr = __shfl_sync(0xffffffffu, src, rr);
                        code[i] = make_uint4(0, 0, 0, 0);
                        if (sr >= 0 && col_ok) code[i] = load_codes(p.codes + sr * p.ld_codes + col, p.out_n - col);
                    }
                    if (hf == 0) {
                        int good = 1;
                        if (lane == 0)
                            good = wait_bar(ptx::smem_u32(&sh->empty[s]), ph ^ 1u, abort_flag, p.dev_status);
                        ok = __shfl_sync(0xffffffffu, good, 0) != 0;
                        __syncwarp();
                        if (!ok) break;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int rr = i * 4 + rsub, row = hf * 32 + rr;
                        const uint32_t word = __shfl_sync(0xffffffffu, sw, rr);
                        const uint32_t sc = kept_scale((word >> (8 * (chunk >> 1))) & 0xFFu);
                        const uint32_t cw4[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
                        uint32_t o[8];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            o[2 * j] = kept_pair(__byte_perm(cw4[j], 0u, 0x1404), sc);
                            o[2 * j + 1] = kept_pair(__byte_perm(cw4[j], 0u, 0x3424), sc);
                        }
                        uint8_t *line = dst + row * 128;
                        *reinterpret_cast<uint4 *>(line + ((q0 ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4 *>(line + (((q0 + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                }
                if (!ok) break;
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_u32(&sh->full[s]), 0));
                ph ^= 1u;
            }
            seq = (seq + (uint32_t)w.stages) % STAGES;
        }
    }

    ptx::tc_fence_before();
    ptx::cluster_sync();                   // neither CTA leaves while the pair still uses its memory
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, TMEM_COLS);
    }
}

// out = sum over splits of the partial results, in split order (+ out).
__global__ void __launch_bounds__(256) k_wgrad_reduce(const float *__restrict__ part, int splits, int64_t n, void *out,
                                                      int out_f32, int accumulate)
{
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += stride) {
        float s = 0.0f;
        for (int k = 0; k < splits; ++k) s += part[(int64_t)k * n + i];
        if (out_f32) {
            float *o = reinterpret_cast<float *>(out) + i;
            *o = accumulate ? *o + s : s;
        } else {
            __nv_bfloat16 *o = reinterpret_cast<__nv_bfloat16 *>(out) + i;
            *o = __float2bfloat16_rn(accumulate ? __bfloat162float(*o) + s : s);
        }
    }
}

// ----------------------------------------------------------------- host side

template <int MODE>
static nvfp4_status launch(const CUtensorMap &tm_a, const CUtensorMap &tm_b, const Params &p, int64_t max_tiles,
                           cudaStream_t st)
{
    static std::once_flag once[64];
    static cudaError_t attr_err[64];
    auto kern = k_ragged_gemm<MODE>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return check_launch("k_ragged_gemm: device");
    std::call_once(once[dev], [&] {
        attr_err[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
    });
    if (attr_err[dev] != cudaSuccess)
        return set_error(NVFP4_ERR_CUDA, "k_ragged_gemm: smem attribute: %s", cudaGetErrorString(attr_err[dev]));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    const int64_t units = std::min<int64_t>(num_sms() / 2, max_tiles);
    cfg.gridDim = dim3((unsigned)(2 * units));
    cfg.blockDim = dim3(Cfg<MODE>::THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kern, tm_a, tm_b, p);
    return check_launch("k_ragged_gemm");
}

// Widest vector store for rows of `row_bytes` from `base`.
static int store_width(const void *base, int64_t row_bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(base) | (uintptr_t)row_bytes;
    return a % 32 == 0 ? 32 : a % 16 == 0 ? 16 : 0;
}

// Row splits of a weight gradient: enough tiles for every CTA pair, but no
// split shorter than 256 rows of an even segment.
static int wgrad_splits(int64_t M, int64_t N, int64_t K, int32_t E)
{
    const int64_t tiles = ((N + TILE - 1) / TILE) * ((K + TILE - 1) / TILE) * E;
    const int64_t by_units = (num_sms() / 2) / std::max<int64_t>(tiles, 1);
    const int64_t by_rows = M / (256 * (int64_t)E);
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min(by_units, by_rows), 64));
}

}  // namespace ragged
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status moe_ragged_gemm(const void *a_dev, int64_t lda, int64_t M, const void *w_dev, int64_t N,
                                        int64_t K, int32_t E, const int32_t *offsets_dev, int32_t transpose,
                                        void *out_dev, int64_t ld_out, int32_t out_f32, int32_t *dev_status,
                                        void *stream)
{
    using namespace nvfp4::ragged;
    NVFP4_REQUIRE(M >= 0 && N >= 0 && K >= 0, NVFP4_ERR_INVALID_ARG, "moe_ragged_gemm: negative size");
    NVFP4_REQUIRE(E >= 1 && E <= MAX_E, NVFP4_ERR_UNSUPPORTED_SHAPE, "moe_ragged_gemm: 1 <= E <= 256");
    const int64_t in = transpose ? N : K, outw = transpose ? K : N;
    if (M == 0 || outw == 0) return NVFP4_OK;
    NVFP4_REQUIRE(in >= 1, NVFP4_ERR_UNSUPPORTED_SHAPE, "moe_ragged_gemm: empty reduction");
    NVFP4_REQUIRE(a_dev && w_dev && offsets_dev && out_dev, NVFP4_ERR_INVALID_ARG, "moe_ragged_gemm: null pointer");
    NVFP4_REQUIRE(M < (1ll << 31) - 512 && N < (1ll << 24) && K < (1ll << 24), NVFP4_ERR_UNSUPPORTED_SHAPE,
                  "moe_ragged_gemm: M must be below 2^31 - 512, N and K below 2^24");
    NVFP4_REQUIRE(K % 8 == 0, NVFP4_ERR_ALIGNMENT, "moe_ragged_gemm: K must be a multiple of 8 (rows of w on 16 bytes)");
    NVFP4_REQUIRE(lda >= in && lda % 8 == 0, NVFP4_ERR_ALIGNMENT,
                  "moe_ragged_gemm: lda must be >= the input width and a multiple of 8");
    NVFP4_REQUIRE(ld_out >= outw, NVFP4_ERR_ALIGNMENT, "moe_ragged_gemm: ld_out must be >= the output width");
    NVFP4_REQUIRE(aligned16(a_dev) && aligned16(w_dev), NVFP4_ERR_ALIGNMENT,
                  "moe_ragged_gemm: a and w must be 16-byte aligned");
    CUtensorMap tm_a, tm_b;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const bool ok = make_tmap_2d(&tm_a, a_dev, bf, (uint64_t)in, (uint64_t)M, (uint64_t)lda * 2, 64, 128, sw) &&
                    make_tmap_3d(&tm_b, w_dev, bf, (uint64_t)K, (uint64_t)N, (uint64_t)E, (uint64_t)K * 2,
                                 (uint64_t)N * K * 2, 64, transpose ? 64 : 128, sw);
    NVFP4_REQUIRE(ok, NVFP4_ERR_CUDA, "moe_ragged_gemm: tensor map encoding failed");
    Params p{};
    p.M = M;
    p.out_n = outw;
    p.red = in;
    p.E = E;
    p.n_tiles = (int)((outw + TILE - 1) / TILE);
    p.splits = 1;
    p.offsets = offsets_dev;
    p.out = out_dev;
    p.ld_out = ld_out;
    p.out_f32 = out_f32 ? 1 : 0;
    p.vec_bytes = store_width(out_dev, ld_out * (out_f32 ? 4 : 2));
    p.dev_status = dev_status;
    // row tiles: at most one partial tile per expert that has rows
    const int64_t max_tiles = (M / TILE + std::min<int64_t>(E, M)) * p.n_tiles;
    cudaStream_t st = (cudaStream_t)stream;
    return transpose ? launch<DGRAD>(tm_a, tm_b, p, max_tiles, st) : launch<FWD>(tm_a, tm_b, p, max_tiles, st);
}

extern "C" size_t moe_ragged_wgrad_workspace_size(int64_t M, int64_t N, int64_t K, int32_t E)
{
    if (M <= 0 || N <= 0 || K <= 0 || E <= 0) return 0;
    const int s = nvfp4::ragged::wgrad_splits(M, N, K, E);
    return s > 1 ? (size_t)s * (size_t)E * (size_t)N * (size_t)K * 4 : 0;
}

extern "C" nvfp4_status moe_ragged_wgrad(const void *g_dev, int64_t ldg, int64_t M, const void *a_dev, int64_t lda,
                                         const uint8_t *a_scales_dev, int64_t ld_scales, const int32_t *a_rows_dev,
                                         int64_t T, int64_t N, int64_t K, int32_t E, const int32_t *offsets_dev,
                                         void *out_dev, int32_t out_f32, int32_t accumulate, void *workspace,
                                         size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    using namespace nvfp4::ragged;
    const bool kept = a_scales_dev != nullptr;
    cudaStream_t st = (cudaStream_t)stream;
    NVFP4_REQUIRE(M >= 0 && N >= 0 && K >= 0 && T >= 0, NVFP4_ERR_INVALID_ARG, "moe_ragged_wgrad: negative size");
    NVFP4_REQUIRE(E >= 1 && E <= MAX_E, NVFP4_ERR_UNSUPPORTED_SHAPE, "moe_ragged_wgrad: 1 <= E <= 256");
    if (N == 0 || K == 0) return NVFP4_OK;
    NVFP4_REQUIRE(out_dev, NVFP4_ERR_INVALID_ARG, "moe_ragged_wgrad: null pointer");
    if (M == 0) {
        if (accumulate) return NVFP4_OK;
        if (cudaMemsetAsync(out_dev, 0, (size_t)E * N * K * (out_f32 ? 4 : 2), st) != cudaSuccess)
            return check_launch("moe_ragged_wgrad: memset");
        return NVFP4_OK;
    }
    NVFP4_REQUIRE(g_dev && (a_dev || (kept && T == 0)) && offsets_dev, NVFP4_ERR_INVALID_ARG,
                  "moe_ragged_wgrad: null pointer");
    NVFP4_REQUIRE(kept || !a_rows_dev, NVFP4_ERR_INVALID_ARG,
                  "moe_ragged_wgrad: a_rows needs an 8-bit a (a bf16 a is read in row order)");
    NVFP4_REQUIRE(!kept || a_rows_dev || T >= M, NVFP4_ERR_INVALID_ARG,
                  "moe_ragged_wgrad: without a_rows the kept tensor needs M rows");
    NVFP4_REQUIRE(M < (1ll << 31) - 512 && T < (1ll << 31) && N < (1ll << 24) && K < (1ll << 24),
                  NVFP4_ERR_UNSUPPORTED_SHAPE, "moe_ragged_wgrad: M and T must be below 2^31 - 512, N and K below 2^24");
    NVFP4_REQUIRE(ldg >= N && ldg % 8 == 0, NVFP4_ERR_ALIGNMENT,
                  "moe_ragged_wgrad: ldg must be >= N and a multiple of 8");
    NVFP4_REQUIRE(lda >= K && lda % (kept ? 16 : 8) == 0, NVFP4_ERR_ALIGNMENT,
                  "moe_ragged_wgrad: lda must be >= K and a multiple of 8 (16 for an 8-bit a)");
    NVFP4_REQUIRE(!kept || (ld_scales >= (K + 127) / 128 * 4 && ld_scales % 4 == 0), NVFP4_ERR_ALIGNMENT,
                  "moe_ragged_wgrad: ld_scales must be >= 4 * ceil(K / 128) and a multiple of 4");
    NVFP4_REQUIRE(aligned16(g_dev) && aligned16(a_dev) && aligned16(a_scales_dev), NVFP4_ERR_ALIGNMENT,
                  "moe_ragged_wgrad: pointers must be 16-byte aligned");
    const int splits = wgrad_splits(M, N, K, E);
    const size_t need = moe_ragged_wgrad_workspace_size(M, N, K, E);
    NVFP4_REQUIRE(need == 0 || (workspace && workspace_bytes >= need && aligned16(workspace)), NVFP4_ERR_WORKSPACE,
                  "moe_ragged_wgrad: workspace of %zu bytes required", need);

    CUtensorMap tm_a, tm_b;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    bool ok = make_tmap_2d(&tm_a, g_dev, bf, (uint64_t)N, (uint64_t)M, (uint64_t)ldg * 2, 64, 64, sw);
    if (!kept) ok = ok && make_tmap_2d(&tm_b, a_dev, bf, (uint64_t)K, (uint64_t)M, (uint64_t)lda * 2, 64, 64, sw);
    else tm_b = tm_a;
    NVFP4_REQUIRE(ok, NVFP4_ERR_CUDA, "moe_ragged_wgrad: tensor map encoding failed");
    Params p{};
    p.M = M;
    p.out_m = N;
    p.out_n = K;
    p.E = E;
    p.n_tiles = (int)((K + TILE - 1) / TILE);
    p.m_tiles = (int)((N + TILE - 1) / TILE);
    p.splits = splits;
    p.offsets = offsets_dev;
    p.out = splits > 1 ? workspace : out_dev;
    p.ld_out = K;
    p.out_f32 = splits > 1 || out_f32 ? 1 : 0;
    p.accumulate = splits > 1 ? 0 : (accumulate ? 1 : 0);
    p.vec_bytes = store_width(p.out, K * (p.out_f32 ? 4 : 2));
    p.codes = reinterpret_cast<const uint8_t *>(a_dev);
    p.ld_codes = lda;
    p.scales = a_scales_dev;
    p.ld_scales = ld_scales;
    p.a_rows = a_rows_dev;
    p.T = T;
    p.dev_status = dev_status;
    const int64_t max_tiles = (int64_t)E * p.m_tiles * p.n_tiles * splits;
    const nvfp4_status rc = kept ? launch<KEPT>(tm_a, tm_b, p, max_tiles, st) : launch<WGRAD>(tm_a, tm_b, p, max_tiles, st);
    if (rc != NVFP4_OK || splits == 1) return rc;
    const int64_t n = (int64_t)E * N * K;
    const unsigned blocks = (unsigned)std::max<int64_t>(1, std::min<int64_t>((n + 255) / 256, (int64_t)num_sms() * 8));
    k_wgrad_reduce<<<blocks, 256, 0, st>>>(reinterpret_cast<const float *>(workspace), splits, n, out_dev,
                                           out_f32 ? 1 : 0, accumulate ? 1 : 0);
    return check_launch("k_wgrad_reduce");
}
