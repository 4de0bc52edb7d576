// ragged.cu -- products grouped by expert over ragged row segments, and their
// gradients, on the sm_100a tensor cores (BF16 operands, f32 accumulation).
//
// Expert e owns rows [off[e], off[e+1]) of the routed row order; segments have
// any length, zero included, and are not padded.
//   FWD    out[r, n]  = sum_k a[r, k] w_e[n, k]
//   DGRAD  out[r, k]  = sum_n g[r, n] w_e[n, k]
//   WGRAD  dw_e[n, k] = sum_{r in e} g[r, n] a[r, k]
//
// Bound by the tensor pipe for segments of a few hundred rows and more, by the
// weights' bytes below that (WGRAD: by the result's bytes).  Measured, one B200,
// single launches with a cold L2, and in a continuous loop, which the power cap
// slows (segments of a skewed router; with equal ones FWD of 128 experts takes
// 211 us in the loop, so half of its distance to the bytes' 159 us is padding to
// 64 rows and uneven work of the pairs):
//   FWD    one segment, 8192 x 4096 x 4096             182 us  1.51 PFLOP/s
//          128 experts, 32768 rows, 2048 -> 1536       210 us  0.98 PFLOP/s, 5.0 TB/s   loop 262 us
//   DGRAD  32 experts, 32768 rows, 4096 -> 1536        300 us  1.37 PFLOP/s             loop 369 us
//   WGRAD  32 experts, 32768 rows, 4096 x 1536, f32    375 us  1.10 PFLOP/s, 3.1 TB/s   loop 447 us
//          128 experts, 32768 rows, 1536 x 2048, f32   347 us  0.59 PFLOP/s, 5.3 TB/s
//          the same from kept rows                     390 us                           loop 440 us
//
// A cluster of two CTAs computes one tile with tcgen05 .cta_group::2: each CTA
// stages half of the M-side operand (128 of 256) and half of the N-side one
// (up to 128), 64 deep, in a ring of stages; the even CTA issues the MMAs.
// TMEM holds two 256-column accumulators, so one tile's epilogue runs under
// the next tile's MMAs.
//
// Which operand goes where: the M side of an MMA has 256 rows whatever the
// tile needs, the N side any multiple of 64 up to 256.  FWD and DGRAD
// therefore put the weights on the M side and the ragged rows on the N side: a
// segment is cut into equal tiles of at most 256 rows, rounded up to 64, and
// neither MMAs nor loads are spent on the rest.
// (The rows on the M side pay for half-empty last tiles.)
//
// The tensor core takes an operand either way round (instruction descriptor
// bits 15 / 16), so no operand is ever transposed in memory:
//   K-major    the reduction runs along a row: row boxes of 64 columns;
//   MN-major   the reduction runs down the rows: 64-column x 64-row boxes.
// FWD is K x K, DGRAD MN x K, WGRAD MN x MN.
// The M side is always the output's contiguous dimension: TMEM lanes are then
// neighbouring columns of one output row, and a warp's store covers a 128-byte
// line.  (WGRAD with one row per lane, 32 lines per store: 528 us at 1536 x
// 2048, 128 experts; the stores held up the barrier traffic of the other warps.)
//
// Ragged reduction (WGRAD): a segment's last stage also holds rows of the next
// expert, or rows nobody wrote.  Zeroing one operand would not do (0 * NaN), so
// that stage lands on a barrier of its own CTA, warp 3 zeroes the surplus rows
// of both operands in shared memory and only then reports the stage to the
// MMA issuer.  A stage that holds a row whose index names no kept row goes the
// same way: its row of a is zeros, but its row of g may be anything.  Stages
// look for such rows only if the expanding launch met one (1536 x 2048, 128
// experts, 32768 rows: 55 us more with a single one, twice the time with a third
// of all rows, which one warp per CTA zeroes).  Without room for that launch's
// word every CTA looks through the whole row index first (one expert of 64 x 64,
// 262144 rows: 43.7 -> 56.7 us).  Ragged rows (FWD, DGRAD) need nothing: a
// surplus row only makes an accumulator column that the epilogue does not store.
//
// Long sums (WGRAD): the tensor core's f32 accumulation truncates, an error
// that grows with the number of additions (1.6e-6 in norm after 1024 rows,
// 2.8e-7 for f32 additions rounded to nearest).  The accumulator is therefore
// handed over after at most CHUNK stages and the chunks are added in the epilogue's
// registers.
//
// Rows kept in 8 bits (E4M3, a power-of-two scale per 32 columns) are first
// expanded, gathered by their row index, into a BF16 copy in the workspace
// (exact).  Converting inside the WGRAD kernel was built and measured: every
// M-side tile converts its rows again, and 6 converter warps could not keep up
// (1536 x 2048, 128 experts, 32768 rows: 731 us when a BF16 operand took 471;
// with the expanded copy it is 390 against 347).
//
// WGRAD with few output tiles splits every segment's rows over several tiles:
// f32 partial results in the workspace, added in split order by a second
// kernel (no atomics: the result does not change from run to run).
//
// Warps: 0, 2 TMA producers (M side, N side); 1 MMA issuer; 3 the surplus-row
// fixer; 4..11 epilogue.  Every mbarrier wait is bounded (1 s); on expiry the
// kernel records NVFP4_ERR_TIMEOUT, its roles stop, copies in flight get 1 ms
// to land, MMAs are drained and TMEM is freed.
#include "common.cuh"
#include "ptx.cuh"

#include <cuda.h>
#include <algorithm>
#include <mutex>

namespace nvfp4 {
namespace ragged {

constexpr int TILE = 256;                        // M side of a pair's tile, most of its N side
constexpr int N_STEP = 64;                       // granularity of the N side
constexpr int BK = 64;                           // reduction depth of a stage
constexpr int CHUNK = 8;                         // WGRAD: most stages summed in one accumulator
constexpr int STAGES = 6;
constexpr uint32_t OPER_BYTES = 128 * BK * 2;    // one operand of one CTA: 16 KB
constexpr uint32_t BOX_BYTES = 64 * BK * 2;      // one MN-major box: 8 KB
constexpr int ROW_BOX = 32;                      // rows per box of the ragged rows (FWD, DGRAD)
constexpr uint32_t STAGE_BYTES = 2 * OPER_BYTES;
constexpr uint32_t SMEM = STAGES * STAGE_BYTES + 1024 /*align*/ + 4096 /*barriers, offsets*/;
static_assert(SMEM <= 232448, "shared memory budget");
constexpr int EPI_WARPS = 8, EPI_WARP0 = 4;
constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
constexpr int PROD_M_WARP = 0, MMA_WARP = 1, PROD_N_WARP = 2, FIX_WARP = 3;
constexpr uint32_t TMEM_COLS = 512;
constexpr int COLS = 16;                         // accumulator columns read at a time
constexpr int MAX_E = 256;
constexpr uint64_t TIMEOUT_NS = 1000000000ull;

enum Mode { FWD = 0, DGRAD = 1, WGRAD = 2 };

struct Params {
    int64_t M;                 // rows of the routed order
    int64_t out_m, out_n;      // M-side extent (FWD: N, DGRAD, WGRAD: K); WGRAD: N-side extent (N)
    int64_t red;               // FWD, DGRAD: reduction length
    int E;
    int m_tiles;               // tiles along the M side
    int n_tiles;               // WGRAD: tiles along the N side
    int splits;                // WGRAD: row splits of every segment
    const int32_t *offsets;
    const int32_t *a_rows;     // INDEXED: kept row of each row
    int64_t kept_rows;         // INDEXED: rows of the kept tensor
    const uint8_t *outside;    // INDEXED: what the expanding launch's blocks met (act8_expand), or null
    int outside_n;
    void *out;
    int64_t ld_out;
    int pairs;                 // bf16 out: two neighbouring columns may be stored at once
    int32_t *dev_status;
    uint64_t wait_limit_ns;    // bound of every mbarrier wait
    int withhold;              // test hook: the first tile's "accumulator ready" is not signalled
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
    int progress;              // WGRAD: stages that the M-side producer has filled
    int dead[EPI_WARP0 + EPI_WARPS];   // INDEXED: the warp saw a row of no kept row
    int off[MAX_E + 1];        // segment bounds, made monotone and in [0, M]
    int tiles[MAX_E + 1];      // FWD / DGRAD: row tiles before expert e
};

// A converged warp's wait, bounded: false on a timeout or another role's.
// `cluster`: the peer CTA's threads wrote shared memory before they arrived.
// `progress`: while this count moves the bound starts anew (for a wait over
// more than the stages in the ring).
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag, const Params &p,
                                         bool ignore_abort = false, bool cluster = false,
                                         const volatile int *progress = nullptr)
{
    bool ok = true;
    uint64_t t0 = 0;
    int seen = 0;
    for (uint32_t i = 1;; ++i) {
        if (cluster ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait_hint(bar, parity)) break;
        if ((i & 15u) == 0u) {
            if (!ignore_abort && *abort_flag) { ok = false; break; }
            const uint64_t now = globaltimer_ns();
            if (t0 == 0 || (progress && *progress != seen)) {
                t0 = now;
                if (progress) seen = *progress;
            } else if (now - t0 > p.wait_limit_ns) {
                *abort_flag = 1;
                report_status(p.dev_status, NVFP4_ERR_TIMEOUT);
                ok = false;
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok ? 1 : 0) != 0;         // a uniform answer
}

// A unit's tiles t = unit, unit + n_units, ...  WGRAD keeps t's digits (expert,
// split, N tile, M tile) and adds n_units digit by digit: a division costs a
// role ~200 clk per tile, and there were five.  The M tiles run innermost: the
// units then write whole output rows together (32 experts of 4096 x 1536:
// 391 us -> 376 us).
template <int MODE>
struct Walk {
    int t;
    int e, split, nt, mt;
    int de, ds, dn, dm;

    __device__ __forceinline__ static void digits(const Params &p, int v, int &e, int &s, int &m, int &n)
    {
        const int mn = p.m_tiles * p.n_tiles, per = mn * p.splits;
        e = v / per;
        v -= e * per;
        s = v / mn;
        v -= s * mn;
        n = v / p.m_tiles;
        m = v - n * p.m_tiles;
    }
    __device__ __forceinline__ Walk(const Params &p, int unit, int n_units) : t(unit)
    {
        if (MODE == WGRAD) {
            digits(p, unit, e, split, mt, nt);
            digits(p, n_units, de, ds, dm, dn);
        }
    }
    __device__ __forceinline__ void next(const Params &p, int n_units)
    {
        t += n_units;
        if (MODE == WGRAD) {
            nt += dn;
            mt += dm;
            split += ds;
            e += de;
            if (mt >= p.m_tiles) { mt -= p.m_tiles; ++nt; }
            if (nt >= p.n_tiles) { nt -= p.n_tiles; ++split; }
            if (split >= p.splits) { split -= p.splits; ++e; }
        }
    }
};

// What a tile covers.
struct Tile {
    int e;
    int64_t m0;                // M-side start
    int64_t n0, n_end;         // N-side start and end
    int nt;                    // N-side size of the MMA
    int r0, r1;                // WGRAD: its rows
    int stages;                // reduction stages (0: WGRAD of an empty segment)
    int chunk;                 // stages per accumulator
    int split;
};

// Values from shared memory are broadcast, so that the compiler knows
// everything here to be the same in all lanes.
template <int MODE>
__device__ __forceinline__ Tile tile_at(const Params &p, const Shared *sh, const Walk<MODE> &at)
{
    const auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    Tile w;
    if (MODE == WGRAD) {
        w.e = at.e;
        w.split = at.split;
        w.m0 = (int64_t)at.mt * TILE;
        w.n0 = (int64_t)at.nt * TILE;
        w.n_end = p.out_n;
        w.nt = TILE;
        w.r0 = same(sh->off[w.e]);
        w.r1 = same(sh->off[w.e + 1]);
        if (p.splits > 1) {
            // whole stages per split, so that only a segment's last stage is ragged
            const int rows = ((w.r1 - w.r0 + p.splits - 1) / p.splits + BK - 1) / BK * BK;
            const int64_t r0 = (int64_t)w.r0 + (int64_t)w.split * rows;
            w.r0 = (int)min((int64_t)w.r1, r0);
            w.r1 = (int)min((int64_t)w.r1, r0 + rows);
        }
        w.stages = (w.r1 - w.r0 + BK - 1) / BK;
        w.chunk = max(1, w.stages);
        if (w.stages > CHUNK) {
            const int chunks = (w.stages + CHUNK - 1) / CHUNK;
            w.chunk = (w.stages + chunks - 1) / chunks;
        }
    } else {
        int lo = 0, hi = p.E;                        // expert: tiles[lo] * m_tiles <= t < tiles[hi] * m_tiles
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (same(sh->tiles[mid]) * p.m_tiles <= at.t) lo = mid; else hi = mid;
        }
        // an expert's tiles: its row tiles innermost, they share a weight tile
        const int first = same(sh->tiles[lo]), row_tiles = same(sh->tiles[lo + 1]) - first;
        const int off = same(sh->off[lo]), end = same(sh->off[lo + 1]);
        int mt = at.t - first * p.m_tiles, i = 0, size = end - off;
        if (row_tiles > 1) {
            const int idx = mt;
            mt = idx / row_tiles;
            i = idx - mt * row_tiles;
            size = (size + row_tiles - 1) / row_tiles;
        }
        size = (size + N_STEP - 1) / N_STEP * N_STEP;
        w.e = lo;
        w.m0 = (int64_t)mt * TILE;
        w.n0 = (int64_t)off + (int64_t)i * size;
        w.n_end = end;
        w.nt = min(size, (int)((w.n_end - w.n0 + N_STEP - 1) / N_STEP) * N_STEP);
        w.r0 = w.r1 = 0;
        w.split = 0;
        w.stages = w.chunk = (int)((p.red + BK - 1) / BK);
    }
    return w;
}

// Which rows of a stage (bit = row - its first one; rows from `end` on: none)
// name no kept row; the same in all lanes.
__device__ __forceinline__ uint64_t dead_rows(const Params &p, int row, int end)
{
    const int r = row + (int)(threadIdx.x & 31);
    const int lo = r < end ? p.a_rows[r] : 0, hi = r + 32 < end ? p.a_rows[r + 32] : 0;
    const unsigned dead_lo = __ballot_sync(0xffffffffu, r < end && (lo < 0 || lo >= p.kept_rows));
    const unsigned dead_hi = __ballot_sync(0xffffffffu, r + 32 < end && (hi < 0 || hi >= p.kept_rows));
    return (uint64_t)dead_hi << 32 | dead_lo;
}

// Is there such a row among this warp's share of all rows?  16-byte loads, eight
// under way, between the ends.
__device__ __forceinline__ bool any_dead_row(const Params &p, int share, int shares)
{
    const int lane = threadIdx.x & 31;
    const auto gone = [&](int v) { return v < 0 || v >= p.kept_rows; };
    const int64_t head = min(p.M, (int64_t)((16 - (reinterpret_cast<uintptr_t>(p.a_rows) & 15u)) & 15u) / 4);
    const int64_t vecs = (p.M - head) / 4, done = head + vecs * 4;
    const int4 *body = reinterpret_cast<const int4 *>(p.a_rows + head);
    bool dead = false;
    if (share == 0) {
        if (lane < head) dead = gone(p.a_rows[lane]);
        if (done + lane < p.M) dead = dead || gone(p.a_rows[done + lane]);
    }
    constexpr int DEEP = 8;
    const int64_t step = (int64_t)shares * 32;
    for (int64_t i = (int64_t)share * 32 + lane; i < vecs; i += DEEP * step) {
        int4 v[DEEP];
#pragma unroll
        for (int j = 0; j < DEEP; ++j) v[j] = body[min(i + j * step, vecs - 1)];
#pragma unroll
        for (int j = 0; j < DEEP; ++j) dead |= gone(v[j].x) | gone(v[j].y) | gone(v[j].z) | gone(v[j].w);
    }
    return __any_sync(0xffffffffu, dead ? 1 : 0) != 0;
}

// WGRAD's epilogue holds 128 sums and 32 columns in flight per thread: the
// control warps pass registers on (56 + 2 x 224 of the 3 x 168 per warpgroup
// that the block starts with).
template <int MODE>
__device__ __forceinline__ void give_registers()
{
    if (MODE == WGRAD) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
}

template <int MODE>
__device__ __forceinline__ void take_registers()
{
    if (MODE == WGRAD) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
}

// R output rows from `row`, of which `rows` exist, at column m = this lane's.
// ADD: to the old value, in f32.  The f32 stores are marked streaming: nothing
// here reads them again, the operands' tiles are (WGRAD, 1536 x 2048, 128
// segments of 256 rows: 398 -> 382 us).
template <bool ADD, int R>
__device__ __forceinline__ void store_rows(const Params &p, float *out, int64_t row, int rows, int64_t m,
                                           const float (&v)[R])
{
    float *dst = out + row * p.ld_out + m;
    if (m >= p.out_m) rows = 0;
#pragma unroll
    for (int j = 0; j < R; ++j, dst += p.ld_out)
        if (j < rows) {
            if (ADD) *dst += v[j];
            else __stcs(dst, v[j]);
        }
}

// n zeros from dst by `threads` threads, 16 bytes a store between the ends.
template <typename T>
__device__ __forceinline__ void zero_run(T *dst, int64_t n, int thread, int threads)
{
    const int64_t head = min(n, (int64_t)((16 - (reinterpret_cast<uintptr_t>(dst) & 15u)) & 15u) / (int64_t)sizeof(T));
    const int64_t vecs = (n - head) * (int64_t)sizeof(T) / 16;
    uint4 *body = reinterpret_cast<uint4 *>(dst + head);
    for (int64_t i = thread; i < vecs; i += threads) body[i] = make_uint4(0, 0, 0, 0);
    const int64_t done = head + vecs * (16 / (int64_t)sizeof(T));
    for (int64_t i = thread; i < head; i += threads) dst[i] = T(0.0f);
    for (int64_t i = done + thread; i < n; i += threads) dst[i] = T(0.0f);
}

// The same as bf16.  Neighbouring lanes exchange values: the even lane stores
// row j, the odd lane row j + 1, both of columns m & ~1 and m | 1, so a store
// instruction writes 2 rows x 64 bytes.
template <bool ADD, int R>
__device__ __forceinline__ void store_rows(const Params &p, __nv_bfloat16 *out, int64_t row, int rows, int64_t m,
                                           const float (&v)[R])
{
    const int odd = (int)(threadIdx.x & 1);
    const int64_t me = m - odd;
    __nv_bfloat16 *dst = out + (row + odd) * p.ld_out + me;
    const bool has_lo = me < p.out_m, has_hi = me + 1 < p.out_m;
    const bool pair = p.pairs != 0 && has_hi;
    rows -= odd;
#pragma unroll
    for (int j = 0; j < R; j += 2, dst += 2 * p.ld_out) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
        float lo = odd ? got : v[j], hi = odd ? v[j + 1] : got;
        if (ADD) {
            if (j < rows && has_lo) lo += __bfloat162float(dst[0]);
            if (j < rows && has_hi) hi += __bfloat162float(dst[1]);
        }
        const uint32_t b = pack_bf16(lo, hi);
        if (j < rows && pair) *reinterpret_cast<uint32_t *>(dst) = b;
        if (j < rows && !pair && has_lo) dst[0] = __ushort_as_bfloat16((unsigned short)b);
        if (j < rows && !pair && has_hi) dst[1] = __ushort_as_bfloat16((unsigned short)(b >> 16));
    }
}

// INDEXED (WGRAD): rows may name no kept row (a_rows).
template <int MODE, typename OutT, bool ADD, bool INDEXED>
__global__ void __launch_bounds__(THREADS, 1)
k_ragged_gemm(const __grid_constant__ CUtensorMap tm_m, const __grid_constant__ CUtensorMap tm_n, const Params p)
{
    constexpr bool A_MN = MODE != FWD, B_MN = MODE == WGRAD;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *stage_base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Shared *sh = reinterpret_cast<Shared *>(stage_base + STAGES * STAGE_BYTES);
    volatile int *abort_flag = &sh->abort_flag;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;
    const int unit = (int)(blockIdx.x >> 1), n_units = (int)(gridDim.x >> 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh->full[s]), 2);
            ptx::mbar_init(ptx::smem_u32(&sh->empty[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh->raw[s]), 2);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_u32(&sh->tmem_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh->tmem_empty[i]), 2 * EPI_WARPS);
        }
        ptx::mbar_init(ptx::smem_u32(&sh->drain), 1);
        sh->abort_flag = 0;
        sh->progress = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 0) {
        ptx::tmem_alloc_pair(ptx::smem_u32(&sh->tmem_base), TMEM_COLS);
        ptx::tmem_relinquish_pair();
    }
    grid_wait();                           // the predecessor's results are visible from here on
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
        if (INDEXED && lane == 0) sh->dead[warp] = 0;
    } else if (INDEXED) {
        // the other warps ask meanwhile whether there is a dead row at all: a
        // routed batch without padding has none, and then no stage looks
        const int share = warp < FIX_WARP ? warp : warp - 1;
        constexpr int SHARES = EPI_WARP0 + EPI_WARPS - 1;
        bool dead = false;
        if (p.outside) {
            for (int i = share * 32 + lane; i < p.outside_n; i += SHARES * 32) dead |= p.outside[i] != 0;
            dead = __any_sync(0xffffffffu, dead ? 1 : 0) != 0;
        } else {
            dead = any_dead_row(p, share, SHARES);
        }
        if (lane == 0) sh->dead[warp] = dead;
    }
    grid_release();
    ptx::tc_fence_before();
    ptx::cluster_sync();                   // barriers of both CTAs initialized before any remote use
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem_base, 0);
    // looking at every stage's rows costs loads that queue behind the epilogue's stores
    bool look = false;
    if (INDEXED) look = __any_sync(0xffffffffu, lane < EPI_WARP0 + EPI_WARPS && sh->dead[lane] != 0) != 0;
    const int total = MODE == WGRAD ? p.E * p.m_tiles * p.n_tiles * p.splits : sh->tiles[p.E] * p.m_tiles;

    if (warp == PROD_M_WARP || warp == PROD_N_WARP) {
        give_registers<MODE>();
        // ----------------------------------------------------- producers
        // The whole warp runs the loop and one elected lane issues: loop state
        // and copy operands then live in uniform registers.  (Issued from a
        // lane == 0 branch, each TMA copy cost ~110 and each MMA ~125 cycles of
        // its thread.)
        {
            const bool one = ptx::elect_one();
            const bool m_side = warp == PROD_M_WARP;
            const CUtensorMap *tm = m_side ? &tm_m : &tm_n;
            if (one) ptx::prefetch_tmap(tm);
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            int filled = 0;
            for (Walk<MODE> at(p, unit, n_units); ok && at.t < total; at.next(p, n_units)) {
                const Tile w = tile_at<MODE>(p, sh, at);
                // this CTA's half of the operand
                const int half_n = w.nt / 2;
                const int mn = (int)(m_side ? w.m0 + rank * 128 : w.n0 + (int)rank * half_n);
                const uint32_t bytes = m_side || MODE == WGRAD ? OPER_BYTES : (uint32_t)half_n * (BK * 2);
                for (int kb = 0; kb < w.stages; ++kb) {
                    const int row = w.r0 + kb * BK;
                    bool fix = MODE == WGRAD && row + BK > w.r1;
                    if (INDEXED && look) fix = dead_rows(p, row, w.r1) != 0 || fix;
                    if (!wait_bar(ptx::smem_u32(&sh->empty[stage]), phase ^ 1u, abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    if (MODE == WGRAD && m_side && one) *(volatile int *)&sh->progress = ++filled;
                    const uint32_t dst = ptx::smem_u32(stage_base + stage * STAGE_BYTES + (m_side ? 0 : OPER_BYTES));
                    const uint32_t fb = ptx::smem_u32(&sh->full[stage]);
                    const uint32_t lfb = ptx::mapa_shared(fb, 0);      // the leader's barrier
                    if (fix) {
                        // rows to zero: land in this CTA, the fixer reports it
                        const uint32_t rb = ptx::smem_u32(&sh->raw[stage]);
                        if (one) {
                            ptx::mbar_arrive_expect_tx(rb, OPER_BYTES);
                            ptx::tma_load_2d(dst, tm, mn, row, rb);
                            ptx::tma_load_2d(dst + BOX_BYTES, tm, mn + 64, row, rb);
                        }
                    } else {
                        if (one && leader) ptx::mbar_arrive_expect_tx(fb, 2 * bytes);
                        if (MODE == WGRAD) {
                            if (one) {
                                ptx::tma_load_2d_pair(dst, tm, mn, row, lfb);
                                ptx::tma_load_2d_pair(dst + BOX_BYTES, tm, mn + 64, row, lfb);
                            }
                        } else if (!m_side) {
                            for (int i = 0; i < half_n; i += ROW_BOX)
                                if (one) ptx::tma_load_2d_pair(dst + i * (BK * 2), tm, kb * BK, mn + i, lfb);
                        } else if (MODE == DGRAD) {
                            if (one) {
                                ptx::tma_load_3d_pair(dst, tm, mn, kb * BK, w.e, lfb);
                                ptx::tma_load_3d_pair(dst + BOX_BYTES, tm, mn + 64, kb * BK, w.e, lfb);
                            }
                        } else {
                            if (one) ptx::tma_load_3d_pair(dst, tm, kb * BK, mn, w.e, lfb);
                        }
                    }
                    __syncwarp();
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
        give_registers<MODE>();
        if (leader) {
            // ----------------------------------------------- MMA issuer
            const bool one = ptx::elect_one();
            uint32_t stage = 0, phase = 0;
            bool ok = true, issued = false, ready = false;
            const uint32_t full0 = ptx::smem_u32(&sh->full[0]), empty0 = ptx::smem_u32(&sh->empty[0]);
            const uint32_t s0 = ptx::smem_u32(stage_base);
            const uint64_t a_desc = A_MN ? ptx::make_sdesc(s0, BOX_BYTES, 1024, 2) : ptx::make_sdesc(s0, 16, 1024, 2);
            const uint64_t b_desc = B_MN ? ptx::make_sdesc(s0 + OPER_BYTES, BOX_BYTES, 1024, 2)
                                         : ptx::make_sdesc(s0 + OPER_BYTES, 16, 1024, 2);
            int iter = 0;                                // accumulators handed over
            for (Walk<MODE> at(p, unit, n_units); ok && at.t < total; at.next(p, n_units)) {
                const Tile w = tile_at<MODE>(p, sh, at);
                const uint32_t idesc = ptx::idesc_bf16(TILE, (uint32_t)w.nt) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
                const int64_t len = MODE == WGRAD ? (int64_t)(w.r1 - w.r0) : p.red;
                for (int kb = 0; kb < w.stages;) {
                    const int acc = iter & 1;
                    if (!wait_bar(ptx::smem_u32(&sh->tmem_empty[acc]), (uint32_t)((iter >> 1) & 1) ^ 1u, abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    ++iter;
                    ptx::tc_fence_after();
                    const uint32_t d = tmem + (uint32_t)acc * TILE;
                    const int kend = min(kb + w.chunk, w.stages);
                    for (uint32_t first = 1; kb < kend; ++kb, first = 0) {
                        if (!ready && !wait_bar(full0 + 8 * stage, phase, abort_flag, p, false, MODE == WGRAD)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                        const uint64_t ad = a_desc + (uint64_t)(stage * (STAGE_BYTES >> 4));
                        const uint64_t bd = b_desc + (uint64_t)(stage * (STAGE_BYTES >> 4));
                        const uint32_t done = empty0 + 8 * stage;
                        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                        // look at the next stage's barrier while this stage's MMAs are issued
                        const bool peek = MODE == WGRAD ? ptx::mbar_test_wait_cluster(full0 + 8 * stage, phase)
                                                        : ptx::mbar_test_wait(full0 + 8 * stage, phase);
                        const int64_t left = len - (int64_t)kb * BK;
                        // K-major: 32 bytes along the row per MMA; MN-major: 16 rows of 128 bytes
                        constexpr uint64_t A_STEP = (A_MN ? 2048 : 32) >> 4, B_STEP = (B_MN ? 2048 : 32) >> 4;
                        if (left >= BK) {
#pragma unroll
                            for (int kk = 0; kk < BK / 16; ++kk)
                                if (one) ptx::mma_bf16_pair(d, ad + kk * A_STEP, bd + kk * B_STEP, idesc, kk == 0 ? 1u - first : 1u);
                        } else {
                            for (int kk = 0; 16 * kk < (int)left; ++kk)
                                if (one) ptx::mma_bf16_pair(d, ad + kk * A_STEP, bd + kk * B_STEP, idesc, kk == 0 ? 1u - first : 1u);
                        }
                        if (one) ptx::tc_commit_pair_mc(done, 3);
                        ready = __all_sync(0xffffffffu, peek ? 1 : 0) != 0;
                        issued = true;
                    }
                    if (!ok) break;
                    if (MODE == FWD && p.withhold) {
                        // test hook: the epilogue's wait runs out; the MMAs are drained
                        // here, before any thread can release TMEM
                        if (one) ptx::tc_commit_pair_mc(ptx::smem_u32(&sh->drain), 1);
                        wait_bar(ptx::smem_u32(&sh->drain), 0, abort_flag, p, true);
                        issued = ok = false;
                        break;
                    }
                    if (one) ptx::tc_commit_pair_mc(ptx::smem_u32(&sh->tmem_full[acc]), 3);
                    __syncwarp();
                }
            }
            if (!ok && issued) {
                // let every issued MMA finish before TMEM is released
                if (one) ptx::tc_commit_pair_mc(ptx::smem_u32(&sh->drain), 1);
                wait_bar(ptx::smem_u32(&sh->drain), 0, abort_flag, p, true);
            }
        }
        __syncwarp();
    } else if (warp == FIX_WARP) {
        give_registers<MODE>();
        if (MODE == WGRAD) {
            // --------------------- zero surplus rows, and rows of no kept row
            uint32_t stage = 0, parity = 0;             // one parity bit per stage's raw barrier
            bool ok = true;
            for (Walk<MODE> at(p, unit, n_units); ok && at.t < total; at.next(p, n_units)) {
                const Tile w = tile_at<MODE>(p, sh, at);
                // without such rows only a segment's last stage can need it
                int kb = INDEXED && look ? 0 : max(0, w.stages - 1);
                stage = (stage + (uint32_t)kb) % STAGES;
                for (; kb < w.stages; ++kb) {
                    const uint32_t s = stage;
                    if (++stage == STAGES) stage = 0;
                    const int row = w.r0 + kb * BK;
                    const int rows = min(BK, w.r1 - row);
                    uint64_t dead = 0;
                    if (INDEXED && look) dead = dead_rows(p, row, w.r1);
                    if (rows == BK && (!INDEXED || dead == 0)) continue;
                    // the stage may lie a whole long segment, or many tiles, ahead
                    if (!wait_bar(ptx::smem_u32(&sh->raw[s]), (parity >> s) & 1u, abort_flag, p, false, false,
                                  &sh->progress)) {
                        ok = false;
                        break;
                    }
                    parity ^= 1u << s;
                    uint8_t *base = stage_base + s * STAGE_BYTES;
                    // 128-byte rows of both operands' boxes; the swizzle stays inside a row
                    const auto zero_16 = [&](uint8_t *at) {
#pragma unroll
                        for (int b = 0; b < 4; ++b) *reinterpret_cast<uint4 *>(at + b * BOX_BYTES) = make_uint4(0, 0, 0, 0);
                    };
                    if (INDEXED && dead != 0) {
                        for (int i = lane; i < rows * 8; i += 32)
                            if (dead >> (i >> 3) & 1) zero_16(base + i * 16);
                    }
                    for (int i = lane; i < (BK - rows) * 8; i += 32) zero_16(base + rows * 128 + i * 16);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_u32(&sh->full[s]), 0));
                }
            }
        }
    } else {
        // --------------------------------------------------- epilogue
        // Warp w reads TMEM lanes 32 (w % 4).. of its CTA (M side) and one
        // half of the columns (N side).
        take_registers<MODE>();
        const int q = warp & 3, half = (warp - EPI_WARP0) >> 2;
        const int m_in_tile = (int)rank * 128 + q * 32 + lane;
        int iter = 0;
        for (Walk<MODE> at(p, unit, n_units); at.t < total; at.next(p, n_units)) {
            const Tile w = tile_at<MODE>(p, sh, at);
            const int64_t m = w.m0 + m_in_tile;
            if (MODE == WGRAD && w.stages == 0) {
                // an empty segment's gradient: its tiles share out the
                // expert's N x K zeros as one contiguous run
                if (!ADD) {
                    const int64_t all = p.out_n * p.ld_out, per = (int64_t)p.m_tiles * p.n_tiles;
                    const int64_t i = w.m0 / TILE * p.n_tiles + w.n0 / TILE;
                    const int64_t share = ((all + per - 1) / per + 15) / 16 * 16;
                    const int64_t lo = min(all, i * share), hi = min(all, lo + share);
                    OutT *base = reinterpret_cast<OutT *>(p.out) + ((int64_t)w.split * p.E + w.e) * all;
                    zero_run(base + lo, hi - lo, (int)rank * 32 * EPI_WARPS + (warp - EPI_WARP0) * 32 + lane,
                             2 * 32 * EPI_WARPS);
                }
                continue;
            }
            // lane = column m of the output, TMEM columns = its rows (WGRAD: rows n
            // of the expert's gradient)
            const int half_n = MODE == WGRAD ? TILE / 2 : w.nt / 2;
            const int64_t n = w.n0 + half * half_n;
            const int64_t row = MODE == WGRAD ? ((int64_t)w.split * p.E + w.e) * p.out_n + n : n;
            const int rows = (int)(w.n_end - n);
            const uint32_t src0 = tmem + (uint32_t)(half * half_n) + ((uint32_t)(q * 32) << 16);
            OutT *out = reinterpret_cast<OutT *>(p.out);
            if (MODE == WGRAD && w.chunk < w.stages) {
                // several accumulators: summed in registers
                float v[128];
#pragma unroll
                for (int i = 0; i < 128; ++i) v[i] = 0.0f;
                bool ok = true;
                for (int kb = 0; kb < w.stages; kb += w.chunk, ++iter) {
                    const int acc = iter & 1;
                    ok = wait_bar(ptx::smem_u32(&sh->tmem_full[acc]), (uint32_t)((iter >> 1) & 1), abort_flag, p);
                    if (!ok) break;
                    ptx::tc_fence_after();
#pragma unroll
                    for (int c = 0; c < 128; c += 32) {
                        uint32_t x[32];
                        ptx::tmem_ld_32x32b_x32(src0 + (uint32_t)(acc * TILE + c), x);
                        ptx::tmem_ld_wait(x);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[c + i] += __uint_as_float(x[i]);
                    }
                    // the accumulator is free once both CTAs' warps have read it
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_cluster_relaxed(ptx::mapa_shared(ptx::smem_u32(&sh->tmem_empty[acc]), 0));
                }
                if (!ok) break;
                store_rows<ADD>(p, out, row, rows, m, v);
                __syncwarp();                            // lanes without an output rejoin before the collective load
                continue;
            }
            const int acc = iter & 1;
            if (!wait_bar(ptx::smem_u32(&sh->tmem_full[acc]), (uint32_t)((iter >> 1) & 1), abort_flag, p)) break;
            ++iter;
            ptx::tc_fence_after();
            // 16 columns are stored while the next 16 come from TMEM
            const uint32_t src = src0 + (uint32_t)(acc * TILE);
            uint32_t x[COLS], y[COLS];
            ptx::tmem_ld_32x32b_x16(src, x);
#pragma unroll 1
            for (int c = 0; c < half_n; c += 2 * COLS) {
                ptx::tmem_ld_wait(x);
                ptx::tmem_ld_32x32b_x16(src + c + COLS, y);
                store_rows<ADD>(p, out, row + c, rows - c, m, reinterpret_cast<const float (&)[COLS]>(x));
                __syncwarp();                            // lanes without an output rejoin before the collective load
                ptx::tmem_ld_wait(y);
                if (c + 2 * COLS < half_n) ptx::tmem_ld_32x32b_x16(src + c + 2 * COLS, x);
                else {
                    // the accumulator is free once both CTAs' warps have read it
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_cluster_relaxed(ptx::mapa_shared(ptx::smem_u32(&sh->tmem_empty[acc]), 0));
                }
                store_rows<ADD>(p, out, row + c + COLS, rows - c - COLS, m, reinterpret_cast<const float (&)[COLS]>(y));
                __syncwarp();
            }
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
__global__ void __launch_bounds__(256) k_wgrad_reduce(const float *part, int splits, int64_t n, void *out,
                                                      int out_f32, int accumulate)
{
    const int64_t stride = (int64_t)gridDim.x * 256;
    grid_wait();
    grid_release();
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

template <int MODE, typename OutT, bool ADD, bool INDEXED = false>
static nvfp4_status launch(const CUtensorMap &tm_m, const CUtensorMap &tm_n, const Params &p, int64_t max_tiles,
                           cudaStream_t st)
{
    static std::once_flag once[64];
    static cudaError_t attr_err[64];
    auto kern = k_ragged_gemm<MODE, OutT, ADD, INDEXED>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return check_launch("k_ragged_gemm: device");
    std::call_once(once[dev], [&] {
        attr_err[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
    });
    if (attr_err[dev] != cudaSuccess)
        return set_error(NVFP4_ERR_CUDA, "k_ragged_gemm: smem attribute: %s", cudaGetErrorString(attr_err[dev]));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    const int64_t units = std::min<int64_t>(num_sms() / 2, max_tiles);
    cfg.gridDim = dim3((unsigned)(2 * units));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1] = overlap_attribute();
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaLaunchKernelEx(&cfg, kern, tm_m, tm_n, p);
    return check_launch("k_ragged_gemm");
}

template <typename OutT, bool ADD>
static nvfp4_status launch_wgrad(const CUtensorMap &tm_m, const CUtensorMap &tm_n, const Params &p, int64_t max_tiles,
                                 cudaStream_t st)
{
    return p.a_rows ? launch<WGRAD, OutT, ADD, true>(tm_m, tm_n, p, max_tiles, st)
                    : launch<WGRAD, OutT, ADD, false>(tm_m, tm_n, p, max_tiles, st);
}

// Rows of bf16 pairs on 4 bytes?
static int pair_stores(const void *base, int64_t ld) { return (reinterpret_cast<uintptr_t>(base) & 3u) == 0 && ld % 2 == 0; }

// Row splits of a weight gradient: enough tiles for every CTA pair, but no
// split shorter than 256 rows of an even segment.  Measured without splits and
// with them: one 256 x 256 result of 512 rows 9.1 and 9.7 us (two splits), of
// 1024 11.5 and 9.6, of 32768 150 and 20; at least 128 or 512 rows a split the
// same within 1 us.  With more tiles a second split gains less than its second
// kernel costs: 5 experts of 520 x 264, 5000 rows, 14.0 and 15.1 us; 8 of 512 x
// 512, 16384 rows, 17.0 and 20.4.
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

static nvfp4_status ragged_gemm(const void *a_dev, int64_t lda, int64_t M, const void *w_dev, int64_t N, int64_t K,
                                int32_t E, const int32_t *offsets_dev, int32_t transpose, void *out_dev, int64_t ld_out,
                                int32_t out_f32, int32_t *dev_status, void *stream, uint64_t wait_limit_ns, int withhold)
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
    NVFP4_REQUIRE(aligned16(a_dev) && aligned16(w_dev) && reinterpret_cast<uintptr_t>(out_dev) % (out_f32 ? 4 : 2) == 0,
                  NVFP4_ERR_ALIGNMENT, "moe_ragged_gemm: a and w must be 16-byte aligned, out aligned to its elements");
    CUtensorMap tm_m, tm_n;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const bool ok = make_tmap_2d(&tm_n, a_dev, bf, (uint64_t)in, (uint64_t)M, (uint64_t)lda * 2, BK, ROW_BOX, sw) &&
                    make_tmap_3d(&tm_m, w_dev, bf, (uint64_t)K, (uint64_t)N, (uint64_t)E, (uint64_t)K * 2,
                                 (uint64_t)N * K * 2, 64, transpose ? BK : 128, sw);
    NVFP4_REQUIRE(ok, NVFP4_ERR_CUDA, "moe_ragged_gemm: tensor map encoding failed");
    Params p{};
    p.M = M;
    p.out_m = outw;
    p.red = in;
    p.E = E;
    p.m_tiles = (int)((outw + TILE - 1) / TILE);
    p.splits = 1;
    p.wait_limit_ns = wait_limit_ns;
    p.withhold = withhold;
    p.offsets = offsets_dev;
    p.out = out_dev;
    p.ld_out = ld_out;
    p.pairs = pair_stores(out_dev, ld_out);
    p.dev_status = dev_status;
    // row tiles: at most one partial tile per expert that has rows
    const int64_t max_tiles = (M / TILE + std::min<int64_t>(E, M)) * p.m_tiles;
    NVFP4_REQUIRE(max_tiles < (1ll << 30), NVFP4_ERR_UNSUPPORTED_SHAPE, "moe_ragged_gemm: too many tiles");
    cudaStream_t st = (cudaStream_t)stream;
    if (transpose)
        return out_f32 ? launch<DGRAD, float, false>(tm_m, tm_n, p, max_tiles, st)
                       : launch<DGRAD, __nv_bfloat16, false>(tm_m, tm_n, p, max_tiles, st);
    return out_f32 ? launch<FWD, float, false>(tm_m, tm_n, p, max_tiles, st)
                   : launch<FWD, __nv_bfloat16, false>(tm_m, tm_n, p, max_tiles, st);
}

extern "C" nvfp4_status moe_ragged_gemm(const void *a_dev, int64_t lda, int64_t M, const void *w_dev, int64_t N,
                                        int64_t K, int32_t E, const int32_t *offsets_dev, int32_t transpose,
                                        void *out_dev, int64_t ld_out, int32_t out_f32, int32_t *dev_status,
                                        void *stream)
{
    return ragged_gemm(a_dev, lda, M, w_dev, N, K, E, offsets_dev, transpose, out_dev, ld_out, out_f32, dev_status, stream,
                       nvfp4::ragged::TIMEOUT_NS, 0);
}

extern "C" nvfp4_status nvfp4_debug_ragged_wait_expiry(const void *a_dev, int64_t lda, int64_t M, const void *w_dev,
                                                       int64_t N, int64_t K, const int32_t *offsets_dev, void *out_dev,
                                                       int64_t ld_out, int32_t *dev_status, int64_t wait_limit_ns,
                                                       void *stream)
{
    NVFP4_REQUIRE(dev_status && wait_limit_ns >= 1000000 && wait_limit_ns <= 1000000000ll, NVFP4_ERR_INVALID_ARG,
                  "nvfp4_debug_ragged_wait_expiry: needs dev_status and 1 ms <= wait_limit_ns <= 1 s");
    NVFP4_REQUIRE(M >= 1 && M <= nvfp4::ragged::TILE && N >= 1 && N <= nvfp4::ragged::TILE, NVFP4_ERR_UNSUPPORTED_SHAPE,
                  "nvfp4_debug_ragged_wait_expiry: one tile (M, N <= 256)");
    return ragged_gemm(a_dev, lda, M, w_dev, N, K, 1, offsets_dev, 0, out_dev, ld_out, 1, dev_status, stream,
                       (uint64_t)wait_limit_ns, 1);
}

// Workspace of a weight gradient: [BF16 copy of the kept rows][partial
// results], and with rows named by an index, where there is room for it, [what
// the expanding launch met].
static size_t expanded_bytes(int64_t M, int64_t K) { return ((size_t)M * (size_t)((K + 7) / 8 * 8) * 2 + 255) / 256 * 256; }

extern "C" size_t moe_ragged_wgrad_workspace_size(int64_t M, int64_t N, int64_t K, int32_t E, int32_t kept)
{
    if (M <= 0 || N <= 0 || K <= 0 || E <= 0) return 0;
    const int s = nvfp4::ragged::wgrad_splits(M, N, K, E);
    return (kept ? expanded_bytes(M, K) : 0) + (s > 1 ? (size_t)s * (size_t)E * (size_t)N * (size_t)K * 4 : 0) +
           (kept == 2 ? (size_t)nvfp4::act8_expand_max_blocks() : 0);
}

static nvfp4_status ragged_wgrad(const void *g_dev, int64_t ldg, int64_t M, const void *a_dev, int64_t lda,
                                 const uint8_t *a_scales_dev, int64_t ld_scales, const int32_t *a_rows_dev, int64_t T,
                                 int64_t N, int64_t K, int32_t E, const int32_t *offsets_dev, void *out_dev,
                                 int32_t out_f32, int32_t accumulate, void *workspace, size_t workspace_bytes,
                                 int32_t *dev_status, void *stream, uint64_t wait_limit_ns)
{
    using namespace nvfp4::ragged;
    const bool kept = a_scales_dev != nullptr;
    cudaStream_t st = (cudaStream_t)stream;
    NVFP4_REQUIRE(M >= 0 && N >= 0 && K >= 0 && T >= 0, NVFP4_ERR_INVALID_ARG, "moe_ragged_wgrad: negative size");
    NVFP4_REQUIRE(E >= 1 && E <= MAX_E, NVFP4_ERR_UNSUPPORTED_SHAPE, "moe_ragged_wgrad: 1 <= E <= 256");
    if (N == 0 || K == 0) return NVFP4_OK;
    NVFP4_REQUIRE(out_dev, NVFP4_ERR_INVALID_ARG, "moe_ragged_wgrad: null pointer");
    NVFP4_REQUIRE(reinterpret_cast<uintptr_t>(out_dev) % (out_f32 ? 4 : 2) == 0, NVFP4_ERR_ALIGNMENT,
                  "moe_ragged_wgrad: out must be aligned to its elements");
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
    const size_t need = moe_ragged_wgrad_workspace_size(M, N, K, E, kept ? 1 : 0);
    NVFP4_REQUIRE(need == 0 || (workspace && workspace_bytes >= need && aligned16(workspace)), NVFP4_ERR_WORKSPACE,
                  "moe_ragged_wgrad: workspace of %zu bytes required", need);

    const int64_t max_tiles = (int64_t)E * ((K + TILE - 1) / TILE) * ((N + TILE - 1) / TILE) * splits;
    NVFP4_REQUIRE(max_tiles < (1ll << 30), NVFP4_ERR_UNSUPPORTED_SHAPE, "moe_ragged_wgrad: too many tiles");
    uint8_t *partials = reinterpret_cast<uint8_t *>(workspace), *outside = nullptr;
    int outside_n = 0;
    if (kept) {
        if (a_rows_dev && workspace_bytes >= moe_ragged_wgrad_workspace_size(M, N, K, E, 2)) outside = partials + need;
        // the kept rows as BF16, in row order
        const int64_t ld = (K + 7) / 8 * 8;
        const nvfp4_status rc = act8_expand(reinterpret_cast<const uint8_t *>(a_dev), lda, a_scales_dev, ld_scales,
                                            a_rows_dev, T, M, K, workspace, ld, outside, &outside_n, st);
        if (rc != NVFP4_OK) return rc;
        a_dev = workspace;
        lda = ld;
        partials += expanded_bytes(M, K);
    }
    CUtensorMap tm_m, tm_n;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const bool ok = make_tmap_2d(&tm_m, a_dev, bf, (uint64_t)K, (uint64_t)M, (uint64_t)lda * 2, 64, BK, sw) &&
                    make_tmap_2d(&tm_n, g_dev, bf, (uint64_t)N, (uint64_t)M, (uint64_t)ldg * 2, 64, BK, sw);
    NVFP4_REQUIRE(ok, NVFP4_ERR_CUDA, "moe_ragged_wgrad: tensor map encoding failed");
    Params p{};
    p.M = M;
    p.out_m = K;
    p.out_n = N;
    p.E = E;
    p.m_tiles = (int)((K + TILE - 1) / TILE);
    p.n_tiles = (int)((N + TILE - 1) / TILE);
    p.splits = splits;
    p.wait_limit_ns = wait_limit_ns;
    p.offsets = offsets_dev;
    p.a_rows = a_rows_dev;
    p.kept_rows = T;
    p.outside = outside;
    p.outside_n = outside_n;
    p.out = splits > 1 ? partials : out_dev;
    p.ld_out = K;
    p.pairs = pair_stores(p.out, K);
    p.dev_status = dev_status;
    if (splits == 1) {
        if (out_f32)
            return accumulate ? launch_wgrad<float, true>(tm_m, tm_n, p, max_tiles, st)
                              : launch_wgrad<float, false>(tm_m, tm_n, p, max_tiles, st);
        return accumulate ? launch_wgrad<__nv_bfloat16, true>(tm_m, tm_n, p, max_tiles, st)
                          : launch_wgrad<__nv_bfloat16, false>(tm_m, tm_n, p, max_tiles, st);
    }
    const nvfp4_status rc = launch_wgrad<float, false>(tm_m, tm_n, p, max_tiles, st);
    if (rc != NVFP4_OK) return rc;
    const int64_t n = (int64_t)E * N * K;
    const unsigned blocks = (unsigned)std::max<int64_t>(1, std::min<int64_t>((n + 255) / 256, (int64_t)num_sms() * 8));
    launch_overlapped(k_wgrad_reduce, dim3(blocks), 256, 0, st, reinterpret_cast<const float *>(partials), splits, n, out_dev,
                      out_f32 ? 1 : 0, accumulate ? 1 : 0);
    return check_launch("k_wgrad_reduce");
}

extern "C" nvfp4_status moe_ragged_wgrad(const void *g_dev, int64_t ldg, int64_t M, const void *a_dev, int64_t lda,
                                         const uint8_t *a_scales_dev, int64_t ld_scales, const int32_t *a_rows_dev,
                                         int64_t T, int64_t N, int64_t K, int32_t E, const int32_t *offsets_dev,
                                         void *out_dev, int32_t out_f32, int32_t accumulate, void *workspace,
                                         size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    return ragged_wgrad(g_dev, ldg, M, a_dev, lda, a_scales_dev, ld_scales, a_rows_dev, T, N, K, E, offsets_dev, out_dev,
                        out_f32, accumulate, workspace, workspace_bytes, dev_status, stream, nvfp4::ragged::TIMEOUT_NS);
}

extern "C" nvfp4_status nvfp4_debug_ragged_wgrad_wait_limit(const void *g_dev, int64_t ldg, int64_t M, const void *a_dev,
                                                            int64_t lda, int64_t N, int64_t K, int32_t E,
                                                            const int32_t *offsets_dev, void *out_dev,
                                                            int32_t *dev_status, int64_t wait_limit_ns, void *stream)
{
    NVFP4_REQUIRE(dev_status && wait_limit_ns >= 1000000 && wait_limit_ns <= 1000000000ll, NVFP4_ERR_INVALID_ARG,
                  "nvfp4_debug_ragged_wgrad_wait_limit: needs dev_status and 1 ms <= wait_limit_ns <= 1 s");
    return ragged_wgrad(g_dev, ldg, M, a_dev, lda, nullptr, 0, nullptr, 0, N, K, E, offsets_dev, out_dev, 1, 0, nullptr, 0,
                        dev_status, stream, (uint64_t)wait_limit_ns);
}
