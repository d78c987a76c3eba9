// k3_grouped_wgrad.cu -- weight gradients grouped by expert, dW_e = dY_e^T X_e, on the
// tensor cores (tcgen05.mma kind::f16, bf16 operands, fp32 sums).
//
// dW_e[n][k] = sum over the rows i of expert e's group of dY[i][n] X[i][k].  The sum
// runs over rows, the slow axis of both matrices, so both operands are read as they
// lie in memory (M- and N-major tiles, the 128-byte swizzle over 64 columns of a row)
// and nothing is transposed.
//
// X's columns k take the MMA's lanes and dY's columns n its columns.  A pair of CTAs
// (cta_group::2) works on 256 k x 256 n: each loads 128 columns of X and 128 of dY and the
// MMA reads both, so that a step of 64 rows brings 32 KB into an SM for its 512 clocks of
// MMAs.  (Lone CTAs with 128 k x 256 n, 48 KB a step: 64 x 1536 x 7168 from 16384 gathered
// rows 518 us, pairs 480; 16 x 2048 x 2048 from 131072 773 and 622, in group order 690 and
// 600.)  Where 128 x 128 tiles make two waves at most, single CTAs take those.
//
// Persistent CTAs or pairs walk (expert, k, n) tiles.  Roles: warp 0 (of the even CTA) issues
// MMAs, warps 4 to 11 read one accumulator out while the other one's products run, and each
// further warp fills a share of a stage of 64 rows: dY's columns by TMA, X's by TMA too
// where it lies in group order, else row by row with asynchronous copies into the same
// swizzled form; in a group's last step rows past it are made zeros in both.  Copies and
// fillers of both CTAs are counted on the even one's barrier.  (TMA gathers of four rows
// take 72 clocks each: 2.06 ms with them.)
//
// Bound: the stores of dW where groups are short (64 x 1536 x 7168 fp32 from 16384 rows, 2.8
// GB, gathered 480 us, 5.9 TB/s), the MMAs beside the copies where they are long (16 x 2048
// x 2048 from 131072 rows 604 us in group order, 1.8 PFLOP/s; gathered 650).
//
// Every wait is bounded (2 s, and 16 us a step where a whole tile is waited for); a
// timeout sets the device error word and the CTA drains its copies and MMAs, frees TMEM
// and exits.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "k3_launch.cuh"
#include "k3_operand.cuh"
#include "k3_tcgen05.cuh"
#include "k3_tmem.cuh"

namespace k3 {
namespace {

constexpr int GW_CTA = 128, GW_K = 64;  // k and n of a CTA in a tile, rows of a step
constexpr int GW_NS = 6;
constexpr int GW_W_MMA = 0, GW_W_EPI = 4;
constexpr int GW_EPI = 8;  // epilogue warps: two per TMEM lane quadrant, on alternate pieces
constexpr int GW_W_FILL = GW_W_EPI + GW_EPI;
constexpr int GW_FILL = 2;  // warps that fill a stage, half of its rows each
constexpr int GW_THREADS = (GW_W_FILL + GW_FILL * GW_NS) * 32;

struct GwArgs {
    const int32_t *offsets, *order;
    int E, top_k, slots, gather, xrows;
    FastDiv tiles_k, tiles_e;  // k tiles of a row of tiles, tiles of an expert
    int N, K, accumulate;
    const __nv_bfloat16 *dy, *x;
    void *dw;
    long lddy, ldx;
    int ns;  // stages in use, at most GW_NS
    int *err;
};

constexpr int GW_PANEL = GW_K * 128;  // 64 rows of 64 columns
constexpr int GW_PANELS = GW_CTA / 64, GW_OFF_Y = GW_PANELS * GW_PANEL, GW_STAGE = 2 * GW_OFF_Y;
constexpr int GW_BOX = 16;  // rows n of a staged box of dW, 32 columns k wide; two boxes a warp
constexpr int GW_OFF_C = GW_NS * GW_STAGE, GW_OFF_BAR = GW_OFF_C + GW_EPI * 2 * GW_BOX * 128;
constexpr int GW_BARS = 2 * GW_NS + 2 * 2 + 1;
constexpr int GW_SMEM = 1024 + GW_OFF_BAR + 256;
static_assert(GW_SMEM <= 232448, "shared memory");
static_assert(GW_K / GW_FILL % 16 == 0, "a share is the rows of whole MMAs");

// Instruction descriptor, kind::f16: fp32 accumulator, bf16 A and B, both M/N-major.
constexpr uint32_t gw_idesc(int m, int n)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// A step: an MMA for each 16 rows, one to four.  Descriptors of M/N-major tiles: panels
// of 64 columns GW_PANEL bytes apart (leading offset), groups of eight rows 1024 bytes
// (stride).
template <int CTAS>
K3_DEV void gw_step(uint32_t tacc, uint32_t xlo, uint32_t ylo, uint32_t acc, int mmas)
{
#define GW_MMA(group, k2, pred, on)                                                                                 \
    "add.u32 x, %1, " #k2 ";\n\tadd.u32 y, %2, " #k2 ";\n\tmov.b64 da, {x, %4};\n\tmov.b64 db, {y, %4};\n\t" \
    "@" on " tcgen05.mma.cta_group::" group ".kind::f16 [%0], da, db, %5, " pred ";\n\t"
#define GW_STEP(group)                                                                                            \
    asm volatile("{\n\t.reg .pred p, t, e, f, g, h;\n\t.reg .b64 da, db;\n\t.reg .b32 x, y;\n\telect.sync _|e, 0xffffffff;\n\t" \
                 "setp.ne.b32 p, %3, 0;\n\tsetp.eq.b32 t, %5, %5;\n\tsetp.gt.and.s32 f, %6, 1, e;\n\t"             \
                 "setp.gt.and.s32 g, %6, 2, e;\n\tsetp.gt.and.s32 h, %6, 3, e;\n\t" GW_MMA(group, 0, "p", "e")      \
                     GW_MMA(group, 128, "t", "f") GW_MMA(group, 256, "t", "g") GW_MMA(group, 384, "t", "h") "}" ::"r"(tacc), \
                 "r"(xlo), "r"(ylo), "r"(acc), "r"(SW128_HI), "r"(gw_idesc(CTAS * GW_CTA, CTAS * GW_CTA)), "r"(mmas)  \
                 : "memory")
    if constexpr (CTAS == 2)
        GW_STEP("2");
    else
        GW_STEP("1");
#undef GW_STEP
#undef GW_MMA
}
K3_DEV uint32_t mn_lo(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | ((uint32_t)(GW_PANEL >> 4) << 16); }

// Chunk c of row r of a panel: eight columns of a row, zeros where `on` is false or the
// columns lie past the matrix.
K3_DEV void gw_chunk(uint32_t panel, int r, int c, const __nv_bfloat16 *row, int col, int cols, bool on)
{
    const uint32_t dst = panel + (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
    if (on && col < cols)
        copy16(dst, row + col);
    else
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0u) : "memory");
}
// Announces copied bytes, without an arrival.
K3_DEV void mbar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Tile u: its expert, n, k, and the group's rows.
struct GwTile {
    int e, n0, k0, row, rows;
};
K3_DEV GwTile gw_tile(const GwArgs &a, int u, int size)  // size: k and n of a tile
{
    GwTile t;
    t.e = (int)a.tiles_e.div((uint32_t)u);
    const int r = u - t.e * (int)a.tiles_e.d, rn = (int)a.tiles_k.div((uint32_t)r);
    t.n0 = rn * size;
    t.k0 = (r - rn * (int)a.tiles_k.d) * size;
    t.row = max(a.offsets[t.e], 0);
    t.rows = max(min(a.offsets[t.e + 1], a.slots) - t.row, 0);
    return t;
}

// A staged box to (k, n) of expert e: stored, or added in fp32.  Stores are the first to
// leave L2, which keeps the rows (64 x 1536 x 7168 from 16384 rows in group order: 522
// against 551 us).
K3_DEV void gw_store(const CUtensorMap *map, uint32_t src, int k, int n, int e, int accumulate)
{
    if (accumulate)
        asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                         (uint64_t)map),
                     "r"(k), "r"(n), "r"(e), "r"(src)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group.L2::cache_hint [%0, {%1, %2, %3}], [%4], "
                     "%5;" ::"l"((uint64_t)map),
                     "r"(k), "r"(n), "r"(e), "r"(src), "l"(l2_evict_first())
                     : "memory");
}

template <int CTAS, typename CT>
__global__ void __launch_bounds__(GW_THREADS, 1)
    k3_grouped_wgrad(const __grid_constant__ CUtensorMap ymap, const __grid_constant__ CUtensorMap xmap,
                     const __grid_constant__ CUtensorMap cmap, const GwArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_addr(sm);
    uint64_t *bars = (uint64_t *)(sm + GW_OFF_BAR);
    constexpr int NS = GW_NS, TILE = CTAS * GW_CTA;
    constexpr int B_FULL = 0, B_EMPTY = NS, B_ACCF = 2 * NS, B_ACCE = B_ACCF + 2, B_FIN = B_ACCE + 2;
    uint32_t *tmem_slot = (uint32_t *)(bars + GW_BARS);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);
    auto bar = [&](int i) { return smem_addr(bars + i); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = CTAS == 2 ? (int)cluster_rank() : 0;  // 0: the CTA that issues

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; i++) {
            mbar_init(bar(B_FULL + i), CTAS * GW_FILL);
            mbar_init(bar(B_EMPTY + i), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(bar(B_ACCF + i), 1);
            mbar_init(bar(B_ACCE + i), CTAS * GW_EPI);  // the epilogue warps of both CTAs
        }
        mbar_init(bar(B_FIN), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == GW_W_MMA) {
        if constexpr (CTAS == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                         "r"(2 * TILE)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                         "r"(2 * TILE)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CTAS == 2) cluster_sync();  // the other CTA's barriers are initialised
    tc_fence_after();
    const uint32_t tmem = __reduce_max_sync(0xffffffffu, *(volatile uint32_t *)tmem_slot);
    griddep_wait();
    const int n_tiles = a.E * (int)a.tiles_e.d, first = (int)blockIdx.x / CTAS, step = (int)gridDim.x / CTAS;
    auto commit = [](uint32_t b) {
        if constexpr (CTAS == 2)
            pair_commit(b);
        else
            mma_commit(b);
    };

    if (warp >= GW_W_FILL) {
        // -------------------------------------------------- a stage's fillers
        // Every ns-th step of these tiles; the GW_FILL warps of a stage have a
        // share of its rows each, the first one issues the TMA copies.
        const int s = (warp - GW_W_FILL) / GW_FILL, share = (warp - GW_W_FILL) % GW_FILL;
        constexpr int ROWS = GW_K / GW_FILL;
        const uint32_t st = sbase + (uint32_t)(s * GW_STAGE), full0 = CTAS == 2 ? addr_of_rank(bar(B_FULL + s), 0) : bar(B_FULL + s);
        uint32_t turn = 0;
        int u = first, r0 = s * GW_K, tile = -1;
        GwTile t = {};
        for (; s < a.ns; r0 += a.ns * GW_K, turn++) {
            for (; u < n_tiles; u += step) {
                if (u != tile) tile = u, t = gw_tile(a, u, TILE);
                if (r0 < t.rows) break;
                r0 -= (t.rows + GW_K - 1) / GW_K * GW_K;
            }
            if (u >= n_tiles) break;
            const int k0 = t.k0 + rank * GW_CTA, n0 = t.n0 + rank * GW_CTA;  // this CTA's columns
            const int n = min(GW_K, t.rows - r0);                            // rows of the group in this step
            const int n16 = (n + 15) & ~15;                                  // rows that its MMAs read
            // lane l: X's row of the share's row l
            int src = 0;
            if (a.gather && lane < ROWS && share * ROWS + lane < n) {
                src = a.order[t.row + r0 + share * ROWS + lane] / a.top_k;
                if (src < 0 || src >= a.xrows) src = 0;
            }
            // before its first completion an EMPTY barrier's odd phase counts as passed
            if (!__all_sync(0xffffffffu, tc_wait(bar(B_EMPTY + s), (turn & 1) ^ 1u, a.err, abort_flag))) break;
            const bool whole = n == n16;
            // where no row past the group is read: dY (and X in group order) by TMA
            if (share == 0 && whole) {
                if (rank == 0 && lane == 0)
                    mbar_expect(bar(B_FULL + s), (uint32_t)CTAS * (uint32_t)(a.gather ? GW_STAGE - GW_OFF_Y : GW_STAGE));
                __syncwarp();
                auto load = [&](uint32_t at, const CUtensorMap *map, int col) {
                    if constexpr (CTAS == 2)
                        pair_load_2d(st + at, map, col, t.row + r0, full0);
                    else
                        tma_load_2d(st + at, map, col, t.row + r0, full0);
                };
                if (lane < GW_PANELS)
                    load((uint32_t)(GW_OFF_Y + lane * GW_PANEL), &ymap, n0 + 64 * lane);
                else if (!a.gather && lane < 2 * GW_PANELS)
                    load((uint32_t)((lane - GW_PANELS) * GW_PANEL), &xmap, k0 + 64 * (lane - GW_PANELS));
                __syncwarp();
            }
            if ((a.gather || !whole) && share * ROWS < n16) {
                // 128 columns of a row are 16 chunks of 16 bytes, two rows a warp
#pragma unroll
                for (int i = 0; i < ROWS; i += 2) {
                    const int r = share * ROWS + i + (lane >> 4), c = lane & 15;
                    const int g = __shfl_sync(0xffffffffu, src, i + (lane >> 4));
                    const long x = a.gather ? g : t.row + r0 + min(r, n - 1);
                    gw_chunk(st + (uint32_t)((c >> 3) * GW_PANEL), r, c & 7, a.x + x * a.ldx, k0 + 8 * c, a.K, r < n);
                }
                if (!whole)
#pragma unroll
                    for (int i = 0; i < ROWS; i += 2) {
                        const int r = share * ROWS + i + (lane >> 4), c = lane & 15;
                        gw_chunk(st + (uint32_t)(GW_OFF_Y + (c >> 3) * GW_PANEL), r, c & 7,
                                 a.dy + (long)(t.row + r0 + min(r, n - 1)) * a.lddy, n0 + 8 * c, a.N, r < n);
                    }
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_async_smem();
                __syncwarp();
            }
            if (lane == 0) pair_arrive(bar(B_FULL + s), full0, rank);
        }
        // drain: the last turn's copies of both CTAs have landed before the even CTA
        // exits; the odd one waits in the closing cluster barrier
        if (rank == 0 && turn) mbar_wait(bar(B_FULL + s), (turn - 1) & 1, a.err);
        __syncwarp();
    } else if (warp == GW_W_MMA && rank == 1) {
        // the even CTA issues for both
    } else if (warp == GW_W_MMA) {
        // -------------------------------------------------------------- MMA
        uint32_t ut = 0, phase = 0;  // ut: tiles with rows
        int s = 0;
        bool ok = true, ready = false;
        const uint32_t lo = mn_lo(sbase);
        auto full = [&](uint32_t b, uint32_t parity) {
            return CTAS == 2 ? tc_wait_pair(b, parity, a.err, abort_flag) : tc_wait(b, parity, a.err, abort_flag);
        };
        for (int u = first; u < n_tiles && ok; u += step) {
            const GwTile t = gw_tile(a, u, TILE);
            if (!t.rows) continue;
            const int buf = (int)(ut & 1);
            if (ut >= 2 && !__all_sync(0xffffffffu, tc_wait(bar(B_ACCE + buf), (ut / 2 - 1) & 1, a.err, abort_flag)))
                break;
            tc_fence_after();
            for (int r0 = 0; r0 < t.rows; r0 += GW_K) {
                if (!ready && !__all_sync(0xffffffffu, full(bar(B_FULL + s), phase))) {
                    ok = false;
                    break;
                }
                if constexpr (CTAS == 2) pair_acquire();
                tc_fence_after();
                const int sn = s + 1 == a.ns ? 0 : s + 1;
                const uint32_t pn = sn ? phase : phase ^ 1u;
                // ask for the next stage before this one is issued, look at the answer after
                const bool next = CTAS == 2 ? mbar_test_pair(bar(B_FULL + sn), pn) : mbar_test(bar(B_FULL + sn), pn);
                const uint32_t d = lo + (uint32_t)(s * (GW_STAGE / 16));
                gw_step<CTAS>(tmem + (uint32_t)(buf * TILE), d, d + GW_OFF_Y / 16, r0 ? 1u : 0u, (t.rows - r0 + 15) / 16);
                commit(bar(B_EMPTY + s));
                ready = __all_sync(0xffffffffu, next);
                s = sn;
                phase = pn;
            }
            if (!ok) break;
            commit(bar(B_ACCF + buf));
            ut++;
        }
        // every MMA issued above has completed before TMEM is freed
        commit(bar(B_FIN));
        mbar_wait(bar(B_FIN), 0, a.err);
        __syncwarp();
    } else if (warp >= GW_W_EPI) {
        // --------------------------------------------------------- epilogue
        // A lane holds one column k of dW, 32 rows n at a time; the two warps of a
        // quadrant take alternate pieces.  Boxes of 16 rows leave by TMA, clipped at the
        // expert's matrix, one being filled while the other is read.  (Stored from
        // registers, 128 bytes of a row at a time, an SM's stores left at 18 bytes a clock:
        // 64 x 1536 x 7168 from 16384 gathered rows took 664 us; with one box of 32 rows,
        // waited for, 558.)
        const int q = warp & 3, half = (warp - GW_W_EPI) >> 2;
        constexpr int NP = TILE / 32;
        CT *const boxes = (CT *)(sm + GW_OFF_C + (warp - GW_W_EPI) * 2 * GW_BOX * 128);
        uint32_t box = 0;
        uint32_t ut = 0;
        for (int u = first; u < n_tiles; u += step) {
            const GwTile t = gw_tile(a, u, TILE);
            if (!t.rows && a.accumulate) continue;
            const int buf = (int)(ut & 1);
            if (t.rows) {
                if (!__all_sync(0xffffffffu, tc_wait_tile(bar(B_ACCF + buf), (ut / 2) & 1, (uint32_t)(t.rows / GW_K), a.err,
                                                          abort_flag)))
                    break;
                tc_fence_after();
            }
            const uint32_t tacc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * TILE);
            const int k = t.k0 + rank * GW_CTA + q * 32 + lane;
#pragma unroll 1
            for (int j = half; j < NP; j += 2) {
                uint32_t r[32];
                if (t.rows) {
                    tmem_ld_chunk(tacc + (uint32_t)(j * 32), r);
                    if (j + 2 >= NP) {  // this warp's last piece
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if constexpr (CTAS == 2)
                                mbar_arrive_rank(bar(B_ACCE + buf), 0);
                            else
                                mbar_arrive(bar(B_ACCE + buf));
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 32; c++) r[c] = 0u;
                }
#pragma unroll
                for (int h = 0; h < 2; h++, box ^= 1) {
                    CT *const o = boxes + box * (GW_BOX * 32) + lane;
                    // the box's last copy, the one before the newest, has been read
                    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < GW_BOX; c++) {
                        if constexpr (sizeof(CT) == 2)
                            o[c * 32] = __float2bfloat16_rn(__uint_as_float(r[h * GW_BOX + c]));
                        else
                            o[c * 32] = __uint_as_float(r[h * GW_BOX + c]);
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        const int n = t.n0 + j * 32 + h * GW_BOX;
                        if (n < a.N && k < a.K) gw_store(&cmap, smem_addr(o), k, n, t.e, a.accumulate);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                }
            }
            if (t.rows) ut++;
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    // The even CTA's last commits have arrived here before this CTA may exit.  The
    // last tile has been read, so they are on their way: a short wait after a call of any
    // length.
    if (rank == 1 && warp == GW_W_MMA) {
        volatile int ignore = 0;  // after an abort too
        if (lane == 0) tc_wait(bar(B_FIN), 0, a.err, &ignore);
        __syncwarp();
    }
    if constexpr (CTAS == 2) cluster_sync();  // neither CTA leaves, or frees TMEM, while the other's work may reach it
    if (warp == GW_W_MMA) {
        tc_fence_after();
        if constexpr (CTAS == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * TILE) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * TILE) : "memory");
    }
}

// ---------------------------------------------------------------- launchers

// A bf16 matrix in boxes of a panel: 64 columns x 64 rows, 128-byte swizzle.
int row_map(CUtensorMap *map, const void *p, int cols, int n_rows, long ld)
{
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)n_rows}, strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, GW_K};
    return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int CTAS, typename CT>
int launch_gw(const GwArgs &a, cudaStream_t s)
{
    CUtensorMap ymap, xmap;
    int st = row_map(&ymap, a.dy, a.N, a.slots, a.lddy);
    if (st == K3MOE_OK) st = row_map(&xmap, a.x, a.K, a.xrows, a.ldx);
    CUtensorMap cmap;
    const cuuint64_t dims[3] = {(cuuint64_t)a.K, (cuuint64_t)a.N, (cuuint64_t)a.E},
                     strides[2] = {(cuuint64_t)a.K * sizeof(CT), (cuuint64_t)a.K * a.N * sizeof(CT)};
    const cuuint32_t box[3] = {32, GW_BOX, 1};
    if (st == K3MOE_OK)
        st = encode_map(&cmap, sizeof(CT) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, a.dw,
                        dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (st != K3MOE_OK) return st;
    if (ensure_smem((const void *)k3_grouped_wgrad<CTAS, CT>, GW_SMEM) != K3MOE_OK) return K3MOE_ECUDA;
    const int grid = CTAS * std::min(a.E * (int)a.tiles_e.d, num_sms() / CTAS);
    if (launch_dependent(true, CTAS, k3_grouped_wgrad<CTAS, CT>, dim3((unsigned)grid), dim3(GW_THREADS), GW_SMEM, s, ymap, xmap, cmap, a) !=
        cudaSuccess) {
        cudaGetLastError();
        return K3MOE_ECUDA;
    }
    return K3MOE_OK;
}

}  // namespace

int launch_grouped_wgrad(const k3moe_grouped_wgrad_desc &d, int *err, cudaStream_t s)
{
    const k3moe_groups *g = d.host_groups;
    GwArgs a = {};
    a.offsets = g->offsets, a.order = g->order;
    a.E = g->E, a.top_k = g->top_k, a.slots = g->tokens * g->top_k, a.gather = d.gather ? 1 : 0, a.xrows = d.xrows;
    // single CTAs or pairs, in us: 66 tiles of single CTAs from few rows 5.9 and 9.2, 128 from
    // 512 rows a group 10.9 and 15.1, 256 from 2048 24.5 and 29.5, 512 from 128 10.6 and 11.0
    const bool pair = (long)a.E * ((d.K + GW_CTA - 1) / GW_CTA) * ((d.N + GW_CTA - 1) / GW_CTA) > 2 * num_sms();
    const int size = pair ? 2 * GW_CTA : GW_CTA, tiles_k = (d.K + size - 1) / size;
    const long tiles = (long)tiles_k * ((d.N + size - 1) / size);
    // In group order, where X comes from HBM, the rows of a short group's tile are read no
    // further ahead than that tile's time (64 x 1536 x 7168, rows a group: 256 488 us with
    // four stages, 553 with six; 320 531, 573; 384 573, 577; 448 618, 569).
    a.ns = !d.gather && a.slots <= 352L * std::min(a.E, a.slots) ? 4 : GW_NS;
    a.tiles_k = FastDiv((uint32_t)tiles_k), a.tiles_e = FastDiv((uint32_t)tiles);
    a.N = d.N, a.K = d.K, a.accumulate = d.accumulate ? 1 : 0, a.err = err;
    a.dy = (const __nv_bfloat16 *)d.dY, a.x = (const __nv_bfloat16 *)d.X, a.dw = d.dW;
    a.lddy = (long)d.lddy, a.ldx = (long)d.ldx;
    if (d.dw_dtype == K3MOE_BF16) return pair ? launch_gw<2, __nv_bfloat16>(a, s) : launch_gw<1, __nv_bfloat16>(a, s);
    return pair ? launch_gw<2, float>(a, s) : launch_gw<1, float>(a, s);
}

}  // namespace k3
