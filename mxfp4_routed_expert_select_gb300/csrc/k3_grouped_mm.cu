// k3_grouped_mm.cu -- products grouped by expert: every row of a routed batch,
// in 8 bits, with its own expert's MXFP4 matrix, on the block-scaled tensor cores
// (tcgen05.mma kind::mxf8f6f4, E2M1 x E4M3).
//
// C[i][n] = sum over blocks b of 2^(ea[i][b] + ew[n][b] - 254) times the sum of the 32
// code products of block b, for the rows i of each expert's group: the tensor core
// takes the codes as they are stored and applies both E8M0 scales itself, fp32 in
// TMEM.
//
// The weights' rows n take the MMA's 128 lanes, the group's rows its NT columns: a
// few tokens then cost a narrow MMA over the streamed weights.  A persistent CTA
// walks (expert, NT rows, 128 n) tiles; which exist follows from the group borders in
// device memory, which each CTA turns into a table of tile numbers.
//
// Roles: warp 0 issues scale copies and MMAs, warps 4 to 7 read the accumulators while
// the next tile's products run, and each further warp fills one stage of 128 of K: the
// weights and their scale atom by TMA (the copy spreads 16 four-bit codes over 16 bytes,
// the form this kind of MMA reads, so HBM and L2 move packed bytes), the rows' codes by
// TMA where they lie in group order, else row by row with asynchronous copies into the
// same swizzled form, and the rows' scale bytes.  (Gathered by TMA, four rows a copy of
// 72 clocks, the first version took 2.94 ms for 65536 rows x 1536 x 7168, as tiles 0.76.)
//
// Bound: few rows stream the weights (1 token x 16 of 896 experts x 1536 x 7168, 94 MB, 21.2
// us; 64 x 16 over 128 experts, 753 MB, 123, 6.1 TB/s), many the pairs' shared memory and
// MMAs (65536 rows with 64 experts x 1536 x 7168 gathered 533 us, 2.7 PFLOP/s, in group
// order 451).
//
// Every wait is bounded (2 s); a timeout sets the device error word and the CTA
// drains its copies and MMAs, frees TMEM and exits.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "k3_e4m3.cuh"
#include "k3_launch.cuh"
#include "k3_tcgen05.cuh"
#include "k3_tmem.cuh"

namespace k3 {
namespace {

constexpr int GM_M = 128;  // weight rows of a tile
constexpr int GM_W_MMA = 0, GM_W_EPI = 4, GM_W_FILL = 8;
constexpr int GM_MAX_E = 1024;
constexpr int GM_CTAS = 192, GM_MAX_NT = 64;  // the workspace has sums of that many CTAs' columns

struct GmArgs {
    const uint8_t *atoms;      // scale atoms of the weights, atoms_stride bytes from expert to expert
    long atoms_stride;
    const uint8_t *codes, *scales;  // of the rows
    int cstride, sstride;
    const int32_t *offsets, *order;
    int E, top_k, slots, gather, xrows;  // xrows: rows of the 8-bit matrix
    int N, nks, nka, tiles_n;  // nks: steps of 128 along K; nka: atoms per row tile
    float *parts;              // sums of parts of tiles, [CTA][columns][128]
    int32_t *counts;           // parts of a tile that are done
    void *C;
    long ldc;
    int accumulate, pairs;     // pairs: two columns of a bf16 C form an aligned word
    int *err;
};

// Instruction descriptor: E2M1 lanes, E4M3 columns, K-major, UE8M0 scales; sfid: which
// byte of the scale words.
__host__ __device__ constexpr uint32_t gm_idesc(int m, int n, uint32_t sfid)
{
    return (sfid << 4) | (5u << 7) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 4) << 24) | (sfid << 29);
}

// One step: the scale atoms of the stage to TMEM, then four MMAs of K = 32.
//   wlo, xlo   descriptor words of the code tiles; +2 per 32 of K
//   sal        descriptor word of the weights' atom, the rows' follow 32 words later
//   sf         TMEM column of the stage's scales: the weights' in 4, the rows' in 4
template <int NT>
K3_DEV void gm_step(uint32_t tacc, uint32_t wlo, uint32_t xlo, uint32_t sal, uint32_t sf, uint32_t acc)
{
    constexpr uint32_t AHI = (128u >> 4) | (1u << 14);  // atoms: 8 rows of 16 bytes 128 bytes apart, no swizzle
#define GM_MMA(k2, id, pred)                                                                                  \
    "add.u32 x, %1, " #k2 ";\n\tadd.u32 y, %2, " #k2 ";\n\tmov.b64 da, {x, %8};\n\tmov.b64 db, {y, %8};\n\t"  \
    "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], da, db, " id ", [%4], [z], " pred ";\n\t"
    asm volatile("{\n\t.reg .pred p, t, e;\n\t.reg .b64 d, da, db;\n\t.reg .b32 x, y, z;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, %6, %6;\n\tadd.u32 z, %4, 4;\n\t"
                 "mov.b64 d, {%3, %7};\n\t@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%4], d;\n\t"
                 "add.u32 x, %3, 32;\n\tmov.b64 d, {x, %7};\n\t@e tcgen05.cp.cta_group::1.32x128b.warpx4 [z], d;\n\t"
                 GM_MMA(0, "%6", "p") GM_MMA(2, "%9", "t") GM_MMA(4, "%10", "t") GM_MMA(6, "%11", "t") "}" ::"r"(tacc),
                 "r"(wlo), "r"(xlo), "r"(sal), "r"(sf), "r"(acc), "r"(gm_idesc(GM_M, NT, 0)), "r"(AHI), "r"(SW128_HI),
                 "r"(gm_idesc(GM_M, NT, 1)), "r"(gm_idesc(GM_M, NT, 2)), "r"(gm_idesc(GM_M, NT, 3))
                 : "memory");
#undef GM_MMA
}

// 128 rows x 128 codes of one expert's matrix, and the atom beside them.
K3_DEV void gm_load_w(uint32_t dst, const CUtensorMap *map, int x, int row, int e, uint32_t adst, const uint8_t *atom,
                      uint32_t bar)
{
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
                 "[%1, {%4, %5, %6}], [%7];\n\t"
                 "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%2], [%3], 512, [%7];\n\t}" ::"r"(
                     dst),
                 "l"((uint64_t)map), "r"(adst), "l"(atom), "r"(x), "r"(row), "r"(e), "r"(bar)
                 : "memory");
}

// The tiles of the batch, made by every CTA in shared memory: before[e] row tiles lie
// before expert e's, off[e] is its first place.
struct GmTable {
    int before[GM_MAX_E + 1], off[GM_MAX_E + 1], sums[32];
};
struct GmTile {
    int e, row, rows, n0;  // first row of C, rows of the group from there on (> 0), first weight row
};
K3_DEV void gm_table(GmTable &tab, const GmArgs &a, int tile_rows)
{
    constexpr int PER = (GM_MAX_E + 256 - 1) / 256;  // experts of each of the first 256 threads (a CTA has more)
    int v[PER], mine = 0;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, e0 = PER * (int)threadIdx.x;
    if (threadIdx.x < 256) {
        int lo = e0 <= a.E ? min(max(a.offsets[e0], 0), a.slots) : 0;
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const int e = e0 + i, hi = e < a.E ? min(max(a.offsets[e + 1], lo), a.slots) : lo;
            if (e <= a.E) tab.off[e] = lo;
            v[i] = (hi - lo + tile_rows - 1) / tile_rows;
            mine += v[i];
            lo = hi;
        }
        if (e0 + PER == a.E) tab.off[a.E] = lo;
    }
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) tab.sums[w] = x;
    __syncthreads();
    if (threadIdx.x < 256) {
        int at = x - mine;
        for (int i = 0; i < w; i++) at += tab.sums[i];
#pragma unroll
        for (int i = 0; i < PER; i++) {
            if (e0 + i <= a.E) tab.before[e0 + i] = at;
            at += v[i];
        }
        if (e0 + PER == a.E) tab.before[a.E] = at;
    }
    __syncthreads();
}
template <int NT>
K3_DEV GmTile gm_tile(const GmTable &tab, const GmArgs &a, int u)
{
    const int r = u / a.tiles_n;
    int lo = 0, hi = a.E;  // before[lo] <= r < before[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (tab.before[m] <= r)
            lo = m;
        else
            hi = m;
    }
    GmTile t;
    t.e = lo;
    t.row = tab.off[lo] + (r - tab.before[lo]) * NT;
    t.rows = tab.off[lo + 1] - t.row;
    t.n0 = (u - r * a.tiles_n) * GM_M;
    return t;
}
// What a CTA works on as its i-th piece: whole tiles in turn over the CTAs, as many as
// make full waves, and of the tiles that are left a part along K, several CTAs to a tile
// where there are enough (1 token x 16 experts x 1536 x 7168, 192 tiles on 152 SMs: 21.2
// us against 24.9).  slot: where a part leaves its sums; u < 0: nothing more.
struct GmPart {
    int u, k0, k1, of, slot;
};
constexpr int GM_MAX_PARTS = 8, GM_JOIN_STEPS = 16;  // joining parts takes as long as so many steps
K3_DEV GmPart gm_part(const GmArgs &a, int n_tiles, int i)
{
    const int ctas = (int)gridDim.x, me = (int)blockIdx.x, whole = n_tiles / ctas, left = n_tiles - whole * ctas;
    if (i < whole) return {i * ctas + me, 0, a.nks, 1, 0};
    int of = left ? min(ctas / left, GM_MAX_PARTS) : 1;
    if (a.nks - a.nks / of < GM_JOIN_STEPS) of = 1;
    if (i > whole || me >= left * of) return {-1, 0, 0, 1, 0};
    const int p = me % of;
    return {whole * ctas + me / of, a.nks * p / of, a.nks * (p + 1) / of, of, me};
}
// Row of the 8-bit matrix behind row i of C (0 should the order name none).
K3_DEV int gm_source(const GmArgs &a, int i)
{
    const int r = a.gather ? a.order[i] / a.top_k : i;
    return r >= 0 && r < a.xrows ? r : 0;
}

template <int NT>
struct GmCfg {
    static constexpr int W_BYTES = GM_M * 128, X_BYTES = NT * 128;
    static constexpr int OFF_X = W_BYTES, OFF_WA = OFF_X + X_BYTES, OFF_XA = OFF_WA + 512;
    static constexpr int STAGE = (OFF_XA + 512 + 1023) / 1024 * 1024;
    static constexpr int ROOM = 227 * 1024 - 1024 - 512 - (int)sizeof(GmTable);
    static constexpr int NS = ROOM / STAGE < 10 ? ROOM / STAGE : 10;
    static constexpr int THREADS = 32 * (GM_W_FILL + NS);  // a warp fills one stage
    static constexpr int TX_W = W_BYTES / 2 + 512, TX_X = X_BYTES;  // bytes as they lie in memory: the weights packed
    static constexpr int SF0 = 2 * NT, SF = 8;
    static constexpr int COLS_USED = SF0 + SF * NS;
    static constexpr int TMEM_COLS = COLS_USED <= 128 ? 128 : COLS_USED <= 256 ? 256 : 512;
    static constexpr int BARS = 2 * NS + 2 * 2 + 1;
    static constexpr int OFF_TAB = NS * STAGE + 256;
    static constexpr int SMEM = 1024 + OFF_TAB + (int)sizeof(GmTable);
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(COLS_USED <= 512, "TMEM layout");
    static_assert(BARS * 8 + 8 <= 256, "barriers");
};

// A lane's column n of C, rows 0 .. rows - 1 of the CH from o on.  pairs (bf16, N even,
// rows of C aligned for it): lanes swap every other value with their neighbour and store
// two columns of every other row, half as many stores (which bounded products of a
// short K: 65536 rows x 7168 x 1536 took 794 us with single ones, 572 with half of them).
template <typename CT, int CH>
K3_DEV void gm_put(const GmArgs &a, CT *o, int n, int rows, const uint32_t (&r)[CH])
{
    if constexpr (sizeof(CT) == 2) {
        if (a.pairs) {
            const int odd = threadIdx.x & 1;
            CT *p = o + (long)odd * a.ldc - odd;
#pragma unroll
            for (int c = 0; c < CH; c += 2) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? r[c] : r[c + 1], 1);
                const __nv_bfloat162 v = odd ? __floats2bfloat162_rn(__uint_as_float(got), __uint_as_float(r[c + 1]))
                                             : __floats2bfloat162_rn(__uint_as_float(r[c]), __uint_as_float(got));
                if (c + odd < rows && n < a.N) *(__nv_bfloat162 *)(p + (long)c * a.ldc) = v;
            }
            return;
        }
    }
    if (n >= a.N) return;
#pragma unroll
    for (int c = 0; c < CH; c++)
        if (c < rows) {
            CT *p = o + (long)c * a.ldc;
            if constexpr (sizeof(CT) == 2)
                *p = __float2bfloat16_rn(__uint_as_float(r[c]));
            else
                *p = a.accumulate ? *p + __uint_as_float(r[c]) : __uint_as_float(r[c]);
        }
}

template <int NT, typename CT>
__global__ void __launch_bounds__(GmCfg<NT>::THREADS, 1)
    k3_grouped_matmul(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, const GmArgs a)
{
    using C = GmCfg<NT>;
    constexpr int NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_addr(sm);
    uint64_t *bars = (uint64_t *)(sm + NS * C::STAGE);
    constexpr int B_FULL = 0, B_EMPTY = NS, B_ACCF = 2 * NS, B_ACCE = B_ACCF + 2, B_FIN = B_ACCE + 2;
    uint32_t *tmem_slot = (uint32_t *)(bars + C::BARS);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);
    GmTable &tab = *(GmTable *)(sm + C::OFF_TAB);
    auto bar = [&](int i) { return smem_addr(bars + i); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&wmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&xmap) : "memory");
        for (int i = 0; i < NS; i++) {
            mbar_init(bar(B_FULL + i), 2);  // the copies' bytes announced; the rows' part done
            mbar_init(bar(B_EMPTY + i), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(bar(B_ACCF + i), 1);
            mbar_init(bar(B_ACCE + i), 4);
        }
        mbar_init(bar(B_FIN), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == GM_W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(C::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *(volatile uint32_t *)tmem_slot;
    griddep_wait();
    gm_table(tab, a, NT);
    const int n_tiles = tab.before[a.E] * a.tiles_n;

    if (warp >= GM_W_FILL) {
        // -------------------------------------------------- a stage's filler
        // Every NS-th step of this CTA's parts.  Lanes 8 q .. 8 q + 7 copy the 16-byte
        // chunks of rows q, q + 4, ..; a lane has the scale words of rows lane, lane +
        // 32, ... of the tile.  Columns past the group keep what the stage held (they are
        // not stored).
        constexpr int J = (NT + 31) / 32, R = NT / 4;
        const int s = warp - GM_W_FILL;
        const uint32_t st = sbase + (uint32_t)(s * C::STAGE), full = bar(B_FULL + s);
        uint32_t turn = 0;
        int i = 0, tile = -1;
        GmPart part = gm_part(a, n_tiles, 0);
        int ks = part.k0 + s;
        GmTile t = {};
        const uint8_t *atoms = nullptr, *sp[J];
        int src[R];
        uint32_t w[J];
        for (;; ks += NS, turn++) {
            while (part.u >= 0 && ks >= part.k1) {
                const int over = ks - part.k1;
                part = gm_part(a, n_tiles, ++i);
                ks = part.k0 + over;
            }
            if (part.u < 0) break;
            const bool entered = i != tile;
            if (entered) {
                tile = i;
                t = gm_tile<NT>(tab, a, part.u);
                atoms = a.atoms + (long)t.e * a.atoms_stride + (long)(t.n0 / 128) * a.nka * 512;
            }
            // before its first completion an EMPTY barrier's odd phase counts as passed
            if (!__all_sync(0xffffffffu, tc_wait(bar(B_EMPTY + s), (turn & 1) ^ 1u, a.err, abort_flag))) break;
            // the weights first: they have the longest way
            if (lane == 0) mbar_arrive_expect_tx(full, C::TX_W + (a.gather ? 0 : C::TX_X));
            __syncwarp();
            gm_load_w(st, &wmap, ks * 128, t.n0, t.e, st + C::OFF_WA, atoms + (long)ks * 512, full);
            if (entered) {
#pragma unroll
                for (int j = 0; j < J; j++)
                    sp[j] = lane + 32 * j < t.rows ? a.scales + (long)gm_source(a, t.row + lane + 32 * j) * a.sstride : nullptr;
                if (a.gather)
#pragma unroll
                    for (int i = 0; i < R; i++) {
                        const int r = 4 * i + (lane >> 3);
                        src[i] = r < t.rows ? gm_source(a, t.row + r) : -1;
                    }
            }
#pragma unroll
            for (int j = 0; j < J; j++) w[j] = sp[j] ? *(const uint32_t *)(sp[j] + 4 * ks) : 0u;
            if (a.gather) {
                const uint8_t *base = a.codes + (long)ks * 128 + (lane & 7) * 16;
#pragma unroll
                for (int i = 0; i < R; i++) {
                    const int r = 4 * i + (lane >> 3);
                    if (src[i] >= 0)
                        copy16(st + C::OFF_X + (uint32_t)(r * 128 + (((lane & 7) ^ (r & 7)) << 4)), base + (long)src[i] * a.cstride);
                }
            } else if (lane == 0) {
                tma_load_2d(st + C::OFF_X, &xmap, ks * 128, t.row, full);
            }
#pragma unroll
            for (int j = 0; j < J; j++) *(uint32_t *)(sm + s * C::STAGE + C::OFF_XA + lane * 16 + j * 4) = w[j];
            if (a.gather) asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full);
        }
        // drain: every copy issued here has landed before the CTA exits (the last turn's;
        // earlier ones were waited for before their stage's reuse)
        if (turn) mbar_wait(full, (turn - 1) & 1, a.err);
        __syncwarp();
    } else if (warp == GM_W_MMA) {
        // -------------------------------------------------------------- MMA
        uint32_t ut = 0, phase = 0;
        int s = 0;
        bool ok = true, ready = false;
        const uint32_t lo = sw128_lo(sbase);
        constexpr uint32_t SD = C::STAGE / 16;  // descriptor words between stages
        for (;; ut++) {
            const GmPart part = gm_part(a, n_tiles, (int)ut);
            if (part.u < 0) break;
            const int buf = (int)(ut & 1);
            if (ut >= 2 && !__all_sync(0xffffffffu, tc_wait(bar(B_ACCE + buf), (ut / 2 - 1) & 1, a.err, abort_flag)))
                break;
            tc_fence_after();
            for (int ks = part.k0; ks < part.k1; ks++) {
                if (!ready && !__all_sync(0xffffffffu, tc_wait(bar(B_FULL + s), phase, a.err, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int sn = s + 1 == NS ? 0 : s + 1;
                const uint32_t pn = sn ? phase : phase ^ 1u;
                // ask for the next stage before this one is issued, look at the answer after
                const bool next = mbar_test(bar(B_FULL + sn), pn);
                const uint32_t d = lo + (uint32_t)s * SD;
                gm_step<NT>(tmem + (uint32_t)(buf * NT), d, d + C::OFF_X / 16, d + C::OFF_WA / 16,
                            tmem + (uint32_t)(C::SF0 + C::SF * s), ks > part.k0 ? 1u : 0u);
                mma_commit(bar(B_EMPTY + s));
                ready = __all_sync(0xffffffffu, next);
                s = sn;
                phase = pn;
            }
            if (!ok) break;
            mma_commit(bar(B_ACCF + buf));
        }
        // every MMA and copy issued above has completed before TMEM is freed
        mma_commit(bar(B_FIN));
        mbar_wait(bar(B_FIN), 0, a.err);
        __syncwarp();
    } else if (warp >= GM_W_EPI) {
        // --------------------------------------------------------- epilogue
        const int q = warp - GM_W_EPI;  // TMEM lane quadrant: weight rows 32 q .. 32 q + 31 of the tile
        constexpr int CH = NT < 32 ? 16 : 32, NCH = NT / CH;
        for (uint32_t ut = 0;; ut++) {
            const GmPart part = gm_part(a, n_tiles, (int)ut);
            if (part.u < 0) break;
            const int buf = (int)(ut & 1);
            const GmTile t = gm_tile<NT>(tab, a, part.u);
            if (!__all_sync(0xffffffffu, tc_wait(bar(B_ACCF + buf), (ut / 2) & 1, a.err, abort_flag))) break;
            tc_fence_after();
            const uint32_t tacc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * NT);
            const int n = t.n0 + q * 32 + lane, cols = min(t.rows, NT);
            float *const mine = a.parts + ((long)part.slot * NT) * GM_M + q * 32 + lane;  // [column][128]
#pragma unroll 1
            for (int j = 0; j < NCH; j++) {
                uint32_t r[CH];
                tmem_ld_chunk(tacc + (uint32_t)(j * CH), r);
                if (j == NCH - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_ACCE + buf));
                }
                if (part.of == 1) {
                    gm_put<CT, CH>(a, (CT *)a.C + (long)(t.row + j * CH) * a.ldc + n, n, t.rows - j * CH, r);
                } else {
#pragma unroll
                    for (int c = 0; c < CH; c++)
                        if (j * CH + c < cols) __stcg(mine + (long)(j * CH + c) * GM_M, __uint_as_float(r[c]));
                }
            }
            if (part.of == 1) continue;
            // A part of a tile: the CTA that is last to leave its sums adds all parts up,
            // in their order, and leaves the count at zero.
            __threadfence();
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (threadIdx.x == GM_W_EPI * 32) tab.sums[0] = atomicAdd(a.counts + part.slot / part.of, 1) == part.of - 1;
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (!tab.sums[0]) continue;
            __threadfence();
            const float *all = a.parts + ((long)(part.slot - part.slot % part.of) * NT) * GM_M + q * 32 + lane;
#pragma unroll 1
            for (int j = 0; j < NCH && j * CH < cols; j++) {
                uint32_t r[CH];
#pragma unroll
                for (int c = 0; c < CH; c++) r[c] = 0u;
#pragma unroll 1
                for (int p = 0; p < part.of; p++)
#pragma unroll
                    for (int c = 0; c < CH; c++)
                        if (j * CH + c < cols)
                            r[c] = __float_as_uint(__uint_as_float(r[c]) + __ldcg(all + ((long)p * NT + j * CH + c) * GM_M));
                gm_put<CT, CH>(a, (CT *)a.C + (long)(t.row + j * CH) * a.ldc + n, n, t.rows - j * CH, r);
            }
            if (threadIdx.x == GM_W_EPI * 32) a.counts[part.slot / part.of] = 0;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == GM_W_MMA) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS)
                     : "memory");
    }
}

// ---------------------------------------------------------------- CTA pairs
//
// Large groups.  A lone CTA's 128 x 128 tile brings 32 KB per 128 of K into its shared
// memory and reads as much, 512 clocks of its bandwidth for 256 clocks of MMAs.  A pair
// (cta_group::2) works on 256 weight rows x up to 256 rows of the group together: each
// CTA loads its own 128 weight rows and half of the group's rows, and the MMA reads both
// halves, so that shared memory and tensor cores are both busy for 512 clocks a step.
//
// The MMA's columns are the rows of the group, so their number follows the tile: a
// group is cut into equal tiles of whole 32 rows, and a short tile costs a short MMA.
//
// The even CTA issues for both.  Every stage has two filling warps in each CTA, and two
// further warps bring the rows' scale bytes of all stages; the copies of both CTAs are
// counted on the even CTA's barrier, and each warp arrives there when its part is in place.
// (A lane reads 16 scale bytes of a row, four steps' worth; a word for each step, by the
// stage's own warps, was a line of L1 a lane: 65536 rows x 1536 x 7168 with 64 experts 547
// us gathered and 457 in group order, so 528 and 440.)  Warp 1 finds out each tile (its
// expert, its rows, which rows of the 8-bit matrix they are) ahead of the others and
// leaves it in a ring: a search takes 1000 clocks, a sixth of a tile with K = 1536.

constexpr int GP_EPI = 8, GP_FILL = 2, GP_NT = 256, GP_RING = 4;
constexpr int GP_SC = 2;  // warps of scale bytes, 128 rows each
constexpr int GP_W_PLAN = 1, GP_W_SCALE = 2, GP_W_FILL = GM_W_EPI + GP_EPI;
constexpr int GP_OFF_X = GM_M * 128, GP_OFF_WA = 2 * GM_M * 128, GP_OFF_XA = GP_OFF_WA + 512;
constexpr int GP_STAGE = GP_OFF_XA + 1024 + 512, GP_NS = 6;
constexpr int GP_THREADS = 32 * (GP_W_FILL + GP_FILL * GP_NS);
constexpr int GP_BOX = 32;  // rows of a TMA copy of the group's rows
// TMEM: two accumulators of up to 256 columns, the second from column 192 on, then five
// slots of scales.  The columns that the accumulators share are read first: the next
// tile's products wait for that.  (Tiles of up to 192 rows with accumulators of their
// own lost: 65536 rows x 1536 x 7168 545 against 508 us, x 7168 x 1536 691 against 671.)
constexpr int GP_OVER = 192, GP_SF0 = GP_OVER + GP_NT, GP_SF = 12, GP_SLOTS = 5;
constexpr int GP_BARS = 2 * GP_NS + 2 * 2 + 1 + 2 * GP_RING;
constexpr int GP_OFF_TAB = GP_NS * GP_STAGE + 256;
// A tile: tiles of a group are equal but for the last.
struct GpTile {
    int e, row, rows, n0, half;  // expert (-1: no more tiles); half: columns of each CTA
    int src[GP_NT];              // rows of the 8-bit matrix behind its rows
};
constexpr int GP_OFF_RING = GP_OFF_TAB + (int)sizeof(GmTable);
constexpr int GP_SMEM = 1024 + GP_OFF_RING + GP_RING * (int)sizeof(GpTile);
static_assert(GP_STAGE % 1024 == 0, "swizzled tiles are 1024-byte aligned");
static_assert(GP_SLOTS == GP_NS - 1, "a slot of scales is free when the next stage is full");
static_assert(GP_SMEM <= 232448 && GP_SF0 + GP_SF * GP_SLOTS <= 512 && GP_BARS * 8 + 8 <= 256, "shared memory, TMEM");

// One step for the pair: each CTA's atoms to its own TMEM, four MMAs of K = 32.
K3_DEV void gp_step(uint32_t tacc, uint32_t wlo, uint32_t xlo, uint32_t sal, uint32_t sf, uint32_t acc, uint32_t id)
{
    constexpr uint32_t AHI = (128u >> 4) | (1u << 14);
    constexpr uint32_t ID1 = (1u << 4) | (1u << 29);  // the next scale byte of both
#define GP_CP(col, off) \
    "add.u32 x, %3, " #off ";\n\tadd.u32 y, %4, " #col ";\n\tmov.b64 d, {x, %7};\n\t@e tcgen05.cp.cta_group::2.32x128b.warpx4 [y], d;\n\t"
#define GP_MMA(k2, pred)                                                                                      \
    "add.u32 x, %1, " #k2 ";\n\tadd.u32 y, %2, " #k2 ";\n\tmov.b64 da, {x, %8};\n\tmov.b64 db, {y, %8};\n\t"  \
    "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], da, db, i, [%4], [z], " pred ";\n\t" \
    "add.u32 i, i, %9;\n\t"
    asm volatile("{\n\t.reg .pred p, t, e;\n\t.reg .b64 d, da, db;\n\t.reg .b32 x, y, z, i;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, %6, %6;\n\tadd.u32 z, %4, 4;\n\t"
                 "mov.b32 i, %6;\n\t" GP_CP(0, 0) GP_CP(4, 32) GP_CP(8, 64) GP_MMA(0, "p") GP_MMA(2, "t") GP_MMA(4, "t")
                     GP_MMA(6, "t") "}" ::"r"(tacc),
                 "r"(wlo), "r"(xlo), "r"(sal), "r"(sf), "r"(acc), "r"(id), "r"(AHI), "r"(SW128_HI), "r"(ID1)
                 : "memory");
#undef GP_CP
#undef GP_MMA
}
// gm_load_w with its bytes counted on barrier `bar`, a shared::cluster address (the
// even CTA's); the atom by a tensor copy, which can name it.
K3_DEV void gp_load_w(uint32_t dst, const CUtensorMap *map, int x, int row, int e, uint32_t adst, const CUtensorMap *amap,
                      int ak, int art, uint32_t bar)
{
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
                 "[%1, {%4, %5, %6}], [%9];\n\t"
                 "@e cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%2], "
                 "[%3, {0, %7, %8, %6}], [%9];\n\t}" ::"r"(dst),
                 "l"((uint64_t)map), "r"(adst), "l"((uint64_t)amap), "r"(x), "r"(row), "r"(e), "r"(ak), "r"(art), "r"(bar)
                 : "memory");
}
// What the CTAs' threads have staged is acquired from both (pair_acquire).  The waits for
// the other CTA's commits and for read accumulators are of the CTA's scope: behind them lie
// MMAs that have completed and tensor memory, ordered by the tcgen05 fences, and no memory
// that a thread has written.  (An acquire at cluster scope makes a warp wait for its own
// stores; with the fence behind every EMPTY wait 443 us in group order were 462.)

// Tile u into the ring, by a whole warp.
K3_DEV void gp_plan(GpTile &t, const GmTable &tab, const GmArgs &a, int u)
{
    const int lane = threadIdx.x & 31, r = u / a.tiles_n;
    int lo = 0, hi = a.E;  // before[lo] <= r < before[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (tab.before[m] <= r)
            lo = m;
        else
            hi = m;
    }
    const int n = tab.off[lo + 1] - tab.off[lo], tiles = tab.before[lo + 1] - tab.before[lo];
    const int h = ((n + tiles - 1) / tiles + 31) & ~31, i = r - tab.before[lo];
    const int row = tab.off[lo] + i * h, rows = min(h, n - i * h);
    if (lane == 0) {
        t.e = lo, t.row = row, t.rows = rows;
        t.half = ((rows + 31) & ~31) / 2;
        t.n0 = (u - r * a.tiles_n) * 2 * GM_M;
    }
#pragma unroll
    for (int j = 0; j < GP_NT / 32; j++)
        if (32 * j < rows) t.src[32 * j + lane] = gm_source(a, row + min(32 * j + lane, rows - 1));
}

template <typename CT>
__global__ void __launch_bounds__(GP_THREADS, 1)
    k3_grouped_matmul_pair(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap,
                           const __grid_constant__ CUtensorMap xmap, const GmArgs a)
{
    constexpr int NS = GP_NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_addr(sm);
    uint64_t *bars = (uint64_t *)(sm + NS * GP_STAGE);
    constexpr int B_FULL = 0, B_EMPTY = NS, B_ACCF = 2 * NS, B_ACCE = B_ACCF + 2, B_FIN = B_ACCE + 2, B_TILEF = B_FIN + 1,
                  B_TILEE = B_TILEF + GP_RING;
    uint32_t *tmem_slot = (uint32_t *)(bars + GP_BARS);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);
    GmTable &tab = *(GmTable *)(sm + GP_OFF_TAB);
    GpTile *ring = (GpTile *)(sm + GP_OFF_RING);
    auto bar = [&](int i) { return smem_addr(bars + i); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();  // 0: the CTA that issues
    const int first = (int)blockIdx.x >> 1, step = (int)gridDim.x >> 1;

    if (threadIdx.x == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&wmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&amap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&xmap) : "memory");
        for (int i = 0; i < NS; i++) {
            mbar_init(bar(B_FULL + i), 1 + 2 * (GP_FILL + GP_SC));  // the bytes announced; each warp's part done
            mbar_init(bar(B_EMPTY + i), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(bar(B_ACCF + i), 1);
            mbar_init(bar(B_ACCE + i), 2 * GP_EPI);  // the epilogue warps of both CTAs
        }
        for (int i = 0; i < GP_RING; i++) {
            mbar_init(bar(B_TILEF + i), 1);
            mbar_init(bar(B_TILEE + i), GP_FILL * NS + GP_SC + GP_EPI + (rank == 0));  // the warps that read it
        }
        mbar_init(bar(B_FIN), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == GM_W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the other CTA's barriers are initialised
    tc_fence_after();
    const uint32_t tmem = __reduce_max_sync(0xffffffffu, *(volatile uint32_t *)tmem_slot);
    griddep_wait();
    gm_table(tab, a, GP_NT);
    const int n_tiles = tab.before[a.E] * a.tiles_n;

    // The ring as a reader sees it: tile i of this pair; a warp that has what it needs of
    // it lets it go.
    auto tile_in = [&](uint32_t i) {
        return __all_sync(0xffffffffu, tc_wait(bar(B_TILEF + (int)(i % GP_RING)), (i / GP_RING) & 1, a.err, abort_flag));
    };
    auto tile_out = [&](uint32_t i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_TILEE + (int)(i % GP_RING)));
    };

    if (warp == GP_W_PLAN) {
        // ------------------------------------------------------------ tiles
        uint32_t i = 0;
        for (int u = first;; u += step, i++) {
            // before its first completion a barrier's odd phase counts as passed
            if (!__all_sync(0xffffffffu,
                            tc_wait(bar(B_TILEE + (int)(i % GP_RING)), ((i / GP_RING) & 1) ^ 1u, a.err, abort_flag)))
                break;
            GpTile &t = ring[i % GP_RING];
            if (u < n_tiles)
                gp_plan(t, tab, a, u);
            else if (lane == 0)
                t.e = -1;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_TILEF + (int)(i % GP_RING)));
            if (u >= n_tiles) break;
        }
    } else if (warp >= GP_W_SCALE && warp < GM_W_EPI) {
        // ------------------------------------------------------- scale bytes
        // Of each tile's 256 rows a warp has 128, a lane every 32nd, four steps at a time,
        // the next four on their way while these are handed out.
        const int f = warp - GP_W_SCALE;
        const bool wide = a.nks % 4 == 0 && ((uintptr_t)a.scales & 15u) == 0;
        uint32_t phase = 1;  // before its first completion a barrier's odd phase counts as passed
        int s = 0;
        for (uint32_t i = 0;; i++) {
            if (!tile_in(i)) break;
            const GpTile *t = ring + i % GP_RING;
            if (t->e < 0) break;
            const uint32_t *row[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int r = 128 * f + 32 * j + lane;
                row[j] = r < t->rows ? (const uint32_t *)(a.scales + (long)t->src[r] * a.sstride) : nullptr;
            }
            tile_out(i);
            uint4 now[4], next[4];
            auto load = [&](int ks) {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    next[j] = make_uint4(0u, 0u, 0u, 0u);
                    if (!row[j] || ks >= a.nks) continue;
                    if (wide) {
                        next[j] = *(const uint4 *)(row[j] + ks);
                    } else {
                        next[j].x = row[j][ks];
                        if (ks + 1 < a.nks) next[j].y = row[j][ks + 1];
                        if (ks + 2 < a.nks) next[j].z = row[j][ks + 2];
                        if (ks + 3 < a.nks) next[j].w = row[j][ks + 3];
                    }
                }
            };
            load(0);
            bool ok = true;
            for (int ks = 0; ks < a.nks && ok; ks += 4) {
#pragma unroll
                for (int j = 0; j < 4; j++) now[j] = next[j];
                load(ks + 4);
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    if (ks + q >= a.nks) break;
                    if (!__all_sync(0xffffffffu, tc_wait(bar(B_EMPTY + s), phase, a.err, abort_flag))) {
                        ok = false;
                        break;
                    }
                    auto word = [&](const uint4 &v) { return q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w; };
                    *(uint4 *)(sm + s * GP_STAGE + GP_OFF_XA + f * 512 + lane * 16) =
                        make_uint4(word(now[0]), word(now[1]), word(now[2]), word(now[3]));
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) pair_arrive(bar(B_FULL + s), addr_of_rank(bar(B_FULL + s), 0), rank);
                    if (++s == NS) s = 0, phase ^= 1u;
                }
            }
            if (!ok) break;
        }
    } else if (warp >= GP_W_FILL) {
        // -------------------------------------------------- a stage's fillers
        // Every NS-th step of this pair's tiles.  Of this CTA's rows (half the tile's)
        // each warp copies 64, lanes 8 q .. 8 q + 7 the 16-byte chunks of rows q, q + 4,
        // ...
        constexpr int R = 64 / 4;
        const int s = (warp - GP_W_FILL) / GP_FILL, f = (warp - GP_W_FILL) % GP_FILL;
        const uint32_t st = sbase + (uint32_t)(s * GP_STAGE), full0 = addr_of_rank(bar(B_FULL + s), 0);
        uint32_t turn = 0, tiles = 0;
        int ks = s;
        bool ok = tile_in(0);
        const GpTile *t = ring;
        for (; ok && t->e >= 0; ks += NS, turn++) {
            while (ks >= a.nks && ok && t->e >= 0) {
                ks -= a.nks;
                tile_out(tiles++);
                ok = tile_in(tiles);
                t = ring + tiles % GP_RING;
            }
            if (!ok || t->e < 0) break;
            const int rows = t->rows, half = t->half;
            if (!__all_sync(0xffffffffu, tc_wait(bar(B_EMPTY + s), (turn & 1) ^ 1u, a.err, abort_flag))) break;
            const int boxes = (half + GP_BOX - 1) / GP_BOX;
            if (f == 0) {
                if (rank == 0 && lane == 0)
                    mbar_arrive_expect_tx(bar(B_FULL + s), 2u * (GM_M * 64 + 512 + (a.gather ? 0 : boxes * GP_BOX * 128)));
                __syncwarp();
                gp_load_w(st, &wmap, ks * 128, t->n0 + rank * GM_M, t->e, st + GP_OFF_WA, &amap, ks, t->n0 / 128 + rank, full0);
            }
            if (a.gather) {
                const uint8_t *base = a.codes + (long)ks * 128 + (lane & 7) * 16;
#pragma unroll
                for (int i = 0; i < R; i++) {
                    const int r = 64 * f + 4 * i + (lane >> 3), c = rank * half + r;
                    if (r < half && c < rows)
                        copy16(st + GP_OFF_X + (uint32_t)(r * 128 + (((lane & 7) ^ (r & 7)) << 4)), base + (long)t->src[c] * a.cstride);
                }
            } else if (f == 1 && lane < boxes) {
                pair_load_2d(st + GP_OFF_X + (uint32_t)(lane * GP_BOX * 128), &xmap, ks * 128, t->row + rank * half + lane * GP_BOX,
                          full0);
            }
            if (a.gather) {
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) pair_arrive(bar(B_FULL + s), full0, rank);
        }
        // drain: the last turn's copies of both CTAs have landed before the even CTA
        // exits; the odd one waits in the closing cluster barrier
        if (rank == 0 && turn) mbar_wait(bar(B_FULL + s), (turn - 1) & 1, a.err);
        __syncwarp();
    } else if (warp == GM_W_MMA && rank == 1) {
        // the even CTA issues for both
    } else if (warp == GM_W_MMA) {
        // -------------------------------------------------------------- MMA
        uint32_t phase = 0, slot = 0, it = 0;
        int s = 0;
        bool ready = false;
        const uint32_t lo = sw128_lo(sbase);
        constexpr uint32_t SD = GP_STAGE / 16;  // descriptor words between stages
        for (uint32_t ut = 0;; ut++) {
            const int buf = (int)(ut & 1);
            bool ok = tile_in(ut);
            const GpTile *t = ring + ut % GP_RING;
            if (!ok || t->e < 0) break;
            const uint32_t id = __reduce_max_sync(0xffffffffu, gm_idesc(2 * GM_M, 2 * t->half, 0));
            tile_out(ut);
            // the epilogue frees the columns that a tile's accumulator shares with the next
            if (ut >= 1) {
                const uint32_t p = ut - 1;
                if (!__all_sync(0xffffffffu, tc_wait(bar(B_ACCE + (int)(p & 1)), (p / 2) & 1, a.err, abort_flag)))
                    break;
            }
            tc_fence_after();
            for (int ks = 0; ks < a.nks; ks++, it++) {
                if (!ready && !__all_sync(0xffffffffu, tc_wait_pair(bar(B_FULL + s), phase, a.err, abort_flag))) {
                    ok = false;
                    break;
                }
                pair_acquire();
                tc_fence_after();
                const int sn = s + 1 == NS ? 0 : s + 1;
                const uint32_t pn = sn ? phase : phase ^ 1u;
                // look at the next stage while this one is issued
                ready = __all_sync(0xffffffffu, mbar_test_pair(bar(B_FULL + sn), pn));
                // The products that read this slot of scales before have completed: the
                // next stage could only be filled behind them.  Where it is not yet, wait.
                if (!ready && it >= (uint32_t)GP_SLOTS &&
                    !__all_sync(0xffffffffu, tc_wait(bar(B_EMPTY + sn), ((it - GP_SLOTS) / NS) & 1, a.err, abort_flag))) {
                    ok = false;
                    break;
                }
                const uint32_t d = lo + (uint32_t)s * SD;
                gp_step(tmem + (uint32_t)(buf * GP_OVER), d, d + GP_OFF_X / 16, d + GP_OFF_WA / 16,
                        tmem + (uint32_t)GP_SF0 + slot, ks ? 1u : 0u, id);
                pair_commit(bar(B_EMPTY + s));
                s = sn;
                phase = pn;
                slot = slot + GP_SF == GP_SF * GP_SLOTS ? 0 : slot + GP_SF;
            }
            if (!ok) break;
            pair_commit(bar(B_ACCF + buf));
        }
        // every MMA and copy issued above has completed before TMEM is freed
        pair_commit(bar(B_FIN));
        mbar_wait(bar(B_FIN), 0, a.err);
        __syncwarp();
    } else if (warp >= GM_W_EPI) {
        // --------------------------------------------------------- epilogue
        // A lane holds one weight row n, 32 columns (rows of C) at a time; the two warps
        // of a quadrant take alternate pieces, first the one each in the columns shared
        // with the other accumulator (the first one's last, the second one's first).
        const int q = warp & 3, other = (warp - GM_W_EPI) >> 2;
        constexpr int PIECES = GP_NT / 32, OVER = GP_OVER / 32;
        static_assert(PIECES - OVER == 2, "a shared piece for each warp of a quadrant");
        for (uint32_t ut = 0;; ut++) {
            const int buf = (int)(ut & 1);
            if (!tile_in(ut)) break;
            const GpTile *t = ring + ut % GP_RING;
            const int e = t->e, row = t->row, rows = t->rows, n = t->n0 + rank * GM_M + q * 32 + lane;
            if (e < 0) break;
            tile_out(ut);
            if (!__all_sync(0xffffffffu, tc_wait(bar(B_ACCF + buf), (ut / 2) & 1, a.err, abort_flag))) break;
            tc_fence_after();
            const uint32_t tacc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * GP_OVER);
#pragma unroll 1
            for (int i = other; i < PIECES; i += 2) {
                const int j = buf ? i : (i + OVER) % PIECES;
                const bool on = j * 32 < rows;
                uint32_t r[32];
                if (on) tmem_ld_chunk(tacc + (uint32_t)(j * 32), r);
                if (i == other) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_rank(bar(B_ACCE + buf), 0);
                }
                if (on) gm_put<CT, 32>(a, (CT *)a.C + (long)(row + j * 32) * a.ldc + n, n, rows - j * 32, r);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // The even CTA's last commits have arrived here before this CTA may exit.  The
    // last tile has been read, so they are on their way: a short wait after a call of any
    // length.
    if (rank == 1 && warp == GM_W_MMA) {
        volatile int ignore = 0;  // after an abort too
        if (lane == 0) tc_wait(bar(B_FIN), 0, a.err, &ignore);
        __syncwarp();
    }
    cluster_sync();  // neither CTA leaves, or frees TMEM, while the other's work may reach it
    if (warp == GM_W_MMA) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// ---------------------------------------------------------------- launchers

int weight_map(CUtensorMap *map, const k3moe_mx_experts *W)
{
    const cuuint64_t wd[3] = {(cuuint64_t)W->in, (cuuint64_t)W->rows, (cuuint64_t)W->E},
                     ws[2] = {(cuuint64_t)W->in / 2, (cuuint64_t)W->codes_stride};
    const cuuint32_t wb[3] = {128, GM_M, 1};
    return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 3, W->codes, wd, ws, wb, CU_TENSOR_MAP_SWIZZLE_128B);
}
// The rows' codes in boxes of 128 bytes x `rows`.
int row8_map(CUtensorMap *map, const k3moe_mx8_rows *A, int rows)
{
    const cuuint64_t xd[2] = {(cuuint64_t)A->in, (cuuint64_t)A->rows}, xs[1] = {(cuuint64_t)op_in_padded(A->in)};
    const cuuint32_t xb[2] = {128, (cuuint32_t)rows};
    return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, A->codes, xd, xs, xb, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int NT, typename CT>
int launch_gm(const k3moe_mx8_rows *A, const k3moe_mx_experts *W, const GmArgs &a, cudaStream_t s)
{
    using C = GmCfg<NT>;
    CUtensorMap wmap, xmap;
    int st = weight_map(&wmap, W);
    if (st == K3MOE_OK) st = row8_map(&xmap, A, NT);
    if (st != K3MOE_OK) return st;
    if (ensure_smem((const void *)k3_grouped_matmul<NT, CT>, C::SMEM) != K3MOE_OK) return K3MOE_ECUDA;
    // as many CTAs as there are SMs and places for parts of tiles
    if (launch_pdl(k3_grouped_matmul<NT, CT>, dim3((unsigned)std::min(num_sms(), GM_CTAS)), dim3(C::THREADS), C::SMEM, s,
                   wmap, xmap, a) != cudaSuccess) {
        cudaGetLastError();
        return K3MOE_ECUDA;
    }
    return K3MOE_OK;
}
template <typename CT>
int launch_gp(const k3moe_mx8_rows *A, const k3moe_mx_experts *W, GmArgs a, cudaStream_t s)
{
    CUtensorMap wmap, amap, xmap;
    int st = weight_map(&wmap, W);
    if (st == K3MOE_OK) st = row8_map(&xmap, A, GP_BOX);
    // the scale atoms, [expert][row tile][k][512 bytes], one at a time
    const cuuint64_t nk = (cuuint64_t)a.nka, ad[4] = {128, nk, (cuuint64_t)op_row_tiles(W->rows), (cuuint64_t)W->E},
                     as[3] = {512, nk * 512, (cuuint64_t)W->atoms_stride};
    const cuuint32_t ab[4] = {128, 1, 1, 1};
    if (st == K3MOE_OK)
        st = encode_map(&amap, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, W->atoms, ad, as, ab, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (st != K3MOE_OK) return st;
    if (ensure_smem((const void *)k3_grouped_matmul_pair<CT>, GP_SMEM) != K3MOE_OK) return K3MOE_ECUDA;
    a.tiles_n = (a.N + 2 * GM_M - 1) / (2 * GM_M);
    const long most = std::min<long>(a.slots, (long)a.E + a.slots / GP_NT) * a.tiles_n;  // tiles there can be
    if (launch_dependent(true, 2, k3_grouped_matmul_pair<CT>, dim3((unsigned)(2 * std::min<long>(most, num_sms() / 2))),
                         dim3(GP_THREADS), GP_SMEM, s, wmap, amap, xmap, a) != cudaSuccess) {
        cudaGetLastError();
        return K3MOE_ECUDA;
    }
    return K3MOE_OK;
}
// The form by the time it would take: a time per step and one per tile, times the tiles of
// an SM (or a pair of them), one at least.  An expert with `avg` rows makes about avg /
// height + 1/2 tiles.  The times are fitted to 157 measured shapes of 8 to 384 experts with
// 1 to 300 rows each; the form they choose is 0.5% behind the best one on average, 13% at
// worst.  Measured on 64 experts, in us, with 16, 32 and 64 rows and pairs:
//   1536 x 7168, 8 rows an expert 68 70 75 100, 16 rows 84 71 82 101, 32 rows 131 88 94
//   106, 64 rows 230 140 116 109, 192 rows 626 351 233 138;
//   7168 x 1536, 8 rows 71 72 82 98, 32 rows 158 114 102 100, 64 rows 282 185 151 105.
// (Single tiles of 128 rows never won: 16 to 35% behind pairs from 128 rows on.)
int tile_rows(int E, long slots, int N, int nks)
{
    const long hit = std::min<long>(E, slots), sms = num_sms(), tiles_n = ((long)N + GM_M - 1) / GM_M;
    const struct {
        int rows, step, tile;  // of a tile; ns
        long columns, at_once;
    } forms[4] = {{16, 226, 600, tiles_n, sms},
                  {32, 225, 700, tiles_n, sms},
                  {64, 210, 1600, tiles_n, sms},
                  {GP_NT, 255, 1500, (tiles_n + 1) / 2, std::max(1L, sms / 2)}};
    int best = 0;
    double cost = 0;
    for (const auto &f : forms) {
        const long half_tiles = std::max(2 * hit, 2 * slots / f.rows + hit);
        const double tiles = std::max(1.0, 0.5 * (double)half_tiles * (double)f.columns / (double)f.at_once);
        const double c = tiles * ((double)f.step * nks + f.tile);
        if (best == 0 || c < cost) cost = c, best = f.rows;
    }
    return best;
}
template <typename CT>
int launch_gm_ct(const k3moe_mx8_rows *A, const k3moe_mx_experts *W, const GmArgs &a, cudaStream_t s)
{
    switch (tile_rows(a.E, a.slots, a.N, a.nks)) {
    case 16: return launch_gm<16, CT>(A, W, a, s);
    case 32: return launch_gm<32, CT>(A, W, a, s);
    case 64: return launch_gm<64, CT>(A, W, a, s);
    default: return launch_gp<CT>(A, W, a, s);
    }
}

}  // namespace

// The workspace: a count for each tile that has parts (zero between calls), and the sums
// of parts of tiles.
size_t grouped_matmul_workspace_bytes() { return GM_CTAS * (sizeof(float) * GM_M * GM_MAX_NT + sizeof(int32_t)); }

int grouped_matmul_rows(int E, long slots, int N, int in) { return tile_rows(E, slots, N, in / 128); }

int launch_grouped_matmul(const k3moe_grouped_matmul_desc &d, int *err, cudaStream_t s)
{
    const k3moe_mx8_rows *A = d.host_A;
    const k3moe_mx_experts *W = d.host_W;
    const k3moe_groups *g = d.host_groups;
    GmArgs a = {};
    a.atoms = W->atoms, a.atoms_stride = (long)W->atoms_stride;
    a.codes = A->codes, a.scales = A->scales, a.cstride = op_in_padded(A->in), a.sstride = mx8_scale_stride(A->in);
    a.offsets = g->offsets, a.order = g->order;
    a.E = g->E, a.top_k = g->top_k, a.slots = g->tokens * g->top_k, a.gather = d.gather ? 1 : 0, a.xrows = A->rows;
    a.N = W->rows, a.nks = W->in / 128, a.nka = op_k_atoms(W->in), a.tiles_n = (W->rows + GM_M - 1) / GM_M;
    a.counts = (int32_t *)g->workspace;
    a.parts = (float *)(a.counts + GM_CTAS);
    a.C = d.C, a.ldc = (long)d.ldc, a.accumulate = d.accumulate ? 1 : 0, a.err = err;
    a.pairs = d.c_dtype == K3MOE_BF16 && a.N % 2 == 0 && d.ldc % 2 == 0 && ((uintptr_t)d.C & 3u) == 0;
    return d.c_dtype == K3MOE_BF16 ? launch_gm_ct<__nv_bfloat16>(A, W, a, s) : launch_gm_ct<float>(A, W, a, s);
}

}  // namespace k3
