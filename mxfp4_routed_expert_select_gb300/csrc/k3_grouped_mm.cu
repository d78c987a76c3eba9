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
// Roles: warp 0 copies the weights (TMA, 128 of K per stage; the copy spreads 16
// four-bit codes over 16 bytes, the form this kind of MMA reads, so HBM and L2 move
// packed bytes) and their scale atoms, warp 2 gathers the rows' codes (TMA gather of
// four rows by index), warp 3 their scale bytes, warp 1 issues scale copies and MMAs,
// warps 4 and up read the accumulators while the next tile's products run.
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
constexpr int GM_THREADS = 256;
constexpr int GM_W_W = 0, GM_W_MMA = 1, GM_W_X = 2, GM_W_SF = 3, GM_W_EPI = 4;
constexpr int GM_MAX_E = 1024;
constexpr int GM_AHEAD = 8;  // steps of row scales in flight

struct GmArgs {
    const uint8_t *atoms;      // scale atoms of the weights, atoms_stride bytes from expert to expert
    long atoms_stride;
    const uint8_t *scales;     // scale bytes of the rows
    int sstride;
    const int32_t *offsets, *order;
    int E, top_k, slots, gather, xrows;  // xrows: rows of the 8-bit matrix
    int N, nks, nka, tiles_n;  // nks: steps of 128 along K; nka: atoms per row tile
    void *C;
    long ldc;
    int accumulate;
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
// Four rows of 128 bytes by index; a row outside the matrix reads as zero.
K3_DEV void gather4(uint32_t dst, const CUtensorMap *map, int x, const int (&r)[4], uint32_t bar)
{
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], "
                 "[%1, {%2, %3, %4, %5, %6}], [%7];\n\t}" ::"r"(dst),
                 "l"((uint64_t)map), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
                 : "memory");
}
K3_DEV void expect_elected(uint32_t bar, uint32_t bytes)
{
    asm volatile("{\n\t.reg .pred e;\n\t.reg .b64 st;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
                 "r"(bytes)
                 : "memory");
}

// The tiles of the batch: tab[e] row tiles lie before expert e's.
struct GmTile {
    int e, row, rows, n0;  // first row of C, rows of the group from there on (> 0), first weight row
};
template <int NT>
K3_DEV void gm_table(int *tab, int *sums, const GmArgs &a)
{
    // four experts a thread
    int v[4], mine = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int e = 4 * (int)threadIdx.x + i;
        const int lo = e < a.E ? min(max(a.offsets[e], 0), a.slots) : 0, hi = e < a.E ? min(a.offsets[e + 1], a.slots) : 0;
        v[i] = hi > lo ? (hi - lo + NT - 1) / NT : 0;
        mine += v[i];
    }
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[w] = x;
    __syncthreads();
    int at = x - mine;
    for (int i = 0; i < w; i++) at += sums[i];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int e = 4 * (int)threadIdx.x + i;
        if (e <= a.E) tab[e] = at;
        at += v[i];
    }
    if (threadIdx.x == GM_THREADS - 1 && a.E == GM_MAX_E) tab[a.E] = at;
    __syncthreads();
}
template <int NT>
K3_DEV GmTile gm_tile(const int *tab, const GmArgs &a, int u)
{
    const int r = u / a.tiles_n;
    int lo = 0, hi = a.E;  // tab[lo] <= r < tab[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (tab[m] <= r)
            lo = m;
        else
            hi = m;
    }
    GmTile t;
    t.e = lo;
    t.row = max(a.offsets[lo], 0) + (r - tab[lo]) * NT;
    t.rows = min(a.offsets[lo + 1], a.slots) - t.row;
    t.n0 = (u - r * a.tiles_n) * GM_M;
    return t;
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
    static constexpr int NS = (227 * 1024 - 8192) / STAGE < 10 ? (227 * 1024 - 8192) / STAGE : 10;
    static constexpr int TX_W = W_BYTES / 2 + 512, TX_X = X_BYTES;  // bytes as they lie in memory: the weights packed
    static constexpr int SF0 = 2 * NT, SF = 8;
    static constexpr int COLS_USED = SF0 + SF * NS;
    static constexpr int TMEM_COLS = COLS_USED <= 128 ? 128 : COLS_USED <= 256 ? 256 : 512;
    static constexpr int BARS = 2 * NS + 2 * 2 + 1;
    static constexpr int OFF_TAB = NS * STAGE + 256;
    static constexpr int SMEM = 1024 + OFF_TAB + (GM_MAX_E + 1 + 8) * 4;
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(COLS_USED <= 512, "TMEM layout");
    static_assert(BARS * 8 + 8 <= 256, "barriers");
};

template <typename CT>
K3_DEV void gm_put(CT *p, float v, int accumulate)
{
    if constexpr (sizeof(CT) == 2)
        *p = __float2bfloat16_rn(v);
    else
        *p = accumulate ? *p + v : v;
}

template <int NT, typename CT>
__global__ void __launch_bounds__(GM_THREADS, 1)
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
    int *tab = (int *)(sm + C::OFF_TAB), *sums = tab + GM_MAX_E + 1;
    auto bar = [&](int i) { return smem_addr(bars + i); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&wmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&xmap) : "memory");
        for (int i = 0; i < NS; i++) {
            mbar_init(bar(B_FULL + i), 3);  // weights, rows, the rows' scales
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
    gm_table<NT>(tab, sums, a);
    const int n_tiles = tab[a.E] * a.tiles_n, first = (int)blockIdx.x, step = (int)gridDim.x;

    if (warp == GM_W_W || warp == GM_W_X) {
        // ----------------------------------- producers of the code tiles
        uint32_t it = 0, phase = 1;  // before its first completion an EMPTY barrier's odd phase counts as passed
        int s = 0;
        bool ok = true;
        for (int u = first; u < n_tiles && ok; u += step) {
            const GmTile t = gm_tile<NT>(tab, a, u);
            const uint8_t *atoms = a.atoms + (long)t.e * a.atoms_stride + (long)(t.n0 / 128) * a.nka * 512;
            // the gathering warp's lane has four rows of the tile; columns past the group
            // repeat its last row (they are not stored)
            int src[4];
#pragma unroll
            for (int i = 0; i < 4; i++) src[i] = warp == GM_W_W ? 0 : gm_source(a, t.row + min(4 * lane + i, t.rows - 1));
            for (int ks = 0; ks < a.nks; ks++, it++) {
                if (!__all_sync(0xffffffffu, tc_wait(bar(B_EMPTY + s), phase, a.err, abort_flag))) {
                    ok = false;
                    break;
                }
                const uint32_t st = sbase + (uint32_t)(s * C::STAGE), full = bar(B_FULL + s);
                if (warp == GM_W_W) {
                    expect_elected(full, C::TX_W);
                    gm_load_w(st, &wmap, ks * 128, t.n0, t.e, st + C::OFF_WA, atoms + (long)ks * 512, full);
                } else {
                    expect_elected(full, C::TX_X);
#pragma unroll
                    for (int q = 0; q < NT / 4; q++) {
                        int r[4];
#pragma unroll
                        for (int i = 0; i < 4; i++) r[i] = __shfl_sync(0xffffffffu, src[i], q);
                        gather4(st + C::OFF_X + (uint32_t)q * 512, &xmap, ks * 128, r, full);
                    }
                }
                if (++s == NS) s = 0, phase ^= 1u;
            }
        }
        // drain: every copy issued here has landed before the CTA exits (the last
        // NS of them; earlier ones were waited for before their reuse)
        for (uint32_t i = it > (uint32_t)NS ? it - NS : 0; i < it; i++)
            mbar_wait(bar(B_FULL + (int)(i % NS)), (i / NS) & 1, a.err);
        __syncwarp();
    } else if (warp == GM_W_SF) {
        // ------------------------------------- producer of the rows' scales
        // A lane has the words of every 32nd row from its own on: a 16-byte store puts
        // them where tensor memory takes them from.  GM_AHEAD steps' words are loaded
        // before they are needed.
        constexpr int J = (NT + 31) / 32;
        uint32_t phase = 1;
        int s = 0;
        bool ok = true;
        for (int u = first; u < n_tiles && ok; u += step) {
            const GmTile t = gm_tile<NT>(tab, a, u);
            const uint8_t *sp[J];
#pragma unroll
            for (int j = 0; j < J; j++)
                sp[j] = a.scales + (long)gm_source(a, t.row + min(lane + 32 * j, t.rows - 1)) * a.sstride;
            uint32_t w[GM_AHEAD][J], wn[GM_AHEAD][J];
            auto load = [&](uint32_t (&d)[GM_AHEAD][J], int k0) {
#pragma unroll
                for (int i = 0; i < GM_AHEAD; i++)
#pragma unroll
                    for (int j = 0; j < J; j++) d[i][j] = k0 + i < a.nks ? *(const uint32_t *)(sp[j] + 4 * (k0 + i)) : 0u;
            };
            load(w, 0);
            for (int k0 = 0; k0 < a.nks && ok; k0 += GM_AHEAD) {
                load(wn, k0 + GM_AHEAD);
#pragma unroll
                for (int i = 0; i < GM_AHEAD; i++) {
                    if (k0 + i >= a.nks || !ok) break;
                    if (!__all_sync(0xffffffffu, tc_wait(bar(B_EMPTY + s), phase, a.err, abort_flag))) {
                        ok = false;
                        break;
                    }
                    *(uint4 *)(sm + s * C::STAGE + C::OFF_XA + lane * 16) =
                        make_uint4(w[i][0], w[i][J > 1 ? 1 : 0], w[i][J > 2 ? 2 : 0], w[i][J > 3 ? 3 : 0]);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_FULL + s));
                    if (++s == NS) s = 0, phase ^= 1u;
                }
#pragma unroll
                for (int i = 0; i < GM_AHEAD; i++)
#pragma unroll
                    for (int j = 0; j < J; j++) w[i][j] = wn[i][j];
            }
        }
        __syncwarp();
    } else if (warp == GM_W_MMA) {
        // -------------------------------------------------------------- MMA
        uint32_t ut = 0, phase = 0;
        int s = 0;
        bool ok = true;
        const uint32_t lo = sw128_lo(sbase);
        constexpr uint32_t SD = C::STAGE / 16;  // descriptor words between stages
        for (int u = first; u < n_tiles && ok; u += step, ut++) {
            const int buf = (int)(ut & 1);
            if (ut >= 2 && !__all_sync(0xffffffffu, tc_wait(bar(B_ACCE + buf), (ut / 2 - 1) & 1, a.err, abort_flag)))
                break;
            tc_fence_after();
            for (int ks = 0; ks < a.nks; ks++) {
                if (!__all_sync(0xffffffffu, tc_wait(bar(B_FULL + s), phase, a.err, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = lo + (uint32_t)s * SD;
                gm_step<NT>(tmem + (uint32_t)(buf * NT), d, d + C::OFF_X / 16, d + C::OFF_WA / 16,
                            tmem + (uint32_t)(C::SF0 + C::SF * s), ks ? 1u : 0u);
                mma_commit(bar(B_EMPTY + s));
                if (++s == NS) s = 0, phase ^= 1u;
            }
            if (!ok) break;
            mma_commit(bar(B_ACCF + buf));
        }
        // every MMA and copy issued above has completed before TMEM is freed
        mma_commit(bar(B_FIN));
        mbar_wait(bar(B_FIN), 0, a.err);
        __syncwarp();
    } else {
        // --------------------------------------------------------- epilogue
        const int q = warp - GM_W_EPI;  // TMEM lane quadrant: weight rows 32 q .. 32 q + 31 of the tile
        constexpr int CH = NT < 32 ? 16 : 32, NCH = NT / CH;
        uint32_t ut = 0;
        for (int u = first; u < n_tiles; u += step, ut++) {
            const int buf = (int)(ut & 1);
            const GmTile t = gm_tile<NT>(tab, a, u);
            if (!__all_sync(0xffffffffu, tc_wait(bar(B_ACCF + buf), (ut / 2) & 1, a.err, abort_flag))) break;
            tc_fence_after();
            const uint32_t tacc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * NT);
            const int n = t.n0 + q * 32 + lane;
#pragma unroll 1
            for (int j = 0; j < NCH; j++) {
                uint32_t r[CH];
                tmem_ld_chunk(tacc + (uint32_t)(j * CH), r);
                if (j == NCH - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_ACCE + buf));
                }
                if (n >= a.N) continue;
                CT *o = (CT *)a.C + (long)(t.row + j * CH) * a.ldc + n;
#pragma unroll
                for (int c = 0; c < CH; c++)
                    if (j * CH + c < t.rows) gm_put(o + (long)c * a.ldc, __uint_as_float(r[c]), a.accumulate);
            }
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

// ---------------------------------------------------------------- launchers

template <int NT, typename CT>
int launch_gm(const k3moe_mx8_rows *A, const k3moe_mx_experts *W, const GmArgs &a, cudaStream_t s)
{
    using C = GmCfg<NT>;
    CUtensorMap wmap, xmap;
    const cuuint64_t wd[3] = {(cuuint64_t)W->in, (cuuint64_t)W->rows, (cuuint64_t)W->E},
                     ws[2] = {(cuuint64_t)W->in / 2, (cuuint64_t)W->codes_stride};
    const cuuint32_t wb[3] = {128, GM_M, 1};
    int st = encode_map(&wmap, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 3, W->codes, wd, ws, wb, CU_TENSOR_MAP_SWIZZLE_128B);
    const cuuint64_t xd[2] = {(cuuint64_t)A->in, (cuuint64_t)A->rows}, xs[1] = {(cuuint64_t)op_in_padded(A->in)};
    const cuuint32_t xb[2] = {128, 1};
    if (st == K3MOE_OK)
        st = encode_map(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, A->codes, xd, xs, xb, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != K3MOE_OK) return st;
    if (ensure_smem((const void *)k3_grouped_matmul<NT, CT>, C::SMEM) != K3MOE_OK) return K3MOE_ECUDA;
    const long most = std::min<long>(a.slots, (long)a.E + a.slots / NT) * a.tiles_n;  // tiles there can be
    if (launch_pdl(k3_grouped_matmul<NT, CT>, dim3((unsigned)std::min<long>(most, num_sms())), dim3(GM_THREADS), C::SMEM, s,
                   wmap, xmap, a) != cudaSuccess) {
        cudaGetLastError();
        return K3MOE_ECUDA;
    }
    return K3MOE_OK;
}
template <typename CT>
int launch_gm_ct(const k3moe_mx8_rows *A, const k3moe_mx_experts *W, const GmArgs &a, cudaStream_t s)
{
    const int avg = (a.slots + a.E - 1) / a.E;
    return avg <= 12   ? launch_gm<16, CT>(A, W, a, s)
           : avg <= 24 ? launch_gm<32, CT>(A, W, a, s)
           : avg <= 48 ? launch_gm<64, CT>(A, W, a, s)
                       : launch_gm<128, CT>(A, W, a, s);
}

}  // namespace

int launch_grouped_matmul(void *C, int cdt, long ldc, const k3moe_mx8_rows *A, const k3moe_mx_experts *W,
                          const k3moe_groups *g, int gather, int accumulate, int *err, cudaStream_t s)
{
    GmArgs a = {};
    a.atoms = W->atoms, a.atoms_stride = W->atoms_stride;
    a.scales = A->scales, a.sstride = mx8_scale_stride(A->in);
    a.offsets = g->offsets, a.order = g->order;
    a.E = g->E, a.top_k = g->top_k, a.slots = g->tokens * g->top_k, a.gather = gather, a.xrows = A->rows;
    a.N = W->rows, a.nks = W->in / 128, a.nka = op_k_atoms(W->in), a.tiles_n = (W->rows + GM_M - 1) / GM_M;
    a.C = C, a.ldc = ldc, a.accumulate = accumulate, a.err = err;
    if (((long)a.E + a.slots) * a.tiles_n > 0x7fffffffL) return K3MOE_EINVAL;
    return cdt == K3MOE_BF16 ? launch_gm_ct<__nv_bfloat16>(A, W, a, s) : launch_gm_ct<float>(A, W, a, s);
}

}  // namespace k3
