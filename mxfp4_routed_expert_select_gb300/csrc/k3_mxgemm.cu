// k3_mxgemm.cu -- the product of two MXFP4 operands, C = A B^T, on the
// block-scaled tensor cores (tcgen05.mma kind::mxf4).
//
// C[m][n] = sum over blocks b of 2^(ea[m][b] + eb[n][b] - 254) times the sum of
// the 32 code products of block b: the tensor core multiplies the E2M1 codes as
// stored and applies both E8M0 scales itself, accumulating in fp32 in TMEM.
//
// Three forms:
//  - pairs (large products): two CTAs on one 256 x NT tile of C; see below.
//  - tiles: one CTA per SM walks 128 x NT tiles; the accumulator of one tile is
//    read out while the next one's products run.
//  - split: with fewer tiles than SMs, a cluster of S CTAs shares one tile, each
//    taking 1/S of K; their partial sums meet in distributed shared memory, where
//    each CTA adds one slice of the columns over the S ranks in rank order (the
//    result does not depend on timing).
//
// On single CTAs (the last two) B's rows (the weights' output features) take the
// MMA's 128 lanes and A's rows (the tokens) its NT columns: a few tokens then cost
// a narrow MMA over the streamed weights, and in the epilogue a warp holds 32
// consecutive n of one m, so that its stores of C are coalesced.
//
// Roles: warps 0 and 2 copy one operand each (TMA, 256 of K per stage: rows x 128
// bytes with the 128-byte swizzle, and their scale atoms, which are stored in the
// order tensor memory takes them in), warp 1 issues the scale copies and MMAs,
// warps 4 and up read the accumulators.  Rows, columns and K past the matrices are
// zero-filled by the copies or not stored.
//
// Every wait is bounded (2 s); a timeout sets the device error word and the CTA
// drains its copies and MMAs, frees TMEM and exits.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "k3_launch.cuh"
#include "k3_operand.cuh"
#include "k3_tcgen05.cuh"

namespace k3 {
namespace {

constexpr int MG_M = 128;       // lanes of one CTA's tile
constexpr int MG_THREADS = 256;
constexpr int MG_MAX_RANKS = 8;  // CTAs that share a tile
constexpr int MG_W_PROD = 0, MG_W_MMA = 1, MG_W_PROD2 = 2, MG_W_EPI = 4;

struct MgArgs {
    const uint8_t *satoms, *tatoms;  // single CTAs: scale atoms of B (lanes) and A (columns)
    void *C;
    long ldc;
    int M, N, nks, nka;              // A rows, B rows, 256-long k-steps, atoms per row tile
    int tiles_t, n_tiles;            // tiles along the MMA columns, all tiles
    int accumulate;
    int vec;                         // split: four consecutive elements of a row of C form an aligned store
    int tma;                         // pairs: rows of C are aligned for TMA stores
    int *err;
};

// ------------------------------------------------------- instruction helpers

// Instruction descriptor: E2M1 x E2M1, K-major, UE8M0 scales, M lanes, N columns;
// sfid: the first of this MMA's two scale bytes within the 32-bit scale words.
__host__ __device__ constexpr uint32_t mg_idesc(int m, int n, uint32_t sfid)
{
    return (sfid << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
           ((uint32_t)(m >> 4) << 24) | (sfid << 29);
}

// One k-step: the scale atoms of the stage to TMEM, then four MMAs of K = 64.
// One block with one election and every address an addition to a stage's: issued
// as separate statements a step took the issuing warp 370 clocks and bounded the
// products.
//   slo, tlo   descriptor words of the code tiles (lanes, columns); +2 per 64 of K
//   sal        descriptor word of the lanes' atoms, the columns' follow; +32 each
//   sf         TMEM column of the stage's scales: the lanes' in 8 columns, the
//              columns' in 8 per 128 rows, k-atom major
//   shift      first scale word of the columns' rows within their atoms
// GRP: cta_group.  1: one row tile of column atoms; 2: two, and each CTA of the pair
// copies its own atoms to its own TMEM.  384 columns are two MMAs of 192, their code
// rows 96 apart in the stage and their scales in three row tiles.
#define MG_HEAD                                                                                              \
    "{\n\t.reg .pred p, t, e;\n\t.reg .b64 d, da, db;\n\t.reg .b32 x, y, z, w;\n\tadd.u32 w, %0, 192;\n\t"       \
    "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, %7, %7;\n\tadd.u32 z, %4, %5;\n\t"
#define MG_CP(grp, col, off)                                                                                 \
    "add.u32 x, %3, " #off ";\n\tadd.u32 y, %4, " #col ";\n\tmov.b64 d, {x, %8};\n\t"                          \
    "@e tcgen05.cp.cta_group::" #grp ".32x128b.warpx4 [y], d;\n\t"
#define MG_MMA(grp, acc, k2, t2, sfa, sfb, id, pred)                                                                \
    "add.u32 x, %1, " #k2 ";\n\tadd.u32 y, %2, " #t2 ";\n\tmov.b64 da, {x, %9};\n\tmov.b64 db, {y, %9};\n\t"   \
    "add.u32 x, %4, " #sfa ";\n\tadd.u32 y, z, " #sfb ";\n\t"                                                \
    "@e tcgen05.mma.cta_group::" #grp ".kind::mxf4.block_scale.scale_vec::2X [" acc "], da, db, " id ", [x], [y], " pred ";\n\t"
#define MG_OPERANDS                                                                                          \
    ::"r"(tacc), "r"(slo), "r"(tlo), "r"(sal), "r"(sf), "r"(shift), "r"(acc), "r"(mg_idesc(M, MN, 0)), "r"(AHI),     \
        "r"(SW128_HI), "r"(mg_idesc(M, MN, 2))                                                               \
        : "memory"
template <int GRP, int NT>
K3_DEV void mg_step(uint32_t tacc, uint32_t slo, uint32_t tlo, uint32_t sal, uint32_t sf, uint32_t shift, uint32_t acc)
{
    constexpr uint32_t AHI = (128u >> 4) | (1u << 14);  // atoms: 8 rows of 16 bytes 128 bytes apart, no swizzle
    constexpr int M = GRP * MG_M, MN = NT > 256 ? NT / 2 : NT;
    if constexpr (NT == 384)
        asm volatile(MG_HEAD MG_CP(2, 0, 0) MG_CP(2, 4, 32) MG_CP(2, 8, 64) MG_CP(2, 12, 128) MG_CP(2, 16, 192)
                         MG_CP(2, 20, 96) MG_CP(2, 24, 160) MG_CP(2, 28, 224)
                             MG_MMA(2, "%0", 0, 0, 0, 8, "%7", "p") MG_MMA(2, "w", 0, 768, 0, 14, "%7", "p")
                                 MG_MMA(2, "%0", 2, 2, 0, 8, "%10", "t") MG_MMA(2, "w", 2, 770, 0, 14, "%10", "t")
                                     MG_MMA(2, "%0", 4, 4, 4, 20, "%7", "t") MG_MMA(2, "w", 4, 772, 4, 26, "%7", "t")
                                         MG_MMA(2, "%0", 6, 6, 4, 20, "%10", "t")
                                             MG_MMA(2, "w", 6, 774, 4, 26, "%10", "t") "}" MG_OPERANDS);
    else if constexpr (GRP == 2)
        asm volatile(MG_HEAD MG_CP(2, 0, 0) MG_CP(2, 4, 32) MG_CP(2, 8, 64) MG_CP(2, 12, 128) MG_CP(2, 16, 96)
                         MG_CP(2, 20, 160) MG_MMA(2, "%0", 0, 0, 0, 8, "%7", "p") MG_MMA(2, "%0", 2, 2, 0, 8, "%10", "t")
                             MG_MMA(2, "%0", 4, 4, 4, 16, "%7", "t") MG_MMA(2, "%0", 6, 6, 4, 16, "%10", "t") "}" MG_OPERANDS);
    else
        asm volatile(MG_HEAD MG_CP(1, 0, 0) MG_CP(1, 4, 32) MG_CP(1, 8, 64) MG_CP(1, 12, 96)
                         MG_MMA(1, "%0", 0, 0, 0, 8, "%7", "p") MG_MMA(1, "%0", 2, 2, 0, 8, "%10", "t")
                             MG_MMA(1, "%0", 4, 4, 4, 12, "%7", "t") MG_MMA(1, "%0", 6, 6, 4, 12, "%10", "t") "}" MG_OPERANDS);
}
#undef MG_HEAD
#undef MG_CP
#undef MG_MMA
#undef MG_OPERANDS

// 16 or 32 columns of the accumulator, one row per lane.  The wait names the
// registers, so that nothing made from them can move above it.
K3_DEV void tmem_ld_chunk(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
K3_DEV void tmem_ld_chunk(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

K3_DEV uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
K3_DEV uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
K3_DEV void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
K3_DEV uint32_t addr_of_rank(uint32_t addr, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
K3_DEV float4 ld_peer4(uint32_t addr, uint32_t rank)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr_of_rank(addr, rank))
                 : "memory");
    return v;
}
// expect_tx arrival by the elected lane of a converged warp.
K3_DEV void mbar_expect_elected(uint32_t bar, uint32_t bytes)
{
    asm volatile("{\n\t.reg .pred e;\n\t.reg .b64 st;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
                 "r"(bytes)
                 : "memory");
}
K3_DEV void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)map) : "memory");
}
// One operand's copies of a stage: its rows' codes and its two scale atoms.  One
// block issued by a converged warp's elected lane, one warp per operand: a step's
// copies by one lane of a diverged warp took 700 clocks and bounded the products,
// by one converged warp 390.
K3_DEV void mg_load(uint32_t dst, const CUtensorMap *map, uint32_t adst, const uint8_t *atoms, int x, int row,
                    uint32_t bar)
{
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
                 "[%1, {%4, %5}], [%6];\n\t"
                 "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%2], [%3], 1024, [%6];\n\t}" ::"r"(
                     dst),
                 "l"((uint64_t)map), "r"(adst), "l"(atoms), "r"(x), "r"(row), "r"(bar)
                 : "memory");
}

// ------------------------------------------------------------ results to C

template <typename CT>
K3_DEV void put(CT *C, long i, float v, int accumulate)
{
    if constexpr (sizeof(CT) == 2)
        C[i] = __float2bfloat16_rn(v);
    else
        C[i] = accumulate ? C[i] + v : v;
}
// Four consecutive columns n .. n + 3 of a row of C (N columns), as one store
// where the rows are aligned for it.
template <typename CT>
K3_DEV void put4(CT *row, int n, int N, const float (&v)[4], int accumulate, int vec)
{
    if (vec && !accumulate && n + 4 <= N) {
        if constexpr (sizeof(CT) == 2) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
            *(uint2 *)(row + n) = make_uint2(*(const uint32_t *)&lo, *(const uint32_t *)&hi);
        } else {
            *(float4 *)(row + n) = make_float4(v[0], v[1], v[2], v[3]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
        if (n + i < N) put(row, n + i, v[i], accumulate);
}
// A lane's column n of C, rows m .. m + CH - 1.
template <typename CT, int CH>
K3_DEV void put_column(const MgArgs &a, int n, int m, const uint32_t (&r)[CH])
{
    CT *o = (CT *)a.C + n;
    if (m + CH <= a.M) {
#pragma unroll
        for (int c = 0; c < CH; c++) put(o, (long)(m + c) * a.ldc, __uint_as_float(r[c]), a.accumulate);
    } else {
#pragma unroll
        for (int c = 0; c < CH; c++)
            if (m + c < a.M) put(o, (long)(m + c) * a.ldc, __uint_as_float(r[c]), a.accumulate);
    }
}

// -------------------------------------------------------------- single CTAs

// This rank's slice of a split tile's columns: the sums of R ranks, in rank order,
// to C.  A warp takes a column, a lane four consecutive rows of it; eight remote
// loads (a few hundred clocks each) are in flight per lane.
template <int NT, int R, typename CT>
K3_DEV void join_ranks(const MgArgs &a, uint32_t sbase, int tile, int rank)
{
    constexpr int J = 8 / R, NW = MG_THREADS / 32;  // columns in flight, warps
    const int lane = threadIdx.x & 31;
    const int n = (tile / a.tiles_t) * MG_M + 4 * lane, m0 = (tile % a.tiles_t) * NT;
    const int c0 = NT * rank / R, c1 = min(NT * (rank + 1) / R, a.M - m0);
    for (int c = c0 + (int)(threadIdx.x >> 5); c < c1; c += J * NW) {
        float4 v[J][R];
#pragma unroll
        for (int j = 0; j < J; j++)
#pragma unroll
            for (int r = 0; r < R; r++)
                if (c + j * NW < c1) v[j][r] = ld_peer4(sbase + (uint32_t)((c + j * NW) * MG_M + 4 * lane) * 4, (uint32_t)r);
#pragma unroll
        for (int j = 0; j < J; j++)
            if (c + j * NW < c1) {
                float t[4] = {v[j][0].x, v[j][0].y, v[j][0].z, v[j][0].w};
#pragma unroll
                for (int r = 1; r < R; r++) t[0] += v[j][r].x, t[1] += v[j][r].y, t[2] += v[j][r].z, t[3] += v[j][r].w;
                put4((CT *)a.C + (long)(m0 + c + j * NW) * a.ldc, n, a.N, t, a.accumulate, a.vec);
            }
    }
}

// Shared memory and TMEM of one CTA with NT columns, one tile per cluster
// (SPLIT) or many per CTA.
template <int NT, bool SPLIT>
struct MgCfg {
    static constexpr int S_BYTES = MG_M * 128, T_BYTES = NT * 128;
    static constexpr int OFF_T = S_BYTES;
    static constexpr int OFF_SA = OFF_T + T_BYTES;           // B's two atoms
    static constexpr int OFF_TA = OFF_SA + 1024;             // A's two atoms
    static constexpr int TX = OFF_TA + 1024;                 // bytes copied per stage
    static constexpr int STAGE = (TX + 1023) / 1024 * 1024;
    // Split: few enough stages that two CTAs fit an SM, although choose_plan gives
    // each one of its own (two per SM lost).
    static constexpr int NS = !SPLIT ? 6 : NT <= 16 ? 5 : 4;
    // TMEM: the accumulators (two of NT columns, one when split), then each
    // stage's scales.
    static constexpr int SF = 16;
    static constexpr int SF0 = SPLIT ? NT : 2 * NT;
    static constexpr int COLS_USED = SF0 + SF * NS;
    static constexpr int TMEM_COLS = COLS_USED <= 128 ? 128 : COLS_USED <= 256 ? 256 : 512;
    static constexpr int BARS = 2 * NS + 2 * 2 + 1;
    static constexpr int SMEM = 1024 + NS * STAGE + 256;
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(COLS_USED <= 512, "TMEM layout");
    static_assert(!SPLIT || NT * MG_M * 4 <= NS * STAGE, "partial sums reuse the stages");
};

template <int NT, bool SPLIT, typename CT>
__global__ void __launch_bounds__(MG_THREADS, 1)
    k3_mx_matmul(const __grid_constant__ CUtensorMap smap, const __grid_constant__ CUtensorMap tmap, const MgArgs a)
{
    using C = MgCfg<NT, SPLIT>;
    constexpr int NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_addr(sm);
    uint64_t *bars = (uint64_t *)(sm + NS * C::STAGE);
    constexpr int B_FULL = 0, B_EMPTY = NS, B_ACCF = 2 * NS, B_ACCE = B_ACCF + 2, B_FIN = B_ACCE + 2;
    uint32_t *tmem_slot = (uint32_t *)(bars + C::BARS);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);
    auto bar = [&](int i) { return smem_addr(bars + i); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // this CTA's tiles and its range of k-steps
    const int rank = SPLIT ? (int)cluster_rank() : 0, ranks = SPLIT ? (int)cluster_size() : 1;
    const int first = SPLIT ? (int)blockIdx.x / ranks : (int)blockIdx.x;
    const int step = SPLIT ? a.n_tiles : (int)gridDim.x;
    const int k0 = (int)((long)a.nks * rank / ranks), k1 = (int)((long)a.nks * (rank + 1) / ranks);

    if (threadIdx.x == 0) {
        prefetch_map(&smap), prefetch_map(&tmap);
        for (int i = 0; i < NS; i++) {
            mbar_init(bar(B_FULL + i), 1);
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
    if (warp == MG_W_MMA) {
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

    if (warp == MG_W_PROD || warp == MG_W_PROD2) {
        // ---------------------------- producers: warp 0 B's rows, warp 2 A's
        const bool is_s = warp == MG_W_PROD;
        const CUtensorMap *map = is_s ? &smap : &tmap;
        const uint32_t dst0 = sbase + (is_s ? 0 : C::OFF_T), adst0 = sbase + (is_s ? C::OFF_SA : C::OFF_TA);
        uint32_t it = 0, phase = 1;  // before its first completion an EMPTY barrier's odd phase counts as passed
        int s = 0;
        bool ok = true, ready = true;
        for (int u = first; u < a.n_tiles && ok; u += step) {
            const int row = is_s ? (u / a.tiles_t) * MG_M : (u % a.tiles_t) * NT;
            const uint8_t *atoms = (is_s ? a.satoms : a.tatoms) + (long)(row / 128) * a.nka * 512;
            for (int ks = k0; ks < k1; ks++, it++) {
                if (!ready && !__all_sync(0xffffffffu, tc_wait(bar(B_EMPTY + s), phase, a.err, abort_flag))) {
                    ok = false;
                    break;
                }
                const int sn = s + 1 == NS ? 0 : s + 1;
                const uint32_t pn = sn ? phase : phase ^ 1u;
                ready = __all_sync(0xffffffffu, mbar_test(bar(B_EMPTY + sn), pn));
                if (is_s) mbar_expect_elected(bar(B_FULL + s), C::TX);
                mg_load(dst0 + (uint32_t)(s * C::STAGE), map, adst0 + (uint32_t)(s * C::STAGE), atoms + (long)ks * 1024,
                        ks * 128, row, bar(B_FULL + s));
                s = sn;
                phase = pn;
            }
        }
        // drain: every copy issued here has landed before the CTA exits (the last
        // NS of them; earlier ones were waited for before their reuse)
        for (uint32_t i = it > (uint32_t)NS ? it - NS : 0; i < it; i++)
            mbar_wait(bar(B_FULL + (int)(i % NS)), (i / NS) & 1, a.err);
        __syncwarp();
    } else if (warp == MG_W_MMA) {
        // -------------------------------------------------------------- MMA
        uint32_t ut = 0, phase = 0;
        int s = 0;
        bool ok = true, ready = false;
        const uint32_t slo = sw128_lo(sbase);
        constexpr uint32_t SD = C::STAGE / 16;  // descriptor words between stages
        for (int u = first; u < a.n_tiles && ok; u += step, ut++) {
            const int buf = (int)(ut & 1);
            // a 64-column tile starts at a half of a scale atom's rows every other time
            const uint32_t shift = NT < 64 ? 0u : (uint32_t)(((u % a.tiles_t) * NT % 128) / 32);
            if (ut >= 2 && !__all_sync(0xffffffffu, tc_wait(bar(B_ACCE + buf), (ut / 2 - 1) & 1, a.err, abort_flag)))
                break;
            tc_fence_after();
            for (int ks = k0; ks < k1; ks++) {
                if (!ready && !__all_sync(0xffffffffu, tc_wait(bar(B_FULL + s), phase, a.err, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int sn = s + 1 == NS ? 0 : s + 1;
                const uint32_t pn = sn ? phase : phase ^ 1u;
                // look at the next stage while this one is issued
                ready = __all_sync(0xffffffffu, mbar_test(bar(B_FULL + sn), pn));
                mg_step<1, NT>(tmem + (uint32_t)(buf * NT), slo + (uint32_t)s * SD, slo + C::OFF_T / 16 + (uint32_t)s * SD,
                                  slo + C::OFF_SA / 16 + (uint32_t)s * SD, tmem + (uint32_t)(C::SF0 + C::SF * s), shift,
                                  ks > k0 ? 1u : 0u);
                mma_commit(bar(B_EMPTY + s));
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
    } else if (warp >= MG_W_EPI) {
        // --------------------------------------------------------- epilogue
        const int q = warp - MG_W_EPI;  // TMEM lane quadrant: rows 32 q .. 32 q + 31 of the tile
        constexpr int CH = NT < 32 ? 16 : 32, NCH = NT / CH;
        uint32_t ut = 0;
        for (int u = first; u < a.n_tiles; u += step, ut++) {
            const int buf = (int)(ut & 1);
            if (!__all_sync(0xffffffffu, tc_wait(bar(B_ACCF + buf), (ut / 2) & 1, a.err, abort_flag))) break;
            tc_fence_after();
            const uint32_t tacc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * NT);
            const int n = (u / a.tiles_t) * MG_M + q * 32 + lane, m0 = (u % a.tiles_t) * NT;
#pragma unroll 1
            for (int j = 0; j < NCH; j++) {
                uint32_t r[CH];
                tmem_ld_chunk(tacc + (uint32_t)(j * CH), r);
                if (!SPLIT && j == NCH - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_ACCE + buf));
                }
                if constexpr (SPLIT) {
                    float *part = (float *)sm;  // [column][128]: every stage has been consumed
#pragma unroll
                    for (int c = 0; c < CH; c++) part[(j * CH + c) * MG_M + q * 32 + lane] = __uint_as_float(r[c]);
                } else if (n < a.N) {
                    put_column<CT, CH>(a, n, m0 + j * CH, r);
                }
            }
        }
    }

    tc_fence_before();
    if constexpr (SPLIT) {
        __syncwarp();
        cluster_sync();  // every rank's partial sums are in its shared memory
        if (!*abort_flag) {
            if (ranks == 2)
                join_ranks<NT, 2, CT>(a, sbase, first, rank);
            else if (ranks == 4)
                join_ranks<NT, 4, CT>(a, sbase, first, rank);
            else
                join_ranks<NT, 8, CT>(a, sbase, first, rank);
        }
        cluster_sync();  // no CTA leaves while another reads its sums
    } else {
        __syncthreads();
    }
    if (warp == MG_W_MMA) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS)
                     : "memory");
    }
}

// ---------------------------------------------------------------- CTA pairs
//
// The large products.  A lone CTA's 128 x 256 tile brings 51 KB per 256 of K into
// its shared memory and reads 48 KB of it, 790 clocks of its bandwidth for 512
// clocks of MMAs (measured 880 a step, 5.3 PFLOP/s at 8192^3).  A pair of CTAs
// (cta_group::2) works on 256 rows of A x NT rows of B together: each loads its own
// 128 rows of A and half of B's, and the MMA reads both halves, so a step brings
// and reads 35 KB per SM: shared memory's 64 bytes a clock (553 clocks a step) and
// the tensor cores (512) are both near full (7.4 PFLOP/s at 8192^3).  192 columns
// leave the MMAs 384 of 490 clocks but split some products into fuller waves; 384,
// for products that are then one wave, are bound by the MMAs (790 of 768 clocks),
// but with one accumulator the epilogue of a tile is not hidden.
//
// A's rows take the lanes here, so that a lane of the epilogue holds consecutive n
// and stages them with 16-byte stores (with B's rows in the lanes its 2-byte ones
// competed with the MMAs for shared memory: a 4096 x 7168 x 1536 product took 29 us
// instead of 23, stored from registers or staged).
//
// The even CTA of a pair issues every scale copy and MMA for both.  Each CTA's
// producers fill its own stages, all copies counted on the even CTA's barrier;
// commits arrive at both CTAs' barriers, and the epilogues of both free an
// accumulator at the even CTA's.

constexpr int MP_EPI = 8;  // epilogue warps per CTA: two per TMEM lane quadrant, on alternate pieces
constexpr int MP_THREADS = (MG_W_EPI + MP_EPI) * 32;
constexpr int MP_BOX = 4096;  // bytes of a staged piece of C: 32 rows of 128 bytes

template <int NT>
struct MpCfg {
    static constexpr int MN = NT > 256 ? NT / 2 : NT;  // columns of an MMA
    static constexpr int QT = NT > 256 ? 3 : 2;       // row tiles of B's scale atoms per tile (192: from a half tile)
    static constexpr int S_BYTES = MG_M * 128, T_BYTES = NT / 2 * 128;
    static constexpr int OFF_T = S_BYTES;
    static constexpr int OFF_SA = OFF_T + T_BYTES;    // this CTA's two A atoms
    static constexpr int OFF_TA = OFF_SA + 1024;      // all of B's atoms of the tile (each CTA needs them)
    static constexpr int STAGE = OFF_TA + QT * 1024;
    static constexpr int NS = NT > 256 ? 4 : 5;
    static constexpr int OFF_C = NS * STAGE;          // a staged piece per epilogue warp
    static constexpr int OFF_BAR = OFF_C + MP_EPI * MP_BOX;
    static constexpr int SMEM = 1024 + OFF_BAR + 256;
    // TMEM: two accumulators, then each stage's scales.  Two accumulators of 256
    // columns do not fit beside the scales: the second starts at OVER, and the
    // columns they share are read first.  Of 384 there is one.
    static constexpr int SF = 8 + 8 * QT;
    static constexpr int OVER = NT > 256 ? 0 : NT == 256 ? 128 : NT;
    static constexpr int SF0 = OVER + NT;
    static constexpr int BARS = 2 * NS + 2 * 2 + 1;
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(SF0 + SF * NS <= 512, "TMEM layout");
    static_assert(STAGE % 1024 == 0 && OFF_SA % 1024 == 0, "swizzled tiles are 1024-byte aligned");
};

// Arrival at the barrier of the same offset in the pair's CTA `rank`, for a
// hand-over of tensor memory alone: the accumulator's loads are ordered by their
// wait and the tcgen05 fence before this, and no ordinary memory is handed over, so
// the arrival is relaxed (a release at cluster scope took 1200 clocks, on the path
// of the next tile's first MMA).
K3_DEV void mbar_arrive_rank(uint32_t bar, uint32_t rank)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr_of_rank(bar, rank)) : "memory");
}
// The waits for barriers that the other CTA's threads, copies or commits arrive
// at: cluster scope, bounded as mbar_wait.
K3_DEV uint32_t mbar_try_wait_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity), "r"(20000u)
                 : "memory");
    return ok;
}
static __device__ __noinline__ bool mbar_wait_cluster_slow(uint32_t bar, uint32_t parity, int *err)
{
    const uint64_t t0 = global_ns();
    for (uint32_t n = 1;; n++) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if ((n & 63u) == 0 && global_ns() - t0 > kWaitLimitNs) {
            set_device_error(err, K3MOE_ETIMEOUT);
            return false;
        }
    }
}
K3_DEV bool tc_wait_cluster(uint32_t bar, uint32_t parity, int *err, volatile int *abort_flag)
{
    if (*abort_flag) return false;
    if (mbar_try_wait_cluster(bar, parity) || mbar_wait_cluster_slow(bar, parity, err)) return true;
    *abort_flag = 1;
    return false;
}
// Non-blocking: has the phase completed?
K3_DEV bool mbar_test_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}
// mg_load with all bytes counted on barrier `bar` (a shared::cluster address: the
// even CTA's), the atoms as boxes [row tile][2][512] at (ka, rt).
K3_DEV void mp_load(uint32_t dst, const CUtensorMap *map, uint32_t adst, const CUtensorMap *amap, int x, int row,
                    int ka, int rt, uint32_t bar)
{
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
                 "[%1, {%4, %5}], [%8];\n\t"
                 "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%2], "
                 "[%3, {0, %6, %7}], [%8];\n\t}" ::"r"(dst),
                 "l"((uint64_t)map), "r"(adst), "l"((uint64_t)amap), "r"(x), "r"(row), "r"(ka), "r"(rt), "r"(bar)
                 : "memory");
}
K3_DEV void mp_load_codes(uint32_t dst, const CUtensorMap *map, int x, int row, uint32_t bar)
{
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
                 "[%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
                 "l"((uint64_t)map), "r"(x), "r"(row), "r"(bar)
                 : "memory");
}
// Arrival at the barrier of this offset in both CTAs once everything issued
// before has completed.
K3_DEV void mp_commit(uint32_t bar)
{
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
                 "%1;\n\t}" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}
// A staged piece of C from shared memory: stored, or added in fp32.
K3_DEV void tma_store_2d(const CUtensorMap *map, uint32_t src, int x, int y, int accumulate)
{
    if (accumulate)
        asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                         (uint64_t)map),
                     "r"(x), "r"(y), "r"(src)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                         (uint64_t)map),
                     "r"(x), "r"(y), "r"(src)
                     : "memory");
}

template <int NT, typename CT>
__global__ void __launch_bounds__(MP_THREADS, 1)
    k3_mx_matmul_pair(const __grid_constant__ CUtensorMap smap, const __grid_constant__ CUtensorMap tmap,
                      const __grid_constant__ CUtensorMap samap, const __grid_constant__ CUtensorMap tamap,
                      const __grid_constant__ CUtensorMap cmap, const MgArgs a)
{
    using C = MpCfg<NT>;
    constexpr int NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_addr(sm);
    uint64_t *bars = (uint64_t *)(sm + C::OFF_BAR);
    constexpr int B_FULL = 0, B_EMPTY = NS, B_ACCF = 2 * NS, B_ACCE = B_ACCF + 2, B_FIN = B_ACCE + 2;
    uint32_t *tmem_slot = (uint32_t *)(bars + C::BARS);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);
    auto bar = [&](int i) { return smem_addr(bars + i); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();  // 0: the CTA that issues
    const int first = (int)blockIdx.x >> 1, step = (int)gridDim.x >> 1;

    if (threadIdx.x == 0) {
        prefetch_map(&smap), prefetch_map(&tmap), prefetch_map(&samap), prefetch_map(&tamap);
        for (int i = 0; i < NS; i++) {
            mbar_init(bar(B_FULL + i), 1);
            mbar_init(bar(B_EMPTY + i), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(bar(B_ACCF + i), 1);
            mbar_init(bar(B_ACCE + i), 2 * MP_EPI);  // the epilogue warps of both CTAs
        }
        mbar_init(bar(B_FIN), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == MG_W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the other CTA's barriers are initialised
    tc_fence_after();
    const uint32_t tmem = *(volatile uint32_t *)tmem_slot;
    griddep_wait();

    if (warp == MG_W_PROD || warp == MG_W_PROD2) {
        // ---------------------------- producers: warp 0 A's rows, warp 2 B's
        const bool is_s = warp == MG_W_PROD;
        const CUtensorMap *map = is_s ? &smap : &tmap, *amap = is_s ? &samap : &tamap;
        const uint32_t full0 = addr_of_rank(bar(B_FULL), 0);
        const uint32_t dst0 = sbase + (is_s ? 0 : C::OFF_T), adst0 = sbase + (is_s ? C::OFF_SA : C::OFF_TA);
        uint32_t it = 0, phase = 1;  // before its first completion an EMPTY barrier's odd phase counts as passed
        int s = 0;
        bool ok = true, ready = true;
        for (int u = first; u < a.n_tiles && ok; u += step) {
            // rows and atoms past the matrices read as zero
            const int m0 = (u / a.tiles_t) * 2 * MG_M + rank * MG_M, n0 = (u % a.tiles_t) * NT;
            const int row = is_s ? m0 : n0 + rank * (C::MN / 2), rt = (is_s ? m0 : n0) / 128;
            for (int ks = 0; ks < a.nks; ks++, it++) {
                if (!ready && !__all_sync(0xffffffffu, tc_wait_cluster(bar(B_EMPTY + s), phase, a.err, abort_flag))) {
                    ok = false;
                    break;
                }
                const int sn = s + 1 == NS ? 0 : s + 1;
                const uint32_t pn = sn ? phase : phase ^ 1u;
                ready = __all_sync(0xffffffffu, mbar_test_cluster(bar(B_EMPTY + sn), pn));
                if (is_s && rank == 0) mbar_expect_elected(bar(B_FULL + s), 2 * C::STAGE);
                mp_load(dst0 + (uint32_t)(s * C::STAGE), map, adst0 + (uint32_t)(s * C::STAGE), amap, ks * 128, row,
                        2 * ks, rt, full0 + 8 * s);
                if (C::MN < NT && !is_s)  // the second MMA's columns
                    mp_load_codes(dst0 + (uint32_t)(s * C::STAGE + C::T_BYTES / 2), map, ks * 128, row + C::MN,
                                  full0 + 8 * s);
                s = sn;
                phase = pn;
            }
        }
        // drain: every copy of the pair has landed before a CTA exits (the last
        // NS of them; earlier ones were waited for before their reuse; the odd
        // CTA waits in the closing cluster barrier)
        if (is_s && rank == 0)
            for (uint32_t i = it > (uint32_t)NS ? it - NS : 0; i < it; i++)
                mbar_wait(bar(B_FULL + (int)(i % NS)), (i / NS) & 1, a.err);
        __syncwarp();
    } else if (warp == MG_W_MMA && rank == 1) {
        // the even CTA's last commits have arrived here before this CTA may exit
        volatile int ignore = 0;  // after an abort too
        if (lane == 0) tc_wait_cluster(bar(B_FIN), 0, a.err, &ignore);
        __syncwarp();
    } else if (warp == MG_W_MMA) {
        // -------------------------------------------------------------- MMA
        uint32_t ut = 0, phase = 0;
        int s = 0;
        bool ok = true, ready = false;
        const uint32_t slo = sw128_lo(sbase);
        constexpr uint32_t SD = C::STAGE / 16;  // descriptor words between stages
        for (int u = first; u < a.n_tiles && ok; u += step, ut++) {
            const int buf = (int)(ut & 1);
            // The epilogue frees the columns that a tile's accumulator shares with
            // the next one's; with none shared, wait for the tile before last.
            const uint32_t prev = C::OVER < NT ? ut : ut - 1;
            if (ut >= 1 && prev >= 1) {
                const uint32_t t = prev - 1;
                if (!__all_sync(0xffffffffu,
                                tc_wait_cluster(bar(B_ACCE + (int)(t & 1)), (t / 2) & 1, a.err, abort_flag)))
                    break;
            }
            tc_fence_after();
            const uint32_t tacc = tmem + (uint32_t)(buf ? C::OVER : 0);
            // a 192-column tile starts at a half of a scale atom's rows every other time
            const uint32_t shift = (uint32_t)(((u % a.tiles_t) * NT % 128) / 32);
            for (int ks = 0; ks < a.nks; ks++) {
                if (!ready && !__all_sync(0xffffffffu, tc_wait_cluster(bar(B_FULL + s), phase, a.err, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int sn = s + 1 == NS ? 0 : s + 1;
                const uint32_t pn = sn ? phase : phase ^ 1u;
                // look at the next stage while this one is issued
                ready = __all_sync(0xffffffffu, mbar_test_cluster(bar(B_FULL + sn), pn));
                mg_step<2, NT>(tacc, slo + (uint32_t)s * SD, slo + C::OFF_T / 16 + (uint32_t)s * SD,
                                      slo + C::OFF_SA / 16 + (uint32_t)s * SD, tmem + (uint32_t)(C::SF0 + C::SF * s),
                                      shift, ks ? 1u : 0u);
                mp_commit(bar(B_EMPTY + s));
                s = sn;
                phase = pn;
            }
            if (!ok) break;
            mp_commit(bar(B_ACCF + buf));
        }
        // every MMA and copy issued above has completed before TMEM is freed
        mp_commit(bar(B_FIN));
        mbar_wait(bar(B_FIN), 0, a.err);
        __syncwarp();
    } else if (warp >= MG_W_EPI) {
        // --------------------------------------------------------- epilogue
        // A lane holds one row m.  A warp stages 32 rows of 128 bytes (64 bf16 or 32
        // fp32 n; 16-byte chunk c of row r at chunk c ^ (r mod 8), as the 128-byte
        // swizzle has it) and they leave by TMA, or, where C's rows are not made of
        // aligned 16-byte units, read back a row at a time.
        const int q = warp & 3, half = (warp - MG_W_EPI) >> 2;
        constexpr int PC = 128 / (int)sizeof(CT), NP = NT / PC;  // columns of a piece, pieces of a tile
        uint8_t *box = sm + C::OFF_C + (warp - MG_W_EPI) * MP_BOX;
        uint32_t ut = 0;
        for (int u = first; u < a.n_tiles; u += step, ut++) {
            const int buf = (int)(ut & 1);
            if (!__all_sync(0xffffffffu, tc_wait_cluster(bar(B_ACCF + buf), (ut / 2) & 1, a.err, abort_flag))) break;
            tc_fence_after();
            const uint32_t tacc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf ? C::OVER : 0);
            const int m0 = (u / a.tiles_t) * 2 * MG_M + rank * MG_M + q * 32, n0 = (u % a.tiles_t) * NT;
            // The two warps of a quadrant take alternate pieces, those in the
            // columns shared with the other accumulator first: the last SHARED of
            // the first accumulator, the first of the second.
            constexpr int SHARED = C::OVER < NT ? NT - C::OVER : NT, SP = SHARED / PC;
            static_assert(SHARED % PC == 0 && SP >= 2, "shared columns in whole pieces");
#pragma unroll 1
            for (int i = half; i < NP; i += 2) {
                const int j = C::OVER < NT && !buf ? (i + C::OVER / PC) % NP : i, n = n0 + j * PC;
                uint32_t r[PC / 32][32];
#pragma unroll
                for (int h = 0; h < PC / 32; h++) tmem_ld_chunk(tacc + (uint32_t)(j * PC + 32 * h), r[h]);
                if (i + 2 >= SP && i < SP) {  // this warp's last shared piece
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_rank(bar(B_ACCE + buf), 0);
                }
                // the piece staged before has been read
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
#pragma unroll
                for (int h = 0; h < PC / 32; h++) {
                    constexpr int W = 32 * (int)sizeof(CT) / 16;  // 16-byte chunks of 32 columns
#pragma unroll
                    for (int c = 0; c < W; c++) {
                        uint4 v;
                        if constexpr (sizeof(CT) == 2) {
                            uint32_t w[4];
#pragma unroll
                            for (int x = 0; x < 4; x++) {
                                const __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(r[h][8 * c + 2 * x]),
                                                                               __uint_as_float(r[h][8 * c + 2 * x + 1]));
                                w[x] = *(const uint32_t *)&p;
                            }
                            v = make_uint4(w[0], w[1], w[2], w[3]);
                        } else {
                            v = make_uint4(r[h][4 * c], r[h][4 * c + 1], r[h][4 * c + 2], r[h][4 * c + 3]);
                        }
                        *(uint4 *)(box + lane * 128 + (((h * W + c) ^ (lane & 7)) << 4)) = v;
                    }
                }
                if (a.tma) {
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0 && m0 < a.M && n < a.N) {
                        tma_store_2d(&cmap, smem_addr(box), n, m0, a.accumulate);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                } else {
                    __syncwarp();
                    for (int r = 0; r < 32 && m0 + r < a.M; r++)
#pragma unroll
                        for (int c = lane; c < PC; c += 32)
                            if (n + c < a.N) {
                                const int at = c * (int)sizeof(CT);
                                const CT v = *(const CT *)(box + r * 128 + (((at >> 4) ^ (r & 7)) << 4) + (at & 15));
                                put((CT *)a.C + n + c, (long)(m0 + r) * a.ldc, (float)v, a.accumulate);
                            }
                    __syncwarp();
                }
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves, or frees TMEM, while the other's work may reach it
    if (warp == MG_W_MMA) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// ---------------------------------------------------------------- launchers

PFN_cuTensorMapEncodeTiled_v12000 map_encoder()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            fn = nullptr;
        }
        return (PFN_cuTensorMapEncodeTiled_v12000)fn;
    }();
    return encode;
}
int make_map(CUtensorMap *map, CUtensorMapDataType type, int nd, const void *p, const cuuint64_t *dims,
             const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle)
{
    const auto encode = map_encoder();
    if (!encode) return K3MOE_ECUDA;
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode(map, type, (cuuint32_t)nd, (void *)p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? K3MOE_OK
               : K3MOE_EINVAL;
}
// Codes plane of an operand in boxes of box_rows x 128 bytes (256 codes),
// 128-byte swizzle; rows and bytes past the plane read as zero.
int code_map(CUtensorMap *map, const k3moe_mx_operand *op, int box_rows)
{
    const cuuint64_t width = (cuuint64_t)(op_in_padded(op->in) / 2);
    const cuuint64_t dims[2] = {width, (cuuint64_t)op->rows}, strides[1] = {width};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, op->codes, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
// The scale atoms of an operand, [row tile][k][512 bytes], in boxes of two k of
// `tiles` row tiles.
int atom_map(CUtensorMap *map, const k3moe_mx_operand *op, int tiles)
{
    const cuuint64_t nk = (cuuint64_t)op_k_atoms(op->in);
    const cuuint64_t dims[3] = {128, nk, (cuuint64_t)op_row_tiles(op->rows)}, strides[2] = {512, nk * 512};
    const cuuint32_t box[3] = {128, 2, (cuuint32_t)tiles};
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, op->atoms, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}
// C in boxes of a staged piece: 32 rows of 128 bytes, 128-byte swizzle.
template <typename CT>
int c_map(CUtensorMap *map, const MgArgs &a)
{
    const cuuint64_t dims[2] = {(cuuint64_t)a.N, (cuuint64_t)a.M}, strides[1] = {(cuuint64_t)a.ldc * sizeof(CT)};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / sizeof(CT)), 32};
    return make_map(map, sizeof(CT) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, a.C, dims,
                    strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Grid of CTAs in clusters of `cluster`, as a programmatic dependent.
template <typename... KArgs, typename... Args>
int launch_clusters(void (*kernel)(KArgs...), int grid, int cluster, int threads, size_t smem, cudaStream_t s,
                    const Args &...args)
{
    if (ensure_smem((const void *)kernel, smem) != K3MOE_OK) return K3MOE_ECUDA;
    if (launch_dependent(true, cluster, kernel, dim3((unsigned)grid), dim3((unsigned)threads), smem, s, args...) !=
        cudaSuccess) {
        cudaGetLastError();
        return K3MOE_ECUDA;
    }
    return K3MOE_OK;
}

template <int NT, bool SPLIT, typename CT>
int launch_tiles(const k3moe_mx_operand *A, const k3moe_mx_operand *B, MgArgs a, int ranks, cudaStream_t s)
{
    using C = MgCfg<NT, SPLIT>;
    CUtensorMap smap, tmap;
    int st = code_map(&smap, B, MG_M);
    if (st == K3MOE_OK) st = code_map(&tmap, A, NT);
    if (st != K3MOE_OK) return st;
    a.tiles_t = (a.M + NT - 1) / NT;
    a.n_tiles = a.tiles_t * ((a.N + MG_M - 1) / MG_M);
    return launch_clusters(k3_mx_matmul<NT, SPLIT, CT>, SPLIT ? a.n_tiles * ranks : std::min(a.n_tiles, num_sms()), ranks,
                           MG_THREADS, C::SMEM, s, smap, tmap, a);
}
template <int NT, typename CT>
int launch_nt(const k3moe_mx_operand *A, const k3moe_mx_operand *B, const MgArgs &a, int ranks, cudaStream_t s)
{
    if constexpr (NT <= 64)
        if (ranks > 1) return launch_tiles<NT, true, CT>(A, B, a, ranks, s);
    return launch_tiles<NT, false, CT>(A, B, a, 1, s);
}

template <int NT, typename CT>
int launch_pair(const k3moe_mx_operand *A, const k3moe_mx_operand *B, MgArgs a, cudaStream_t s)
{
    CUtensorMap smap, tmap, samap, tamap, cmap;
    int st = code_map(&smap, A, MG_M);
    if (st == K3MOE_OK) st = code_map(&tmap, B, MpCfg<NT>::MN / 2);
    if (st == K3MOE_OK) st = atom_map(&samap, A, 1);
    if (st == K3MOE_OK) st = atom_map(&tamap, B, MpCfg<NT>::QT);
    if (st != K3MOE_OK) return st;
    // C by TMA needs rows of whole, aligned 16-byte units: a store clips at the
    // edge of the matrix in such units (measured: it wrote past an odd N)
    a.tma = ((uintptr_t)a.C & 15u) == 0 && a.ldc * (long)sizeof(CT) % 16 == 0 && a.N * (long)sizeof(CT) % 16 == 0 &&
            c_map<CT>(&cmap, a) == K3MOE_OK;
    if (!a.tma) cmap = smap;  // unused
    a.tiles_t = (a.N + NT - 1) / NT;
    a.n_tiles = a.tiles_t * ((a.M + 2 * MG_M - 1) / (2 * MG_M));
    return launch_clusters(k3_mx_matmul_pair<NT, CT>, 2 * std::min(a.n_tiles, num_sms() / 2), 2, MP_THREADS,
                           MpCfg<NT>::SMEM, s, smap, tmap, samap, tamap, cmap, a);
}

// How a product runs: CTA pairs or single CTAs, columns per tile, CTAs per tile.
struct MgPlan {
    bool pair;
    int nt, ranks;
};

// The form by a model of its time, fitted on one GB300: a start, and for every wave of
// tiles over the SMs a time per k-step and one per tile.  Forms: narrow tiles (as
// many columns as there are rows of A, 64 at most), tiles of 128 columns, pairs of
// 192, 256 and 384.  Few narrow tiles with a long K are split over 2 to 8 CTAs, no
// more than there are SMs (two per SM lost: 32 x 4096 x 4096 over 8 took 7.1 us, over
// 4 5.1, whole 5.6); the join grows with the ranks and columns.
// Fitted to 27 products of 200 to 8192 rows, 1024 to 20000 columns and K 256 to 8192,
// 54 of 65 to 1024 rows and 48 of 1 to 128, in bf16 and fp32, each run in every form:
// the choice was the fastest form or within 5% of it in nearly all.  Some, in us:
//   1 x 1536 x 7168      narrow over 8 4.6, whole 7.5
//   128 x 1536 x 7168    narrow over 4 6.7, whole 8.2, 128 columns over 8 7.8
//   512 x 2048 x 2048    narrow 4.5, 128 columns 5.4
//   1536 x 1536 x 7168   128 columns 9.5, pairs of 192 11.8
//   2048 x 1536 x 7168   pairs of 192 12.0, one wave of 256 13.3, 128 columns 15.6
//   4096 x 1536 x 7168   pairs of 384, one wave, 17.9, 192, two waves, 19.4
//   4096 x 7168 x 1536   pairs of 256 20.2, 192 21.6, 384 23.0
MgPlan choose_plan(int M, int N, int nks, int sms, bool bf16)
{
    const int nt = M <= 16 ? 16 : M <= 32 ? 32 : 64;
    const long tn = ((long)N + MG_M - 1) / MG_M, tm = ((long)M + 2 * MG_M - 1) / (2 * MG_M);
    const long pairs = std::max(1, sms / 2);
    const struct {
        MgPlan plan;
        long tiles, at_once, start, step, tile;  // ns
    } forms[5] = {{{false, nt, 1}, tn * ((M + nt - 1L) / nt), sms, nt == 64 ? 2650 : 2400, nt == 64 ? 185 : 170,
                   nt < 64 ? 350 : bf16 ? 400 : 450},
                  {{false, 128, 1}, tn * (((long)M + 127) / 128), sms, 2610, 199, bf16 ? 840 : 1000},
                  {{true, 192, 1}, tm * (((long)N + 191) / 192), pairs, 4400, 252, bf16 ? 640 : 1250},
                  {{true, 256, 1}, tm * (((long)N + 255) / 256), pairs, 4400, 284, bf16 ? 950 : 2000},
                  {{true, 384, 1}, tm * (((long)N + 383) / 384), pairs, 4400, 410, bf16 ? 2000 : 3300}};
    MgPlan best = forms[0].plan;
    long cost = 0;
    for (const auto &f : forms) {
        const long c = f.start + (f.tiles + f.at_once - 1) / f.at_once * (f.step * nks + f.tile);
        if (!cost || c < cost) cost = c, best = f.plan;
    }
    const long start = nt == 16 ? 3900 : nt == 32 ? 4300 : 4600, rank = nt == 16 ? 40 : nt == 32 ? 60 : 100;
    for (int r = 2; r <= MG_MAX_RANKS && r <= nks && forms[0].tiles * r <= sms; r *= 2) {
        const long c = start + rank * r + (nt == 64 ? 225L : 170L) * ((nks + r - 1) / r);
        if (c < cost) cost = c, best = {false, nt, r};
    }
    return best;
}

template <typename CT>
int launch_ct(const k3moe_mx_operand *A, const k3moe_mx_operand *B, const MgArgs &a, cudaStream_t s)
{
    const MgPlan p = choose_plan(a.M, a.N, a.nks, num_sms(), sizeof(CT) == 2);
    if (p.pair)
        return p.nt == 384   ? launch_pair<384, CT>(A, B, a, s)
               : p.nt == 256 ? launch_pair<256, CT>(A, B, a, s)
                             : launch_pair<192, CT>(A, B, a, s);
    switch (p.nt) {
    case 16: return launch_nt<16, CT>(A, B, a, p.ranks, s);
    case 32: return launch_nt<32, CT>(A, B, a, p.ranks, s);
    case 64: return launch_nt<64, CT>(A, B, a, p.ranks, s);
    default: return launch_nt<128, CT>(A, B, a, p.ranks, s);
    }
}

}  // namespace

void mx_matmul_form(int M, int N, int in, int cdt, int *pair, int *columns, int *ranks)
{
    const MgPlan p = choose_plan(M, N, (in + 255) / 256, num_sms(), cdt == K3MOE_BF16);
    *pair = p.pair, *columns = p.nt, *ranks = p.ranks;
}

int launch_mx_matmul(void *C, int cdt, long ldc, const k3moe_mx_operand *A, const k3moe_mx_operand *B, int accumulate,
                     int *err, cudaStream_t s)
{
    MgArgs a = {};
    a.satoms = B->atoms;
    a.tatoms = A->atoms;
    a.C = C;
    a.ldc = ldc;
    a.M = A->rows;
    a.N = B->rows;
    a.nks = (A->in + 255) / 256;
    a.nka = op_k_atoms(A->in);
    a.accumulate = accumulate;
    a.vec = ldc % 4 == 0 && ((uintptr_t)C & (cdt == K3MOE_BF16 ? 7u : 15u)) == 0;
    a.err = err;
    const long tiles = (((long)a.M + 15) / 16) * (((long)a.N + MG_M - 1) / MG_M);
    if (tiles > 0x7fffffffL / 8) return K3MOE_EINVAL;
    return cdt == K3MOE_BF16 ? launch_ct<__nv_bfloat16>(A, B, a, s) : launch_ct<float>(A, B, a, s);
}

}  // namespace k3
