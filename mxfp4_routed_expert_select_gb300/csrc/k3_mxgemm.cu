// k3_mxgemm.cu -- the product of two MXFP4 operands, C = A B^T, on the
// block-scaled tensor cores (tcgen05.mma kind::mxf4).
//
// C[m][n] = sum over blocks b of 2^(ea[m][b] + eb[n][b] - 254) times the sum of
// the 32 code products of block b: the tensor core multiplies the E2M1 codes as
// stored and applies both E8M0 scales itself, accumulating in fp32 in TMEM.
//
// B's rows (the weights' output features) take the MMA's 128 lanes and A's rows
// (the tokens) its NT columns, whatever their number: a few tokens then cost a
// narrow MMA over the streamed weights, and in the epilogue a warp holds 32
// consecutive n of one m, so that its stores of C are coalesced with no
// transposition.
//
// Roles (256 threads): warp 0 copies the operands (TMA, 256 of K per stage: B
// 128 rows x 128 bytes, A NT rows x 128 bytes, 128-byte swizzle, and their
// scale atoms, which are stored in the order tensor memory takes them in), warp
// 1 issues the scale copies and MMAs, warps 4 to 7 read the accumulators.  Rows,
// columns and K past the matrices are zero-filled by the copies.
//
// Two launch forms of one kernel:
//  - tiles: one CTA per SM walks the 128 x NT tiles; the accumulator of one tile
//    is read out while the next one's products run.
//  - split: with fewer tiles than SMs, a cluster of S CTAs shares one tile, each
//    taking 1/S of K; their partial sums meet in distributed shared memory, where
//    each CTA adds one slice of the columns over the S ranks in rank order (the
//    result does not depend on timing).
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

constexpr int MG_M = 128;       // B rows per tile
constexpr int MG_THREADS = 256;
constexpr int MG_MAX_RANKS = 8;  // CTAs that share a tile
constexpr int MG_W_PROD = 0, MG_W_MMA = 1, MG_W_EPI = 4;

struct MgArgs {
    const uint8_t *satoms, *tatoms;  // scale atoms of B (lanes) and A (columns)
    void *C;
    long ldc;
    int M, N, nks, nka;              // A rows, B rows, 256-long k-steps, atoms per row tile
    int tiles_m, n_tiles;            // column tiles, all tiles
    int accumulate;
    int *err;
};

// Shared memory and TMEM of one CTA with NT columns, one tile per cluster
// (SPLIT) or many per CTA.
template <int NT, bool SPLIT>
struct MgCfg {
    static constexpr int QT = (NT + 127) / 128;             // row tiles of A's scale atoms
    static constexpr int S_BYTES = MG_M * 128, T_BYTES = NT * 128;
    static constexpr int OFF_T = S_BYTES;
    static constexpr int OFF_SA = OFF_T + T_BYTES;           // B's two atoms
    static constexpr int OFF_TA = OFF_SA + 1024;             // A's two atoms per row tile
    static constexpr int TX = OFF_TA + QT * 1024;            // bytes copied per stage
    static constexpr int STAGE = (TX + 1023) / 1024 * 1024;
    // Split CTAs share an SM in pairs where the stages allow it.
    static constexpr int NS = SPLIT ? (NT >= 256 ? 4 : NT == 128 ? 3 : NT <= 16 ? 5 : 4) : (NT >= 256 ? 4 : 6);
    // A stage's scales: B's atoms in 8 columns, A's in 8 per row tile (k-atom
    // major, 4 columns per 128 rows).
    static constexpr int SF = 8 + 8 * QT;
    // Accumulators: two of NT columns.  Two of 256 do not fit beside the
    // scales: the second starts at OVER, and the columns they share are read
    // first.
    static constexpr int NACC = SPLIT ? 1 : 2;
    static constexpr int OVER = NACC == 2 && NT == 256 ? 512 - SF * NS - 256 : NT;  // start of the second accumulator
    static constexpr int SF0 = NACC == 2 ? OVER + NT : NT;                          // start of the scales
    static constexpr int COLS_USED = SF0 + SF * NS;
    static constexpr int TMEM_COLS = COLS_USED <= 128 ? 128 : COLS_USED <= 256 ? 256 : 512;
    static constexpr int BARS = 2 * NS + 2 * 2 + 1;
    static constexpr int SMEM = 1024 + NS * STAGE + 256;
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(COLS_USED <= 512, "TMEM layout");
    static_assert(!SPLIT || NT * MG_M * 4 <= NS * STAGE, "partial sums reuse the stages");
};

K3_DEV uint32_t mg_idesc(int n, uint32_t sfid)
{
    // E2M1 x E2M1, K-major, UE8M0 scales, M = 128; sfid: the first of this MMA's
    // two scale bytes within the 32-bit scale words of A and B
    return (sfid << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
           ((uint32_t)(MG_M >> 4) << 24) | (sfid << 29);
}
K3_DEV void mg_mma(uint32_t td, uint32_t slo, uint32_t tlo, uint32_t idesc, uint32_t sfs, uint32_t sft, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "mov.b64 da, {%1, %7};\n\tmov.b64 db, {%2, %7};\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %3, [%5], [%6], p;\n\t}"
                 ::"r"(td), "r"(slo), "r"(tlo), "r"(idesc), "r"(acc), "r"(sfs), "r"(sft), "r"(SW128_HI)
                 : "memory");
}
// One 512-byte scale atom (32 rows x 16 bytes) from shared memory to TMEM
// columns taddr .. taddr + 3, repeated in the four lane quadrants.
K3_DEV void mg_cp_atom(uint32_t taddr, uint32_t saddr)
{
    const uint32_t lo = ((saddr & 0x3FFFFu) >> 4) | (1u << 16), hi = (128u >> 4) | (1u << 14);
    asm volatile("{\n\t.reg .pred e;\n\t.reg .b64 d;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "mov.b64 d, {%1, %2};\n\t@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr),
                 "r"(lo), "r"(hi)
                 : "memory");
}
// 16 or 32 columns of the accumulator, one row per lane.  The wait names the
// registers, so that nothing made from them can move above it.
K3_DEV void tmem_ld_chunk(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
        "}, [%16];"
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
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
        "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
        "}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
          "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
          "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
          "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
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
K3_DEV float ld_peer(uint32_t addr, uint32_t rank)
{
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

template <typename CT>
K3_DEV void put(CT *C, long i, float v, int accumulate)
{
    if constexpr (sizeof(CT) == 2)
        C[i] = __float2bfloat16_rn(v);
    else
        C[i] = accumulate ? C[i] + v : v;
}

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
    auto stage = [&](int s) { return sbase + (uint32_t)(s * C::STAGE); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // this CTA's tiles and its range of k-steps
    const int rank = SPLIT ? (int)cluster_rank() : 0, ranks = SPLIT ? (int)cluster_size() : 1;
    const int first = SPLIT ? (int)blockIdx.x / ranks : (int)blockIdx.x;
    const int step = SPLIT ? a.n_tiles : (int)gridDim.x;
    const int k0 = (int)((long)a.nks * rank / ranks), k1 = (int)((long)a.nks * (rank + 1) / ranks);

    if (threadIdx.x == 0) {
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
    griddep_launch_dependents();
    griddep_wait();

    if (warp == MG_W_PROD) {
        // --------------------------------------------------------- producer
        uint32_t issued[NS];
#pragma unroll
        for (int i = 0; i < NS; i++) issued[i] = 0;
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int u = first; u < a.n_tiles && ok; u += step) {
                const int tn = u / a.tiles_m, tm = u % a.tiles_m;
                const uint8_t *sa = a.satoms + (long)tn * a.nka * 512;
                const uint8_t *ta = a.tatoms + (long)tm * C::QT * a.nka * 512;
                // with 256 columns the last tile's second row tile may not exist
                const int qt = C::QT == 1 || tm * NT + 128 < a.M ? C::QT : 1;
                for (int ks = k0; ks < k1; ks++, it++) {
                    const int s = it % NS;
                    if (it >= (uint32_t)NS && !tc_wait(bar(B_EMPTY + s), ((it / NS) - 1) & 1, a.err, abort_flag)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(bar(B_FULL + s), (uint32_t)(C::OFF_TA + qt * 1024));
#pragma unroll
                    for (int i = 0; i < NS; i++) issued[i] += i == s;
                    tma_load_2d(stage(s), &smap, ks * 128, tn * MG_M, bar(B_FULL + s));
                    tma_load_2d(stage(s) + C::OFF_T, &tmap, ks * 128, tm * NT, bar(B_FULL + s));
                    bulk_g2s(stage(s) + C::OFF_SA, sa + (long)ks * 1024, 1024, bar(B_FULL + s));
                    for (int q = 0; q < qt; q++)
                        bulk_g2s(stage(s) + C::OFF_TA + 1024 * q, ta + ((long)q * a.nka + 2 * ks) * 512, 1024,
                                 bar(B_FULL + s));
                }
            }
            // drain: every copy issued here has landed before the CTA exits
#pragma unroll
            for (int s = 0; s < NS; s++)
                if (issued[s]) mbar_wait(bar(B_FULL + s), (issued[s] - 1) & 1, a.err);
        }
        __syncwarp();
    } else if (warp == MG_W_MMA) {
        // -------------------------------------------------------------- MMA
        uint32_t it = 0, ut = 0;
        bool ok = true;
        for (int u = first; u < a.n_tiles && ok; u += step, ut++) {
            const int buf = (int)(ut & 1);
            // The epilogue frees the columns that a tile's accumulator shares
            // with the next one's (all of the tile's, when they share none and
            // the tile before last used the same ones).
            const uint32_t prev = C::OVER < NT ? ut : ut - 1;  // this many earlier tiles must be free
            if (ut >= 1 && prev >= 1) {
                const uint32_t t = prev - 1;
                if (!__all_sync(0xffffffffu, tc_wait(bar(B_ACCE + (int)(t & 1)), (t / 2) & 1, a.err, abort_flag)))
                    break;
            }
            tc_fence_after();
            const uint32_t tacc = tmem + (uint32_t)(buf ? C::OVER : 0);
            for (int ks = k0; ks < k1; ks++, it++) {
                const int s = it % NS;
                if (!__all_sync(0xffffffffu, tc_wait(bar(B_FULL + s), (it / NS) & 1, a.err, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sfs = tmem + (uint32_t)(C::SF0 + C::SF * s), sft = sfs + 8;
                mg_cp_atom(sfs, stage(s) + C::OFF_SA);
                mg_cp_atom(sfs + 4, stage(s) + C::OFF_SA + 512);
#pragma unroll
                for (int ka = 0; ka < 2; ka++)
#pragma unroll
                    for (int q = 0; q < C::QT; q++)
                        mg_cp_atom(sft + (uint32_t)(4 * C::QT * ka + 4 * q),
                                   stage(s) + (uint32_t)(C::OFF_TA + 1024 * q + 512 * ka));
                const uint32_t slo = sw128_lo(stage(s)), tlo = sw128_lo(stage(s) + C::OFF_T);
#pragma unroll
                for (int q4 = 0; q4 < 4; q4++)  // K = 64 per MMA
                    mg_mma(tacc, slo + 2u * q4, tlo + 2u * q4, mg_idesc(NT, 2u * (q4 & 1)), sfs + 4 * (q4 >> 1),
                           sft + 4 * C::QT * (q4 >> 1), (ks == k0 && q4 == 0) ? 0u : 1u);
                mma_commit(bar(B_EMPTY + s));
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
            const uint32_t tacc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf ? C::OVER : 0);
            const int n = (u / a.tiles_m) * MG_M + q * 32 + lane, m0 = (u % a.tiles_m) * NT;
            // the columns shared with the other accumulator come first: the
            // last SHARED of the first accumulator, the first of the second
            constexpr int SHARED = C::OVER < NT ? NT - C::OVER : NT;
            static_assert(SPLIT || SHARED % CH == 0, "shared columns in whole chunks");
#pragma unroll 1
            for (int i = 0; i < NCH; i++) {
                const int j = C::OVER < NT && !buf ? (i + C::OVER / CH) % NCH : i;
                uint32_t r[CH];
                tmem_ld_chunk(tacc + (uint32_t)(j * CH), r);
                if (!SPLIT && i == SHARED / CH - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_ACCE + buf));
                }
                if constexpr (SPLIT) {
                    float *part = (float *)sm;  // [column][128]: every stage has been consumed
#pragma unroll
                    for (int c = 0; c < CH; c++) part[(j * CH + c) * MG_M + q * 32 + lane] = __uint_as_float(r[c]);
                } else if (n < a.N) {
                    CT *o = (CT *)a.C + n;
                    const int m = m0 + j * CH;
                    if (m + CH <= a.M) {
#pragma unroll
                        for (int c = 0; c < CH; c++)
                            put(o, (long)(m + c) * a.ldc, __uint_as_float(r[c]), a.accumulate);
                    } else {
#pragma unroll
                        for (int c = 0; c < CH; c++)
                            if (m + c < a.M) put(o, (long)(m + c) * a.ldc, __uint_as_float(r[c]), a.accumulate);
                    }
                }
            }
        }
    }

    tc_fence_before();
    if constexpr (SPLIT) {
        __syncwarp();
        cluster_sync();  // every rank's partial sums are in its shared memory
        const int u = first, n = (u / a.tiles_m) * MG_M + (int)(threadIdx.x & 127), m0 = (u % a.tiles_m) * NT;
        const int c0 = NT * rank / ranks, c1 = min(NT * (rank + 1) / ranks, a.M - m0);
        if (n < a.N && !*abort_flag)
            // four columns' partial sums of all ranks in flight at a time (a
            // remote load takes a few hundred cycles)
            for (int c = c0 + (int)(threadIdx.x >> 7); c < c1; c += 4 * (MG_THREADS / 128)) {
                float v[4][MG_MAX_RANKS];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int cj = min(c + j * (MG_THREADS / 128), c1 - 1);
                    const uint32_t at = sbase + (uint32_t)(cj * MG_M + (int)(threadIdx.x & 127)) * 4;
#pragma unroll
                    for (int r = 0; r < MG_MAX_RANKS; r++) v[j][r] = r < ranks ? ld_peer(at, (uint32_t)r) : 0.f;
                }
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int cj = c + j * (MG_THREADS / 128);
                    float t = v[j][0];
#pragma unroll
                    for (int r = 1; r < MG_MAX_RANKS; r++) t += v[j][r];
                    if (cj < c1) put((CT *)a.C, (long)(m0 + cj) * a.ldc + n, t, a.accumulate);
                }
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

// Codes plane of an operand in boxes of box_rows x 128 bytes (256 codes),
// 128-byte swizzle; rows and bytes past the plane read as zero.
int code_map(CUtensorMap *map, const k3moe_mx_operand *op, int box_rows)
{
    const auto encode = map_encoder();
    if (!encode) return K3MOE_ECUDA;
    const cuuint64_t width = (cuuint64_t)(op_in_padded(op->in) / 2);
    const cuuint64_t dims[2] = {width, (cuuint64_t)op->rows}, strides[1] = {width};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows}, estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (void *)op->codes, dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? K3MOE_OK
               : K3MOE_EINVAL;
}

template <int NT, bool SPLIT, typename CT>
int launch_tiles(const k3moe_mx_operand *A, const k3moe_mx_operand *B, MgArgs a, int ranks, cudaStream_t s)
{
    using C = MgCfg<NT, SPLIT>;
    const auto kernel = k3_mx_matmul<NT, SPLIT, CT>;
    CUtensorMap smap, tmap;
    int st = code_map(&smap, B, MG_M);
    if (st == K3MOE_OK) st = code_map(&tmap, A, NT);
    if (st == K3MOE_OK) st = ensure_smem((const void *)kernel, C::SMEM);
    if (st != K3MOE_OK) return st;
    a.tiles_m = (a.M + NT - 1) / NT;
    a.n_tiles = a.tiles_m * ((a.N + MG_M - 1) / MG_M);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(SPLIT ? a.n_tiles * ranks : std::min(a.n_tiles, num_sms())));
    cfg.blockDim = dim3(MG_THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = SPLIT ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, smap, tmap, a) != cudaSuccess) {
        cudaGetLastError();
        return K3MOE_ECUDA;
    }
    return K3MOE_OK;
}

template <int NT, typename CT>
int launch_nt(const k3moe_mx_operand *A, const k3moe_mx_operand *B, const MgArgs &a, int ranks, cudaStream_t s)
{
    return ranks > 1 ? launch_tiles<NT, true, CT>(A, B, a, ranks, s) : launch_tiles<NT, false, CT>(A, B, a, 1, s);
}

// Columns per tile and CTAs per tile.  With at most 128 rows of A one column
// tile holds them all.  Above that, 256 columns read B half as often and come
// nearer the tensor cores' rate, 128 fill the last wave better: the fewer waves
// win, a 128-column tile counting 0.6 of a 256-column one.  Tiles that leave
// SMs idle are split along K while every rank keeps at least two steps.
void choose_tiles(int M, int N, int nks, int sms, int &nt, int &ranks)
{
    const long tn = (N + MG_M - 1) / MG_M;
    nt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    if (M > 128) {
        const long t256 = tn * ((M + 255) / 256), t128 = tn * ((M + 127) / 128);
        if (t256 >= sms && 10 * ((t256 + sms - 1) / sms) <= 6 * ((t128 + sms - 1) / sms)) nt = 256;
    }
    const long tiles = tn * ((M + nt - 1) / nt);
    ranks = 1;
    while (ranks < MG_MAX_RANKS && tiles * ranks * 2 <= 2L * sms && nks >= 4 * ranks) ranks *= 2;
}

template <typename CT>
int launch_ct(const k3moe_mx_operand *A, const k3moe_mx_operand *B, const MgArgs &a, cudaStream_t s)
{
    int nt, ranks;
    choose_tiles(a.M, a.N, a.nks, num_sms(), nt, ranks);
    switch (nt) {
    case 16: return launch_nt<16, CT>(A, B, a, ranks, s);
    case 32: return launch_nt<32, CT>(A, B, a, ranks, s);
    case 64: return launch_nt<64, CT>(A, B, a, ranks, s);
    case 128: return launch_nt<128, CT>(A, B, a, ranks, s);
    default: return launch_tiles<256, false, CT>(A, B, a, 1, s);
    }
}

}  // namespace

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
    a.err = err;
    const long tiles = (((long)a.M + 15) / 16) * (((long)a.N + MG_M - 1) / MG_M);
    if (tiles > 0x7fffffffL / 8) return K3MOE_EINVAL;
    return cdt == K3MOE_BF16 ? launch_ct<__nv_bfloat16>(A, B, a, s) : launch_ct<float>(A, B, a, s);
}

}  // namespace k3
