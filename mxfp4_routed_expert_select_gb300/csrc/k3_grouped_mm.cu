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
// 72 clocks, 65536 rows x 1536 x 7168 took 2.94 ms; the same rows as tiles 0.76.)
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

struct GmArgs {
    const uint8_t *atoms;      // scale atoms of the weights, atoms_stride bytes from expert to expert
    long atoms_stride;
    const uint8_t *codes, *scales;  // of the rows
    int cstride, sstride;
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
// 16 bytes from global to shared memory, asynchronously.
K3_DEV void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The tiles of the batch, made by every CTA in shared memory: before[e] row tiles lie
// before expert e's, off[e] is its first place.
struct GmTable {
    int before[GM_MAX_E + 1], off[GM_MAX_E + 1], sums[32];
};
struct GmTile {
    int e, row, rows, n0;  // first row of C, rows of the group from there on (> 0), first weight row
};
template <int NT, int THREADS>
K3_DEV void gm_table(GmTable &tab, const GmArgs &a)
{
    constexpr int PER = (GM_MAX_E + 256 - 1) / 256;  // experts of each of the first 256 threads
    static_assert(THREADS >= 256, "threads of the table");
    int v[PER], mine = 0;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, e0 = PER * (int)threadIdx.x;
    if (threadIdx.x < 256) {
        int lo = e0 <= a.E ? min(max(a.offsets[e0], 0), a.slots) : 0;
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const int e = e0 + i, hi = e < a.E ? min(max(a.offsets[e + 1], lo), a.slots) : lo;
            if (e <= a.E) tab.off[e] = lo;
            v[i] = (hi - lo + NT - 1) / NT;
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

template <typename CT>
K3_DEV void gm_put(CT *p, float v, int accumulate)
{
    if constexpr (sizeof(CT) == 2)
        *p = __float2bfloat16_rn(v);
    else
        *p = accumulate ? *p + v : v;
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
    gm_table<NT, C::THREADS>(tab, a);
    const int n_tiles = tab.before[a.E] * a.tiles_n, first = (int)blockIdx.x, step = (int)gridDim.x;

    if (warp >= GM_W_FILL) {
        // -------------------------------------------------- a stage's filler
        // Every NS-th step of this CTA's tiles.  Lanes 8 q .. 8 q + 7 copy the 16-byte
        // chunks of rows q, q + 4, ..; a lane has the scale words of rows lane, lane +
        // 32, ... of the tile, loaded a turn ahead.  Columns past the group keep what
        // the stage held (they are not stored).
        constexpr int J = (NT + 31) / 32, R = NT / 4;
        const int s = warp - GM_W_FILL;
        const uint32_t st = sbase + (uint32_t)(s * C::STAGE), full = bar(B_FULL + s);
        uint32_t turn = 0;
        int u = first, ks = s, tile = -1;
        GmTile t = {};
        const uint8_t *atoms = nullptr, *sp[J];
        int src[R];
        uint32_t w[J];
        for (;; ks += NS, turn++) {
            while (ks >= a.nks) ks -= a.nks, u += step;
            if (u >= n_tiles) break;
            if (u != tile) {
                tile = u;
                t = gm_tile<NT>(tab, a, u);
                atoms = a.atoms + (long)t.e * a.atoms_stride + (long)(t.n0 / 128) * a.nka * 512;
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
            // before its first completion an EMPTY barrier's odd phase counts as passed
            if (!__all_sync(0xffffffffu, tc_wait(bar(B_EMPTY + s), (turn & 1) ^ 1u, a.err, abort_flag))) break;
            if (lane == 0) mbar_arrive_expect_tx(full, C::TX_W + (a.gather ? 0 : C::TX_X));
            __syncwarp();
            gm_load_w(st, &wmap, ks * 128, t.n0, t.e, st + C::OFF_WA, atoms + (long)ks * 512, full);
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
    } else if (warp >= GM_W_EPI) {
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
    const cuuint32_t xb[2] = {128, NT};
    if (st == K3MOE_OK)
        st = encode_map(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, A->codes, xd, xs, xb, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != K3MOE_OK) return st;
    if (ensure_smem((const void *)k3_grouped_matmul<NT, CT>, C::SMEM) != K3MOE_OK) return K3MOE_ECUDA;
    const long most = std::min<long>(a.slots, (long)a.E + a.slots / NT) * a.tiles_n;  // tiles there can be
    if (launch_pdl(k3_grouped_matmul<NT, CT>, dim3((unsigned)std::min<long>(most, num_sms())), dim3(C::THREADS), C::SMEM, s,
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
    a.codes = A->codes, a.scales = A->scales, a.cstride = op_in_padded(A->in), a.sstride = mx8_scale_stride(A->in);
    a.offsets = g->offsets, a.order = g->order;
    a.E = g->E, a.top_k = g->top_k, a.slots = g->tokens * g->top_k, a.gather = gather, a.xrows = A->rows;
    a.N = W->rows, a.nks = W->in / 128, a.nka = op_k_atoms(W->in), a.tiles_n = (W->rows + GM_M - 1) / GM_M;
    a.C = C, a.ldc = ldc, a.accumulate = accumulate, a.err = err;
    if (((long)a.E + a.slots) * a.tiles_n > 0x7fffffffL) return K3MOE_EINVAL;
    return cdt == K3MOE_BF16 ? launch_gm_ct<__nv_bfloat16>(A, W, a, s) : launch_gm_ct<float>(A, W, a, s);
}

}  // namespace k3
