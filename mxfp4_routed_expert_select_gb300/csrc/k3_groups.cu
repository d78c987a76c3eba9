// k3_groups.cu -- the slots of a routed batch grouped by expert, and the weighted
// sum of each token's expert rows with its gradients.
//
// Grouping is a stable counting sort of ids[T][k] (slot t k + j): offsets[e] counts
// the slots of lower experts, order lists the slots expert by expert in rising
// order, pos is its inverse.  One CTA sorts up to GR_WHOLE slots: each warp counts
// its own run of slots per expert, the counts are scanned over the warps and the
// experts, and the warps place their slots 32 at a time (the lanes that hold one
// expert rank themselves by a match).  More slots are cut in chunks: every chunk's
// counts, one CTA's scan over them, and the placing.  Ranks come from positions,
// never from the order of atomics, so the result is one and the same.
#include <cuda_runtime.h>

#include <algorithm>

#include "k3_e4m3.cuh"
#include "k3_launch.cuh"

namespace k3 {
size_t grouped_matmul_workspace_bytes();
namespace {

constexpr int GR_THREADS = 1024, GR_WARPS = GR_THREADS / 32;
constexpr int GR_WHOLE = 4096;  // slots that one CTA sorts alone; a warp's run fits the 16-bit counts
constexpr int GR_CHUNK = 2048;  // slots of a CTA where there are more
constexpr int GR_FEW = 256;     // chunks whose counts each CTA sums itself

struct GroupArgs {
    const int32_t *ids;
    int32_t *offsets, *order, *pos, *counts;  // counts [chunks][E]: of a chunk, then where its slots start
    int S, E, chunks;
};

// Exclusive sum over the block's threads; *total receives the whole sum.
K3_DEV int block_scan(int v, int *warp_sums, int *total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[w] = x;
    __syncthreads();
    if (w == 0) {
        int s = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    *total = warp_sums[31];
    return x - v + (w ? warp_sums[w - 1] : 0);
}

// The expert of a slot, -1 for a dropped one.
K3_DEV int expert_of(const GroupArgs &a, int slot, int end)
{
    if (slot >= end) return -1;
    const int e = a.ids[slot];
    return e >= 0 && e < a.E ? e : -1;
}

// WHOLE: one chunk is the batch (4096 slots of 896 experts: 9.8 us, 10.7 in chunks; 2048:
// 6.7 and 10.5).  Otherwise COUNT leaves the chunk's counts, and the placing pass reads
// where each expert's slots of this chunk start: sums over the chunks' counts, which each
// CTA forms itself where there are few (SCAN; one launch less: 65536 slots 12.2 us, with
// a scan's results 15.0; 2^19 42 and 54, 2^20 122 and 104).
template <bool WHOLE, bool COUNT, bool SCAN>
__global__ void __launch_bounds__(GR_THREADS) k3_groups(const GroupArgs a)
{
    extern __shared__ uint16_t cnt[];  // [GR_WARPS][E]: of a warp, then of the warps before it
    __shared__ int warp_sums[32];
    __shared__ int starts[1024];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int first = (int)blockIdx.x * GR_CHUNK, n = WHOLE ? a.S : min(GR_CHUNK, a.S - first);
    const int run = (n + GR_THREADS - 1) / GR_THREADS * 32, warps = (n + run - 1) / run;  // warps with slots
    for (int i = threadIdx.x; i < (warps * a.E + 7) / 8; i += GR_THREADS) ((uint4 *)cnt)[i] = make_uint4(0u, 0u, 0u, 0u);
    griddep_wait();
    griddep_launch_dependents();
    const int s0 = first + w * run, s1 = min(first + n, s0 + run);
    uint16_t *mine = cnt + w * a.E;
    constexpr int IT = (WHOLE ? GR_WHOLE : GR_CHUNK) / GR_THREADS;
    int x[IT];
    uint32_t same[IT];
#pragma unroll
    for (int i = 0; i < IT; i++) x[i] = expert_of(a, s0 + 32 * i + lane, s1);
#pragma unroll
    for (int i = 0; i < IT; i++) same[i] = __match_any_sync(0xffffffffu, x[i]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < IT; i++) {
        if (x[i] >= 0 && (same[i] & ((1u << lane) - 1)) == 0) mine[x[i]] += (uint16_t)__popc(same[i]);
        __syncwarp();
    }
    __syncthreads();
    const int e = threadIdx.x;
    int total = 0;
    if (e < a.E) {
        int c[GR_WARPS];
#pragma unroll
        for (int i = 0; i < GR_WARPS; i++) c[i] = i < warps ? cnt[i * a.E + e] : 0;
#pragma unroll
        for (int i = 0; i < GR_WARPS; i++) {
            if (i < warps) cnt[i * a.E + e] = (uint16_t)total;
            total += c[i];
        }
    }
    if constexpr (COUNT) {
        if (e < a.E) a.counts[(long)blockIdx.x * a.E + e] = total;
        return;
    }
    int kept;
    if constexpr (WHOLE) {
        const int at = block_scan(total, warp_sums, &kept);
        if (e < a.E) starts[e] = at, a.offsets[e] = at;
        if (e == 0) a.offsets[a.E] = kept;
    } else if constexpr (SCAN) {
        int before = 0, all = 0;
        if (e < a.E)
#pragma unroll 8
            for (int c = 0; c < a.chunks; c++) {
                const int v = a.counts[(long)c * a.E + e];
                before += c < (int)blockIdx.x ? v : 0;
                all += v;
            }
        const int at = block_scan(all, warp_sums, &kept);
        if (e < a.E) {
            starts[e] = at + before;
            if (blockIdx.x == 0) a.offsets[e] = at;
        }
        if (e == 0 && blockIdx.x == 0) a.offsets[a.E] = kept;
    } else {
        if (e < a.E) starts[e] = a.counts[(long)blockIdx.x * a.E + e];
        kept = a.offsets[a.E];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < IT; i++) {
        const uint32_t before = same[i] & ((1u << lane) - 1);
        const int p = x[i] >= 0 ? starts[x[i]] + mine[x[i]] + __popc(before) : -1, s = s0 + 32 * i + lane;
        __syncwarp();
        if (x[i] >= 0 && before == 0) mine[x[i]] += (uint16_t)__popc(same[i]);
        __syncwarp();
        if (s < s1) {
            a.pos[s] = p;
            if (p >= 0) a.order[p] = s;
        }
    }
    // the places behind the last group
    for (int i = first + threadIdx.x; i < first + n; i += GR_THREADS)
        if (i >= kept) a.order[i] = -1;
}

// Counts of the chunks to where their slots start, and the offsets.
__global__ void __launch_bounds__(GR_THREADS) k3_groups_scan(const GroupArgs a)
{
    __shared__ int warp_sums[32];
    griddep_wait();
    griddep_launch_dependents();
    const int e = threadIdx.x;
    int total = 0, kept;
    if (e < a.E)
#pragma unroll 8
        for (int c = 0; c < a.chunks; c++) total += a.counts[(long)c * a.E + e];
    int at = block_scan(total, warp_sums, &kept);
    if (e < a.E) {
        a.offsets[e] = at;
#pragma unroll 8
        for (int c = 0; c < a.chunks; c++) {
            const int v = a.counts[(long)c * a.E + e];
            a.counts[(long)c * a.E + e] = at;
            at += v;
        }
    }
    if (e == 0) a.offsets[a.E] = kept;
}

// ------------------------------------------------------------- the combine
//
// out[t] (+)= sum_j w[t][j] y[pos[t][j]] over a token's slots, in rising j.
// Bound: HBM, each row of y read once.  A thread takes eight columns of a token and
// has up to CB_DEEP slots' loads in flight (4096 tokens x 16 x 7168 bf16, 1 GB: 135 us;
// backward, 1.9 GB: 296).

constexpr int CB_DEEP = 8;

struct CombineArgs {
    const void *y, *dout;
    void *out, *dy;
    long ldy, ldo, lddy;  // ldo: of out, or of dout
    const float *w;
    float *dw;
    const int32_t *pos;
    int T, k, n, rows, accumulate;  // rows: slots, what pos stays below
    int blocks;                     // CTAs of a token
};

// Where slot j of a token's row is, -1 for a dropped one; its weight.
K3_DEV int place_of(const CombineArgs &a, long slot)
{
    const int p = a.pos[slot];
    return p >= 0 && p < a.rows ? p : -1;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(128) k3_combine(const CombineArgs a)
{
    griddep_wait();
    griddep_launch_dependents();
    const int t = (int)(blockIdx.x / (uint32_t)a.blocks), c = ((int)(blockIdx.x % (uint32_t)a.blocks) * 128 + (int)threadIdx.x) * 8;
    if (c >= a.n) return;
    float v[8] = {};
    if (a.accumulate) {
        const Raw<T> o = load8<T, VEC>(a.out, a.ldo, t, c, a.n);
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = value(o, i);
    }
    for (int j0 = 0; j0 < a.k; j0 += CB_DEEP) {
        Raw<T> r[CB_DEEP];
        float w[CB_DEEP];
#pragma unroll
        for (int j = 0; j < CB_DEEP; j++) {
            const long slot = (long)t * a.k + j0 + j;
            const int p = j0 + j < a.k ? place_of(a, slot) : -1;
            w[j] = p < 0 ? 0.f : a.w ? a.w[slot] : 1.f;
            r[j] = load8<T, VEC>(a.y, a.ldy, max(p, 0), p < 0 ? a.n : c, a.n);
        }
#pragma unroll
        for (int j = 0; j < CB_DEEP; j++)
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] += w[j] * value(r[j], i);
    }
    store8<T, VEC>(a.out, a.ldo, t, c, a.n, v);
}

// dy[pos[t][j]] = w[t][j] dout[t],  dw[t][j] = <dout[t], y[pos[t][j]]>.  A CTA takes
// DEEP slots of a token, its threads eight columns at a time; the dot products are
// joined together.  Its threads are the fewer the more CTAs there are: 512 where they
// all run at once, 256, and 128 from three CTAs an SM on (7168 bf16, us, 512, 256 and 128:
// 64 tokens x 4 3.4 3.8 4.7, 64 x 16 5.1 5.0 5.9, 256 x 16 19.9 17.7 16.6, 4096 x 16 325 293
// 296; 2048 bf16, 4096 x 16 101 101 85).  Eight slots to a CTA of 256: 64 x 16 6.4,
// 256 x 16 20.7, 4096 x 16 318.
constexpr int CBB_DEEP = 4;

template <typename T, bool VEC>
__global__ void __launch_bounds__(512) k3_combine_backward(const CombineArgs a)
{
    constexpr int DEEP = CBB_DEEP;
    __shared__ float sh[DEEP][32];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int t = (int)(blockIdx.x / (uint32_t)a.blocks), j0 = (int)(blockIdx.x % (uint32_t)a.blocks) * DEEP;
    int p[DEEP];
    float w[DEEP], dot[DEEP];
#pragma unroll
    for (int j = 0; j < DEEP; j++) {
        const long slot = (long)t * a.k + j0 + j;
        p[j] = j0 + j < a.k ? place_of(a, slot) : -1;
        w[j] = p[j] < 0 ? 0.f : a.w ? a.w[slot] : 1.f;
        dot[j] = 0.f;
    }
    for (int c = (int)threadIdx.x * 8; c < a.n; c += (int)blockDim.x * 8) {
        const Raw<T> g = load8<T, VEC>(a.dout, a.ldo, t, c, a.n);
        Raw<T> r[DEEP];
        if (a.dw)
#pragma unroll
            for (int j = 0; j < DEEP; j++) r[j] = load8<T, VEC>(a.y, a.ldy, max(p[j], 0), p[j] < 0 ? a.n : c, a.n);
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; i++) d[i] = value(g, i);
        if (a.dw)
#pragma unroll
            for (int j = 0; j < DEEP; j++)
                if (p[j] >= 0)
#pragma unroll
                    for (int i = 0; i < 8; i++) dot[j] += d[i] * value(r[j], i);
        asm volatile("" ::: "memory");  // y is read before dy is written: they may be one
#pragma unroll
        for (int j = 0; j < DEEP; j++)
            if (p[j] >= 0) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] = w[j] * d[i];
                store8<T, VEC>(a.dy, a.lddy, p[j], c, a.n, v);
            }
    }
    if (!a.dw) return;
#pragma unroll
    for (int j = 0; j < DEEP; j++) {
#pragma unroll
        for (int o = 16; o; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
        if (lane == 0) sh[j][warp] = dot[j];
    }
    __syncthreads();
    if ((int)threadIdx.x < DEEP && j0 + (int)threadIdx.x < a.k) {
        float v = 0.f;
        for (int i = 0; i < nw; i++) v += sh[threadIdx.x][i];
        a.dw[(long)t * a.k + j0 + threadIdx.x] = v;
    }
}

template <typename... KArgs, typename... Args>
int launch(void (*kernel)(KArgs...), long grid, int threads, size_t smem, cudaStream_t s, const Args &...args)
{
    if (ensure_smem((const void *)kernel, smem) != K3MOE_OK) return K3MOE_ECUDA;
    if (launch_pdl(kernel, dim3((unsigned)grid), dim3((unsigned)threads), smem, s, args...) != cudaSuccess) {
        cudaGetLastError();
        return K3MOE_ECUDA;
    }
    return K3MOE_OK;
}

}  // namespace

// The workspace: the grouped product's part, then the counts of the chunks.
size_t groups_workspace_bytes(int E, long slots)
{
    const size_t chunks = slots <= GR_WHOLE ? 0 : (size_t)((slots + GR_CHUNK - 1) / GR_CHUNK);
    return grouped_matmul_workspace_bytes() + chunks * (size_t)E * sizeof(int32_t);
}

int launch_groups_plan(const k3moe_groups *g, const int32_t *ids, cudaStream_t s)
{
    GroupArgs a = {ids, g->offsets, g->order, g->pos, (int32_t *)((char *)g->workspace + grouped_matmul_workspace_bytes()), g->tokens * g->top_k, g->E, 0};
    a.chunks = (a.S + GR_CHUNK - 1) / GR_CHUNK;
    const size_t smem = (size_t)GR_WARPS * a.E * sizeof(uint16_t);
    if (a.S <= GR_WHOLE) return launch(k3_groups<true, false, false>, 1, GR_THREADS, smem, s, a);
    int st = launch(k3_groups<false, true, false>, a.chunks, GR_THREADS, smem, s, a);
    if (st != K3MOE_OK) return st;
    if (a.chunks <= GR_FEW) return launch(k3_groups<false, false, true>, a.chunks, GR_THREADS, smem, s, a);
    st = launch(k3_groups_scan, 1, GR_THREADS, 0, s, a);
    if (st == K3MOE_OK) st = launch(k3_groups<false, false, false>, a.chunks, GR_THREADS, smem, s, a);
    return st;
}

int launch_combine(const k3moe_combine_desc &d, cudaStream_t s)
{
    CombineArgs a = {};
    a.y = d.y, a.out = d.out, a.ldy = (long)d.ldy, a.ldo = (long)d.ldo, a.w = d.w, a.pos = d.host_groups->pos;
    a.T = d.host_groups->tokens, a.k = d.host_groups->top_k, a.n = d.n, a.rows = a.T * a.k, a.accumulate = d.accumulate;
    a.blocks = (a.n + 1023) / 1024;
    const bool vec = a.n % 8 == 0 && rows16(a.y, a.ldy, d.dtype) && rows16(a.out, a.ldo, d.dtype);
    void (*const kernel)(CombineArgs) = d.dtype == K3MOE_BF16
                                            ? (vec ? k3_combine<uint16_t, true> : k3_combine<uint16_t, false>)
                                            : (vec ? k3_combine<uint32_t, true> : k3_combine<uint32_t, false>);
    return launch(kernel, (long)a.T * a.blocks, 128, 0, s, a);
}

int launch_combine_backward(const k3moe_combine_backward_desc &d, cudaStream_t s)
{
    CombineArgs a = {};
    a.y = d.y, a.dout = d.dout, a.dy = d.dy, a.dw = d.dw, a.ldy = (long)d.ldy, a.ldo = (long)d.lddo, a.lddy = (long)d.lddy;
    a.w = d.w, a.pos = d.host_groups->pos;
    a.T = d.host_groups->tokens, a.k = d.host_groups->top_k, a.n = d.n, a.rows = a.T * a.k;
    const bool vec = a.n % 8 == 0 && rows16(a.dout, a.ldo, d.dtype) && rows16(a.dy, a.lddy, d.dtype) &&
                     (!a.dw || rows16(a.y, a.ldy, d.dtype));
    a.blocks = (a.k + CBB_DEEP - 1) / CBB_DEEP;
    const long ctas = (long)a.T * a.blocks;
    const int threads = ctas <= num_sms() ? 512 : ctas <= 3 * num_sms() ? 256 : 128;
    void (*const kernel)(CombineArgs) = d.dtype == K3MOE_BF16
                                            ? (vec ? k3_combine_backward<uint16_t, true> : k3_combine_backward<uint16_t, false>)
                                            : (vec ? k3_combine_backward<uint32_t, true> : k3_combine_backward<uint32_t, false>);
    return launch(kernel, ctas, std::min(threads, (a.n + 255) / 256 * 32), 0, s, a);
}

}  // namespace k3
