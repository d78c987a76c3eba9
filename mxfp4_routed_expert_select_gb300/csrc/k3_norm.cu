// k3_norm.cu -- root-mean-square norm of a residual stream's rows, forward and
// backward, and the 8-bit rows (k3moe_mx8_rows) by themselves.
//
// r = x + delta, rounded to its type (the stream that the next layer adds to);
// s = 1 / sqrt(mean r^2 + eps);  y = r s gain.  With g = dy gain and xhat = r s
//   dx = dr + s (g - xhat mean(g xhat)),   dgain = sum over rows of dy xhat.
//
// Bound: HBM, one pass each way.  A team of warps holds a row, C chunks of eight
// values a thread, and takes one row after the other, so that its gains (and the
// sums of dgain) stay in registers and the next row's loads are in flight while
// this one's sum is joined.  The column sums of the teams meet in a second small
// kernel, in an order that does not depend on timing.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "k3_e4m3.cuh"
#include "k3_launch.cuh"

namespace k3 {
namespace {

constexpr int NORM_PARTS = 512;    // rows of column sums in the workspace
constexpr int NORM_THREADS = 512;  // of a CTA at most

struct NormArgs {
    const void *x, *delta, *dy, *dr;  // backward: x is r
    void *y, *r, *dx;
    long ldx, ldd, lddy, lddr, ldy, ldr, lddx;
    const float *gain;
    float *rstd, *parts;
    uint8_t *codes, *scales;
    int T, n, warps;  // warps of a team
    float eps, inv_n;
};

// v rounded to the rows' type.
template <typename T>
K3_DEV float rounded(float v)
{
    return sizeof(T) == 2 ? __bfloat162float(__float2bfloat16_rn(v)) : v;
}
K3_DEV float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
K3_DEV float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// A team's warps, its barrier and its slots for partial results.  Two sets of
// slots in turn: a warp that has passed one barrier cannot reach the second next
// one's writes before the others have read.
struct Team {
    int warps, warp, lane, bar;
    float *slots;  // [2][32]
    uint32_t turn;

    template <bool MAX>
    K3_DEV float all(float v)
    {
        v = MAX ? warp_max(v) : warp_sum(v);
        if (warps == 1) return v;
        float *s = slots + (turn++ & 1) * 32;
        if (lane == 0) s[warp] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(warps * 32) : "memory");
        v = lane < warps ? s[lane] : 0.f;
        return MAX ? warp_max(v) : warp_sum(v);
    }
    K3_DEV float sum(float v) { return all<false>(v); }
    K3_DEV float max(float v) { return all<true>(v); }  // of magnitudes
};

// 1 / sqrt(ss / n + eps): the instruction's result (2 ulp) with a Newton step that also
// takes what the division left, since y in 8 bits shows an error of the whole row in
// every code that lies next to a border.  Outside the range the plain result.
// (Sums in two floats and y from unrounded products as well, 4096 x 7168 in 8 bits took
// 52 us instead of 39.)
K3_DEV float fine_rstd(float ss, float n, float inv_n, float eps)
{
    const float q = ss * inv_n, m = q + eps, s = rsqrtf(m);
    if (!(m > 1e-36f && m < 1e36f)) return s;
    const float t = m * s, left = fmaf(-q, n, ss) * inv_n + (eps - (m - q));  // of the true mean + eps above m
    return fmaf(0.5f * s, fmaf(-fmaf(m, s, -t) - left * s, s, fmaf(-t, s, 1.f)), s);
}

// 1 / sqrt(mean v^2 + eps) where the sum of squares left fp32's range or its normal
// numbers while its root need not: the values scaled by a power of two.
template <int C>
K3_DEV float far_rstd(Team &team, const float (&v)[C][8], float ss, float inv_n, float eps)
{
    float m = 0.f;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
        for (int i = 0; i < 8; i++) m = fmaxf(m, fabsf(v[c][i]));
    m = team.max(m);
    if (!(m > 0.f) || m > 3.4028235e38f || ss != ss) return rsqrtf(ss * inv_n + eps);
    const int e = max(-126, min(126, 126 - (int)(__float_as_uint(m) >> 23)));
    const float s = __uint_as_float((uint32_t)(127 + e) << 23);
    float t = 0.f;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
        for (int i = 0; i < 8; i++) t += v[c][i] * s * (v[c][i] * s);
    t = team.sum(t);
    const float es = eps * s * s;
    return es > 1e37f ? rsqrtf(eps) : rsqrtf(t * inv_n + es) * s;
}

// Where this thread's row team stands: first row, rows to the next.
K3_DEV Team make_team(int warps, float (*slots)[64], int &first, int &step)
{
    const int teams = (int)(blockDim.x >> 5) / warps, w = threadIdx.x >> 5, id = w / warps;
    first = (int)blockIdx.x * teams + id;
    step = (int)gridDim.x * teams;
    return Team{warps, w - id * warps, (int)threadIdx.x & 31, 1 + id, slots[id], 0};
}
// A thread's columns.  WIDE (every row 16-byte aligned, n a multiple of 8): C chunks of
// eight, 16-byte accesses.  Otherwise 8 C single values, 32 neighbours to a warp, so
// that rows of any alignment are read and written whole sectors at a time.
template <bool WIDE, int C>
struct Cols {
    int first, step, n;  // of chunk 0 or value 0; to the next chunk or value

    K3_DEV Cols(const Team &team, int n_) : n(n_)
    {
        first = WIDE ? (team.warp * 32 + team.lane) * 8 : team.warp * 32 + team.lane;
        step = WIDE ? team.warps * 256 : team.warps * 32;
    }
    K3_DEV int at(int c, int i) const { return WIDE ? first + c * step + i : first + (c * 8 + i) * step; }
    template <typename T>
    K3_DEV Raw<T> load(const void *base, long ld, int t, int c, bool on) const
    {
        if constexpr (WIDE) return load8<T, true>(base, ld, t, on ? first + c * step : n, n);
        Raw<T> r;
        const T *p = (const T *)base + (long)t * ld;
#pragma unroll
        for (int i = 0; i < (int)(2 * sizeof(T)); i++) r.w[i] = 0u;
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (on && at(c, i) < n) {
                if constexpr (sizeof(T) == 2)
                    r.w[i >> 1] |= (uint32_t)p[at(c, i)] << (16 * (i & 1));
                else
                    r.w[i] = p[at(c, i)];
            }
        return r;
    }
    template <typename T>
    K3_DEV void store(void *base, long ld, int t, int c, const float (&v)[8]) const
    {
        if constexpr (WIDE) {
            store8<T, true>(base, ld, t, first + c * step, n, v);
            return;
        }
        T *p = (T *)base + (long)t * ld;
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (at(c, i) < n) {
                if constexpr (sizeof(T) == 2)
                    p[at(c, i)] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
                else
                    p[at(c, i)] = __float_as_uint(v[i]);
            }
    }
    K3_DEV void load_gain(float (&g)[C][8], const float *gain) const
    {
#pragma unroll
        for (int c = 0; c < C; c++) {
            if (WIDE && gain && ((uintptr_t)gain & 15u) == 0) {
                const int col = min(first + c * step, n - 8);
                const float4 a = *(const float4 *)(gain + col), b = *(const float4 *)(gain + col + 4);
                g[c][0] = a.x, g[c][1] = a.y, g[c][2] = a.z, g[c][3] = a.w;
                g[c][4] = b.x, g[c][5] = b.y, g[c][6] = b.z, g[c][7] = b.w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) g[c][i] = gain && at(c, i) < n ? gain[at(c, i)] : 1.f;
            }
        }
    }
    // Row t in 8 bits; called by whole warps.
    K3_DEV void store_8bit(uint8_t *codes, uint8_t *scales, int t, const float (&v)[C][8]) const
    {
#pragma unroll
        for (int c = 0; c < C; c++) {
            if constexpr (WIDE) {
                Raw<uint32_t> q;
#pragma unroll
                for (int i = 0; i < 8; i++) q.w[i] = first + c * step < n ? __float_as_uint(v[c][i]) : 0u;
                store_mx8(codes, scales, n, t, first + c * step, q);
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) store_mx8_block(codes, scales, n, t, at(c, i), at(c, i) < n ? v[c][i] : 0.f);
            }
        }
    }
};

template <typename T, bool WIDE, int C>
__global__ void __launch_bounds__(NORM_THREADS, C <= 2 && sizeof(T) == 2 ? 2 : 1) k3_norm_forward(const NormArgs a)
{
    __shared__ float slots[8][64];
    griddep_wait();
    griddep_launch_dependents();
    int t, step;
    Team team = make_team(a.warps, slots, t, step);
    const Cols<WIDE, C> cols(team, a.n);
    Raw<T> x[C], d[C];
    auto load = [&](int row) {
#pragma unroll
        for (int c = 0; c < C; c++) {
            x[c] = cols.template load<T>(a.x, a.ldx, row, c, row < a.T);
            if (a.delta) d[c] = cols.template load<T>(a.delta, a.ldd, row, c, row < a.T);
        }
    };
    load(t);
    float gn[C][8];
    cols.load_gain(gn, a.gain);
    for (; t < a.T; t += step) {
        float v[C][8], ss = 0.f;
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int i = 0; i < 8; i++) {
                v[c][i] = value(x[c], i);
                if (a.delta) v[c][i] = rounded<T>(v[c][i] + value(d[c], i));
                ss += v[c][i] * v[c][i];
            }
        load(t + step);
        if (a.r)
#pragma unroll
            for (int c = 0; c < C; c++) cols.template store<T>(a.r, a.ldr, t, c, v[c]);
        ss = team.sum(ss);
        // the sum is exact enough unless it left the normal range, or fell below
        // where eps outweighs what it lost
        float s = fine_rstd(ss, (float)a.n, a.inv_n, a.eps);
        if (!(ss < 1e37f) || (ss < 1e-30f && a.eps < 1e-12f)) s = far_rstd<C>(team, v, ss, a.inv_n, a.eps);
        if (a.rstd && team.warp == 0 && team.lane == 0) a.rstd[t] = s;
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int i = 0; i < 8; i++) v[c][i] = v[c][i] * s * gn[c][i];
        if (a.y)
#pragma unroll
            for (int c = 0; c < C; c++) cols.template store<T>(a.y, a.ldy, t, c, v[c]);
        if (a.codes) cols.store_8bit(a.codes, a.scales, t, v);
    }
}

template <typename T, bool WIDE, int C>
__global__ void __launch_bounds__(NORM_THREADS) k3_norm_backward(const NormArgs a)
{
    __shared__ float slots[8][64];
    griddep_wait();
    griddep_launch_dependents();
    int t, step;
    Team team = make_team(a.warps, slots, t, step);
    const int part = t;
    const Cols<WIDE, C> cols(team, a.n);
    Raw<T> x[C], dy[C], dr[C];
    float s = 0.f;
    auto load = [&](int row) {
#pragma unroll
        for (int c = 0; c < C; c++) {
            x[c] = cols.template load<T>(a.x, a.ldx, row, c, row < a.T);
            dy[c] = cols.template load<T>(a.dy, a.lddy, row, c, row < a.T);
            if (a.dr) dr[c] = cols.template load<T>(a.dr, a.lddr, row, c, row < a.T);
        }
        s = row < a.T ? a.rstd[row] : 0.f;
    };
    load(t);
    float gn[C][8], sum[C][8];
    cols.load_gain(gn, a.gain);
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
        for (int i = 0; i < 8; i++) sum[c][i] = 0.f;
    for (; t < a.T; t += step) {
        float xh[C][8], g[C][8], res[C][8], dot = 0.f;
        const float sc = s;
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int i = 0; i < 8; i++) {
                xh[c][i] = value(x[c], i) * sc;
                const float dv = value(dy[c], i);
                sum[c][i] += dv * xh[c][i];
                g[c][i] = dv * gn[c][i];
                dot += g[c][i] * xh[c][i];
                res[c][i] = a.dr ? value(dr[c], i) : 0.f;
            }
        load(t + step);
        dot = team.sum(dot) * a.inv_n;
#pragma unroll
        for (int c = 0; c < C; c++) {
#pragma unroll
            for (int i = 0; i < 8; i++) g[c][i] = res[c][i] + sc * (g[c][i] - xh[c][i] * dot);
            cols.template store<T>(a.dx, a.lddx, t, c, g[c]);
        }
    }
    if (a.parts)
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (cols.at(c, i) < a.n) a.parts[(long)part * a.n + cols.at(c, i)] = sum[c][i];
}

// dgain[c] (+)= the sum of its column over the parts.  A block takes 32 columns, its
// warps a share of the parts each.
constexpr int NC_WARPS = 32;
__global__ void __launch_bounds__(NC_WARPS * 32) k3_norm_columns(float *dgain, const float *parts, int n, int n_parts, int accumulate)
{
    __shared__ float sh[NC_WARPS][32];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, col = (int)blockIdx.x * 32 + lane;
    float v = 0.f;
    if (col < n)
#pragma unroll 8
        for (int p = w; p < n_parts; p += NC_WARPS) v += parts[(long)p * n + col];
    sh[w][lane] = v;
    __syncthreads();
    if (w == 0 && col < n) {
#pragma unroll
        for (int i = 1; i < NC_WARPS; i++) v += sh[i][lane];
        dgain[col] = accumulate ? dgain[col] + v : v;
    }
}

// ------------------------------------------------------------- 8-bit rows

constexpr int M8_THREADS = 256, M8_U = 2;

struct Mx8Args {
    const void *x;
    void *y;
    long ld;
    uint8_t *codes, *scales;
    uint32_t n;   // eight-value chunks of this launch, rows x cpr, below 2^31
    int in;
    FastDiv cpr;  // chunks per row, ceil128(in) / 8
};

// A thread has U chunks, a CTA's threads apart, all loaded before the first is used
// (4096 x 7168 bf16: quantised in 16.3 us, with one in 18.5; the values in 12.6, 15.2).
template <typename T, bool VEC, int U>
__global__ void __launch_bounds__(M8_THREADS) k3_mx8_quantize(const Mx8Args a)
{
    griddep_wait();
    const uint32_t i0 = blockIdx.x * (M8_THREADS * U) + threadIdx.x;
    Raw<T> v[U];
    int t[U], c[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const uint32_t i = i0 + u * M8_THREADS;
        t[u] = (int)a.cpr.div(i);
        c[u] = i < a.n ? (int)(i - (uint32_t)t[u] * a.cpr.d) * 8 : INT_MAX - 8;
        v[u] = load8<T, VEC>(a.x, a.ld, t[u], c[u], a.in);
    }
#pragma unroll
    for (int u = 0; u < U; u++) store_mx8(a.codes, a.scales, a.in, t[u], c[u], v[u]);
}
template <typename T, bool VEC, int U>
__global__ void __launch_bounds__(M8_THREADS) k3_mx8_dequantize(const Mx8Args a)
{
    griddep_wait();
    const uint32_t i0 = blockIdx.x * (M8_THREADS * U) + threadIdx.x;
    uint2 q[U];
    uint32_t e[U];
    int t[U], c[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const uint32_t i = i0 + u * M8_THREADS;
        t[u] = (int)a.cpr.div(i);
        c[u] = i < a.n ? (int)(i - (uint32_t)t[u] * a.cpr.d) * 8 : a.in;
        if (c[u] < a.in) {
            q[u] = *(const uint2 *)(a.codes + (long)t[u] * op_in_padded(a.in) + c[u]);
            e[u] = a.scales[(long)t[u] * mx8_scale_stride(a.in) + c[u] / 32];
        }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        if (c[u] >= a.in) continue;
        float v[8];
        from_e4m3x8(q[u], e[u], v);
        store8<T, VEC>(a.y, a.ld, t[u], c[u], a.in, v);
    }
}

bool rows16(const void *p, long ld, int dtype)
{
    return ((uintptr_t)p & 15u) == 0 && ld % (dtype == K3MOE_BF16 ? 8 : 4) == 0;
}

// Chunks a thread, by the row's length: few, so that the next row's chunks fit in
// registers beside this one's.
template <typename T, bool WIDE>
auto pick(int c, bool backward) -> void (*)(NormArgs)
{
    if (backward)
        return c == 1 ? k3_norm_backward<T, WIDE, 1> : c == 2 ? k3_norm_backward<T, WIDE, 2>
               : c == 4 ? k3_norm_backward<T, WIDE, 4> : k3_norm_backward<T, WIDE, 8>;
    return c == 1 ? k3_norm_forward<T, WIDE, 1> : c == 2 ? k3_norm_forward<T, WIDE, 2>
           : c == 4 ? k3_norm_forward<T, WIDE, 4> : k3_norm_forward<T, WIDE, 8>;
}
struct NormPlan {
    int c, warps, teams, grid;
};
NormPlan norm_plan(int T, int n)
{
    NormPlan p;
    const int chunks = (n + 7) / 8;
    p.c = chunks <= 128 ? 1 : chunks <= 1024 ? 2 : chunks <= 2048 ? 4 : 8;
    p.warps = (chunks + 32 * p.c - 1) / (32 * p.c);
    p.teams = std::max(1, 8 / p.warps);
    const int threads = p.warps * p.teams * 32;
    p.grid = (int)std::min<long>((T + p.teams - 1L) / p.teams, (long)num_sms() * std::max(1, 1024 / threads));
    return p;
}
int launch_norm(NormArgs a, int dtype, bool wide, bool backward, const NormPlan &p, cudaStream_t s)
{
    a.warps = p.warps;
    a.inv_n = 1.f / (float)a.n;
    wide = wide && a.n % 8 == 0;
    void (*const kernel)(NormArgs) = dtype == K3MOE_BF16
                                         ? (wide ? pick<uint16_t, true>(p.c, backward) : pick<uint16_t, false>(p.c, backward))
                                         : (wide ? pick<uint32_t, true>(p.c, backward) : pick<uint32_t, false>(p.c, backward));
    if (launch_pdl(kernel, dim3((unsigned)p.grid), dim3((unsigned)(p.warps * p.teams * 32)), 0, s, a) != cudaSuccess) {
        cudaGetLastError();
        return K3MOE_ECUDA;
    }
    return K3MOE_OK;
}

template <typename K>
int launch_mx8(K pick_kernel, Mx8Args a, int dtype, int rows, bool vec, cudaStream_t s)
{
    const int es = dtype == K3MOE_BF16 ? 2 : 4;
    const uint32_t cpr = (uint32_t)mx8_scale_stride(a.in) * 4;
    a.cpr = FastDiv(cpr);
    vec = vec && a.in % 8 == 0;
    void (*const kernel)(Mx8Args) = pick_kernel(dtype == K3MOE_BF16, vec);
    const int step = (int)std::min<long>(rows, std::max<long>(1, (1L << 28) / cpr));
    for (int t = 0; t < rows; t += step) {
        const int r = std::min(step, rows - t);
        a.n = (uint32_t)r * cpr;
        const uint32_t each = M8_THREADS * M8_U;
        if (launch_pdl(kernel, dim3((a.n + each - 1) / each), dim3(M8_THREADS), 0, s, a) != cudaSuccess) {
            cudaGetLastError();
            return K3MOE_ECUDA;
        }
        if (a.x) a.x = (const char *)a.x + (size_t)r * a.ld * es;
        if (a.y) a.y = (char *)a.y + (size_t)r * a.ld * es;
        a.codes += (size_t)r * op_in_padded(a.in);
        a.scales += (size_t)r * mx8_scale_stride(a.in);
    }
    return K3MOE_OK;
}

}  // namespace

size_t norm_workspace_bytes(int n) { return (size_t)NORM_PARTS * (size_t)n * sizeof(float); }

int launch_norm_forward(const k3moe_norm_forward_desc &d, cudaStream_t s)
{
    NormArgs a = {};
    a.x = d.x, a.delta = d.delta, a.y = d.y, a.r = d.r;
    a.ldx = (long)d.ldx, a.ldd = (long)d.ldd, a.ldy = (long)d.ldy, a.ldr = (long)d.ldr;
    a.gain = d.gain, a.rstd = d.rstd;
    if (d.host_y8) a.codes = d.host_y8->codes, a.scales = d.host_y8->scales;
    a.T = d.T, a.n = d.n, a.eps = d.eps;
    const bool wide = rows16(d.x, a.ldx, d.dtype) && (!d.delta || rows16(d.delta, a.ldd, d.dtype)) &&
                      (!d.y || rows16(d.y, a.ldy, d.dtype)) && (!d.r || rows16(d.r, a.ldr, d.dtype));
    return launch_norm(a, d.dtype, wide, false, norm_plan(d.T, d.n), s);
}

int launch_norm_backward(const k3moe_norm_backward_desc &d, cudaStream_t s)
{
    NormArgs a = {};
    a.x = d.r, a.dy = d.dy, a.dr = d.dr, a.dx = d.dx;
    a.ldx = (long)d.ldr, a.lddy = (long)d.lddy, a.lddr = (long)d.lddr, a.lddx = (long)d.lddx;
    a.gain = d.gain, a.rstd = (float *)d.rstd;
    a.parts = d.dgain ? (float *)d.workspace : nullptr;
    a.T = d.T, a.n = d.n;
    const bool wide = rows16(d.r, a.ldx, d.dtype) && rows16(d.dy, a.lddy, d.dtype) &&
                      (!d.dr || rows16(d.dr, a.lddr, d.dtype)) && rows16(d.dx, a.lddx, d.dtype);
    NormPlan p = norm_plan(d.T, d.n);
    p.grid = std::min(p.grid, NORM_PARTS / p.teams);
    const int st = launch_norm(a, d.dtype, wide, true, p, s);
    if (st != K3MOE_OK || !d.dgain) return st;
    if (launch_pdl(k3_norm_columns, dim3((unsigned)((d.n + 31) / 32)), dim3(NC_WARPS * 32), 0, s, d.dgain,
                   (const float *)d.workspace, (int)d.n, p.grid * p.teams, d.accumulate ? 1 : 0) != cudaSuccess) {
        cudaGetLastError();
        return K3MOE_ECUDA;
    }
    return K3MOE_OK;
}

int launch_mx8_quantize(const k3moe_mx8_rows *o, const void *x, int dtype, long ld, cudaStream_t s)
{
    Mx8Args a = {};
    a.x = x, a.ld = ld, a.codes = o->codes, a.scales = o->scales, a.in = o->in;
    return launch_mx8(
        [](bool bf16, bool vec) {
            return bf16 ? (vec ? k3_mx8_quantize<uint16_t, true, M8_U> : k3_mx8_quantize<uint16_t, false, M8_U>)
                        : (vec ? k3_mx8_quantize<uint32_t, true, M8_U> : k3_mx8_quantize<uint32_t, false, M8_U>);
        },
        a, dtype, o->rows, rows16(x, ld, dtype), s);
}
int launch_mx8_dequantize(void *y, int dtype, long ld, const k3moe_mx8_rows *o, cudaStream_t s)
{
    Mx8Args a = {};
    a.y = y, a.ld = ld, a.codes = o->codes, a.scales = o->scales, a.in = o->in;
    return launch_mx8(
        [](bool bf16, bool vec) {
            return bf16 ? (vec ? k3_mx8_dequantize<uint16_t, true, M8_U> : k3_mx8_dequantize<uint16_t, false, M8_U>)
                        : (vec ? k3_mx8_dequantize<uint32_t, true, M8_U> : k3_mx8_dequantize<uint32_t, false, M8_U>);
        },
        a, dtype, o->rows, rows16(y, ld, dtype), s);
}

}  // namespace k3
