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
// this one's sum is joined.  The column sums of the CTAs meet in a second small
// kernel, in an order that does not depend on timing.  Rows too long for that are read
// twice by a CTA, the second time from L2.
//
// bf16, x, delta, r and y or the backward call's four: 8192 x 4096 43 us (6.2 TB/s) and
// 50, 8192 x 8192 85 (6.3) and 99, 8192 x 32768 385 (5.6) and 602; 4096 x 7168 to 8 bits
// 36 us (with x + delta value by value 40: issue, 28 instructions each, was in the way).
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

// a + b, each sum rounded once to the rows' type.
template <typename T>
K3_DEV Raw<T> sum8(const Raw<T> &a, const Raw<T> &b)
{
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < (int)(2 * sizeof(T)); i++) {
        if constexpr (sizeof(T) == 2) {
            const __nv_bfloat162 v = __hadd2(*(const __nv_bfloat162 *)&a.w[i], *(const __nv_bfloat162 *)&b.w[i]);
            r.w[i] = *(const uint32_t *)&v;
        } else {
            r.w[i] = __float_as_uint(__uint_as_float(a.w[i]) + __uint_as_float(b.w[i]));
        }
    }
    return r;
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

// The sum of eight squares, in pairs.
K3_DEV float squares(const float (&v)[8])
{
    const float a = fmaf(v[1], v[1], v[0] * v[0]), b = fmaf(v[3], v[3], v[2] * v[2]);
    const float c = fmaf(v[5], v[5], v[4] * v[4]), d = fmaf(v[7], v[7], v[6] * v[6]);
    return (a + b) + (c + d);
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

// The sum of squares is exact enough unless it, or its mean with eps, left the normal range,
// or fell below where eps outweighs what it lost.
K3_DEV bool sum_out_of_range(float ss, float eps)
{
    return !(ss < 1e37f && eps < 1e37f) || (ss < 1e-30f && eps < 1e-12f);
}

// 1 / sqrt(mean v^2 + eps) where the sum of squares left fp32's range or its normal
// numbers while its root need not: the values scaled by a power of two.
// each(f) calls f with this thread's values.
template <typename F>
K3_DEV float far_rstd(Team &team, F each, float ss, float inv_n, float eps)
{
    float m = 0.f;
    each([&](float v) { m = fmaxf(m, fabsf(v)); });
    m = team.max(m);
    if (!(m > 0.f) || m > 3.4028235e38f || ss != ss) return rsqrtf(ss * inv_n + eps);
    const int e = max(-126, min(126, 126 - (int)(__float_as_uint(m) >> 23)));
    const float s = __uint_as_float((uint32_t)(127 + e) << 23);
    float t = 0.f;
    each([&](float v) { t += v * s * (v * s); });
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
// A thread's columns.  WIDE (every row 16-byte aligned, n a multiple of 8): chunks of
// eight, 16-byte accesses.  Otherwise a chunk is eight single values, each the neighbour
// of the next lane's, so that rows of any alignment are read and written whole sectors
// at a time.
template <bool WIDE>
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
    K3_DEV void store(void *base, long ld, int t, int c, const Raw<T> &v) const
    {
        T *p = (T *)base + (long)t * ld;
        if constexpr (WIDE) {
            if (first + c * step < n)
#pragma unroll
                for (int i = 0; i < (int)sizeof(T) / 2; i++)
                    ((uint4 *)(p + first + c * step))[i] = make_uint4(v.w[4 * i], v.w[4 * i + 1], v.w[4 * i + 2], v.w[4 * i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (at(c, i) < n) {
                    if constexpr (sizeof(T) == 2)
                        p[at(c, i)] = (T)(v.w[i >> 1] >> (16 * (i & 1)));
                    else
                        p[at(c, i)] = v.w[i];
                }
        }
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
    K3_DEV void load_gain(float (&g)[8], const float *gain, int c) const
    {
        if (WIDE && gain && ((uintptr_t)gain & 15u) == 0) {
            const int col = min(first + c * step, n - 8);
            const float4 a = *(const float4 *)(gain + col), b = *(const float4 *)(gain + col + 4);
            g[0] = a.x, g[1] = a.y, g[2] = a.z, g[3] = a.w;
            g[4] = b.x, g[5] = b.y, g[6] = b.z, g[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) g[i] = gain && at(c, i) < n ? gain[at(c, i)] : 1.f;
        }
    }
    // A chunk of row t in 8 bits; called by whole warps.
    K3_DEV void store_8bit(uint8_t *codes, uint8_t *scales, int t, int c, const float (&v)[8]) const
    {
        if constexpr (WIDE) {
            Raw<uint32_t> q;
#pragma unroll
            for (int i = 0; i < 8; i++) q.w[i] = first + c * step < n ? __float_as_uint(v[i]) : 0u;
            store_mx8(codes, scales, n, t, first + c * step, q);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) store_mx8_block(codes, scales, n, t, at(c, i), at(c, i) < n ? v[i] : 0.f);
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
    const Cols<WIDE> cols(team, a.n);
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
#pragma unroll
    for (int c = 0; c < C; c++) cols.load_gain(gn[c], a.gain, c);
    for (; t < a.T; t += step) {
        float v[C][8], ss = 0.f;
#pragma unroll
        for (int c = 0; c < C; c++) {
            if (a.delta) x[c] = sum8(x[c], d[c]);
            if (a.r) cols.template store<T>(a.r, a.ldr, t, c, x[c]);
#pragma unroll
            for (int i = 0; i < 8; i++) v[c][i] = value(x[c], i);
            ss += squares(v[c]);
        }
        load(t + step);
        ss = team.sum(ss);
        float s = fine_rstd(ss, (float)a.n, a.inv_n, a.eps);
        if (sum_out_of_range(ss, a.eps))
            s = far_rstd(
                team, [&](auto &&take) {
#pragma unroll
                    for (int c = 0; c < C; c++)
#pragma unroll
                        for (int i = 0; i < 8; i++) take(v[c][i]);
                },
                ss, a.inv_n, a.eps);
        if (a.rstd && team.warp == 0 && team.lane == 0) a.rstd[t] = s;
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int i = 0; i < 8; i++) v[c][i] = v[c][i] * s * gn[c][i];
        if (a.y)
#pragma unroll
            for (int c = 0; c < C; c++) cols.template store<T>(a.y, a.ldy, t, c, v[c]);
        if (a.codes)
#pragma unroll
            for (int c = 0; c < C; c++) cols.store_8bit(a.codes, a.scales, t, c, v[c]);
    }
}

template <typename T, bool WIDE, int C>
__global__ void __launch_bounds__(NORM_THREADS) k3_norm_backward(const NormArgs a)
{
    extern __shared__ __align__(16) float sums[];  // [teams][n] where there are several
    __shared__ float slots[8][64];
    griddep_wait();
    griddep_launch_dependents();
    int t, step;
    Team team = make_team(a.warps, slots, t, step);
    const Cols<WIDE> cols(team, a.n);
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
#pragma unroll
    for (int c = 0; c < C; c++) {
        cols.load_gain(gn[c], a.gain, c);
#pragma unroll
        for (int i = 0; i < 8; i++) sum[c][i] = 0.f;
    }
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
    if (!a.parts) return;
    // the CTA's sums: its teams', added in their order
    const int teams = (int)(blockDim.x >> 5) / a.warps;
    float *const part = a.parts + (long)blockIdx.x * a.n, *const mine = teams > 1 ? sums + (team.bar - 1) * a.n : part;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (cols.at(c, i) < a.n) mine[cols.at(c, i)] = sum[c][i];
    if (teams == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < a.n; c += blockDim.x) {
        float v = sums[c];
        for (int i = 1; i < teams; i++) v += sums[i * a.n + c];
        part[c] = v;
    }
}

// Rows that do not fit in registers: a CTA holds one after the other and reads each
// twice, the second time from L2, U chunks a thread at a time (a load does not pass the
// stores before it).
constexpr int LONG_THREADS = 512, LONG_CTAS = 2;  // of an SM

K3_DEV Team long_team(float *slots)
{
    return Team{LONG_THREADS / 32, (int)threadIdx.x >> 5, (int)threadIdx.x & 31, 1, slots, 0};
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(LONG_THREADS, LONG_CTAS) k3_norm_long_forward(const NormArgs a)
{
    constexpr int U = WIDE && sizeof(T) == 2 ? 2 : 1;
    __shared__ float slots[64];
    griddep_wait();
    griddep_launch_dependents();
    Team team = long_team(slots);
    const Cols<WIDE> cols(team, a.n);
    const int chunks = (a.n + LONG_THREADS * 8 - 1) / (LONG_THREADS * 8);
    for (int t = (int)blockIdx.x; t < a.T; t += (int)gridDim.x) {
        // f(c, r) with the chunks of r, read as such (stored) or made from x and delta
        auto row = [&](bool stored, auto &&f) {
#pragma unroll U == 2 || !WIDE ? 1 : 2
            for (int c0 = 0; c0 < chunks; c0 += U) {
                Raw<T> x[U], d[U];
#pragma unroll
                for (int u = 0; u < U; u++) {
                    x[u] = cols.template load<T>(stored ? a.r : a.x, stored ? a.ldr : a.ldx, t, c0 + u, true);
                    if (a.delta && !stored) d[u] = cols.template load<T>(a.delta, a.ldd, t, c0 + u, true);
                }
#pragma unroll
                for (int u = 0; u < U; u++) {
                    if (a.delta && !stored) x[u] = sum8(x[u], d[u]);
                    f(c0 + u, x[u]);
                }
            }
        };
        float ss = 0.f;
        row(false, [&](int c, const Raw<T> &r) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = value(r, i);
            ss += squares(v);
            if (a.r) cols.template store<T>(a.r, a.ldr, t, c, r);
        });
        asm volatile("" ::: "memory");  // r, which may lie over x, is stored before it is read again
        const bool stored = a.r != nullptr;
        ss = team.sum(ss);
        float s = fine_rstd(ss, (float)a.n, a.inv_n, a.eps);
        if (sum_out_of_range(ss, a.eps))
            s = far_rstd(
                team, [&](auto &&take) {
                    row(stored, [&](int, const Raw<T> &r) {
#pragma unroll
                        for (int i = 0; i < 8; i++) take(value(r, i));
                    });
                },
                ss, a.inv_n, a.eps);
        if (a.rstd && threadIdx.x == 0) a.rstd[t] = s;
        row(stored, [&](int c, const Raw<T> &r) {
            float g[8], v[8];
            cols.load_gain(g, a.gain, c);
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = value(r, i) * s * g[i];
            if (a.y) cols.template store<T>(a.y, a.ldy, t, c, v);
            if (a.codes) cols.store_8bit(a.codes, a.scales, t, c, v);
        });
    }
}

// The sums of dgain stay in shared memory, [n].
template <typename T, bool WIDE>
__global__ void __launch_bounds__(LONG_THREADS, LONG_CTAS) k3_norm_long_backward(const NormArgs a)
{
    constexpr int U = WIDE ? 8 / sizeof(T) : 1, V = WIDE ? 4 / sizeof(T) : 1;
    extern __shared__ __align__(16) float sums[];
    __shared__ float slots[64];
    griddep_wait();
    griddep_launch_dependents();
    Team team = long_team(slots);
    const Cols<WIDE> cols(team, a.n);
    const int chunks = (a.n + LONG_THREADS * 8 - 1) / (LONG_THREADS * 8);
    if (a.parts)
        for (int c = 0; c < chunks; c++)
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (cols.at(c, i) < a.n) sums[cols.at(c, i)] = 0.f;
    for (int t = (int)blockIdx.x; t < a.T; t += (int)gridDim.x) {
        const float s = a.rstd[t];
        float dot = 0.f;
#pragma unroll WIDE ? 1 : 4
        for (int c0 = 0; c0 < chunks; c0 += U) {
            Raw<T> x[U], dy[U];
#pragma unroll
            for (int u = 0; u < U; u++) {
                x[u] = cols.template load<T>(a.x, a.ldx, t, c0 + u, true);
                dy[u] = cols.template load<T>(a.dy, a.lddy, t, c0 + u, true);
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                float g[8];
                cols.load_gain(g, a.gain, c0 + u);
#pragma unroll
                for (int i = 0; i < 8; i++) dot += value(dy[u], i) * g[i] * (value(x[u], i) * s);
            }
        }
        dot = team.sum(dot) * a.inv_n;
#pragma unroll WIDE ? 1 : 2
        for (int c0 = 0; c0 < chunks; c0 += V) {
            Raw<T> x[V], dy[V], dr[V];
#pragma unroll
            for (int u = 0; u < V; u++) {
                x[u] = cols.template load<T>(a.x, a.ldx, t, c0 + u, true);
                dy[u] = cols.template load<T>(a.dy, a.lddy, t, c0 + u, true);
                dr[u] = Raw<T>{};
                if (a.dr) dr[u] = cols.template load<T>(a.dr, a.lddr, t, c0 + u, true);
            }
#pragma unroll
            for (int u = 0; u < V; u++) {
                const int c = c0 + u;
                float g[8], add[8];
                cols.load_gain(g, a.gain, c);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float xh = value(x[u], i) * s, dv = value(dy[u], i);
                    g[i] = value(dr[u], i) + s * (dv * g[i] - xh * dot);
                    add[i] = dv * xh;
                }
                cols.template store<T>(a.dx, a.lddx, t, c, g);
                if (!a.parts) continue;
                if constexpr (WIDE) {
                    if (cols.at(c, 0) >= a.n) continue;
                    float4 *const p = (float4 *)(sums + cols.at(c, 0));
                    const float4 q = p[0], r = p[1];
                    p[0] = make_float4(q.x + add[0], q.y + add[1], q.z + add[2], q.w + add[3]);
                    p[1] = make_float4(r.x + add[4], r.y + add[5], r.z + add[6], r.w + add[7]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        if (cols.at(c, i) < a.n) sums[cols.at(c, i)] += add[i];
                }
            }
        }
    }
    if (a.parts)
        for (int c = 0; c < chunks; c++)
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (cols.at(c, i) < a.n) a.parts[(long)blockIdx.x * a.n + cols.at(c, i)] = sums[cols.at(c, i)];
}

// dgain[c] (+)= the sum of its column over the parts.  A block takes 32 columns, its
// warps a share of the parts each; the shares are joined pair by pair.
constexpr int NC_WARPS = 32;
__global__ void __launch_bounds__(NC_WARPS * 32) k3_norm_columns(float *dgain, const float *parts, int n, int n_parts, int accumulate)
{
    __shared__ float sh[NC_WARPS][33];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, col = (int)blockIdx.x * 32 + lane;
    float v = 0.f;
    if (col < n)
#pragma unroll 8
        for (int p = w; p < n_parts; p += NC_WARPS) v += parts[(long)p * n + col];
    sh[w][lane] = v;
    __syncthreads();
    const int mine = (int)blockIdx.x * 32 + w;  // the column that this warp joins
    v = warp_sum(sh[lane][w]);
    if (lane == 0 && mine < n) dgain[mine] = accumulate ? dgain[mine] + v : v;
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

// Chunks a thread: few, so that the next row's fit in registers beside this one's; of
// unaligned rows, whose values come one by one, one.  Measured in us on 8192 rows, forward
// and backward: bf16 4096 wide with one chunk a thread 44 and 61, two 47 and 55, four 44
// and (with spills) 396; 8192 wide two 89 and 98, four 85, long 102 and 136; 16384 wide four
// 166 and 2340, long 190 and 252.  fp32 1024 wide one 27 and 24, two 22 and 33; 8192 wide
// two 176 and 253, long 183 and 235.  bf16 4093 wide, unaligned, one 154 and 220, long 88 and
// 96; 2045 wide one 74 and 121, long 79 and 85, but on 256 rows one 4.0 and 6.5.
struct NormPlan {
    int c, warps, teams, grid;  // c: chunks a thread, 0 for the kernels of long rows
};
NormPlan norm_plan(int T, int n, int dtype, bool wide, bool backward)
{
    NormPlan p;
    const int chunks = (n + 7) / 8;
    const bool two_bytes = dtype == K3MOE_BF16;
    if (!wide)
        p.c = chunks <= 256 ? 1 : 0;
    else if (two_bytes)
        p.c = backward ? (chunks <= 128 ? 1 : chunks <= 1024 ? 2 : 0) : (chunks <= 512 ? 1 : chunks <= 2048 ? 4 : 0);
    else
        p.c = backward ? (chunks <= 512 ? 1 : 0) : (chunks <= 32 ? 1 : chunks <= 1024 ? 2 : 0);
    if (!p.c) {
        p.warps = LONG_THREADS / 32, p.teams = 1;
        p.grid = std::min(T, num_sms() * LONG_CTAS);
        return p;
    }
    p.warps = (chunks + 32 * p.c - 1) / (32 * p.c);
    p.teams = std::max(1, 8 / p.warps);
    const int threads = p.warps * p.teams * 32;
    // backward no more CTAs than run at once, by registers (76 a thread, 93 to 128 the
    // others): 8192 x 4096 bf16 50 us, with twice as many 56; 8192 x 1024 15.0 with 768
    // threads an SM, 17.7 with 512, 18.0 with 1024
    const int at_once = !backward ? 1024 : two_bytes && wide && p.c == 1 ? 768 : 512;
    p.grid = (int)std::min<long>((T + p.teams - 1L) / p.teams, (long)num_sms() * std::max(1, at_once / threads));
    return p;
}
template <typename T>
auto pick(int c, bool wide, bool backward) -> void (*)(NormArgs)
{
    if (backward)
        return c == 0 ? (wide ? k3_norm_long_backward<T, true> : k3_norm_long_backward<T, false>)
               : !wide ? k3_norm_backward<T, false, 1>
               : c == 1 ? k3_norm_backward<T, true, 1> : k3_norm_backward<T, true, sizeof(T) == 2 ? 2 : 1>;
    if (c == 0) return wide ? k3_norm_long_forward<T, true> : k3_norm_long_forward<T, false>;
    return !wide ? k3_norm_forward<T, false, 1> : c == 1 ? k3_norm_forward<T, true, 1>
           : k3_norm_forward<T, true, sizeof(T) == 2 ? 4 : 2>;
}
int launch_norm(NormArgs a, int dtype, bool wide, bool backward, const NormPlan &p, cudaStream_t s)
{
    a.warps = p.warps;
    a.inv_n = 1.f / (float)a.n;
    void (*const kernel)(NormArgs) =
        dtype == K3MOE_BF16 ? pick<uint16_t>(p.c, wide, backward) : pick<uint32_t>(p.c, wide, backward);
    const size_t smem = a.parts && (p.c == 0 || p.teams > 1) ? (size_t)p.teams * a.n * sizeof(float) : 0;
    if (smem && ensure_smem((const void *)kernel, smem) != K3MOE_OK) return K3MOE_ECUDA;
    if (launch_pdl(kernel, dim3((unsigned)p.grid), dim3((unsigned)(p.warps * p.teams * 32)), smem, s, a) != cudaSuccess) {
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
    const bool wide = d.n % 8 == 0 && rows16(d.x, a.ldx, d.dtype) && (!d.delta || rows16(d.delta, a.ldd, d.dtype)) &&
                      (!d.y || rows16(d.y, a.ldy, d.dtype)) && (!d.r || rows16(d.r, a.ldr, d.dtype));
    return launch_norm(a, d.dtype, wide, false, norm_plan(d.T, d.n, d.dtype, wide, false), s);
}

int launch_norm_backward(const k3moe_norm_backward_desc &d, cudaStream_t s)
{
    NormArgs a = {};
    a.x = d.r, a.dy = d.dy, a.dr = d.dr, a.dx = d.dx;
    a.ldx = (long)d.ldr, a.lddy = (long)d.lddy, a.lddr = (long)d.lddr, a.lddx = (long)d.lddx;
    a.gain = d.gain, a.rstd = (float *)d.rstd;
    a.parts = d.dgain ? (float *)d.workspace : nullptr;
    a.T = d.T, a.n = d.n;
    const bool wide = d.n % 8 == 0 && rows16(d.r, a.ldx, d.dtype) && rows16(d.dy, a.lddy, d.dtype) &&
                      (!d.dr || rows16(d.dr, a.lddr, d.dtype)) && rows16(d.dx, a.lddx, d.dtype);
    NormPlan p = norm_plan(d.T, d.n, d.dtype, wide, true);
    p.grid = std::min(p.grid, NORM_PARTS);
    const int st = launch_norm(a, d.dtype, wide, true, p, s);
    if (st != K3MOE_OK || !d.dgain) return st;
    if (launch_pdl(k3_norm_columns, dim3((unsigned)((d.n + 31) / 32)), dim3(NC_WARPS * 32), 0, s, d.dgain,
                   (const float *)d.workspace, (int)d.n, p.grid, d.accumulate ? 1 : 0) != cudaSuccess) {
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
