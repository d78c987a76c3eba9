// k3_swiglu.cu -- h = silu(g) * u with g and u kept in 8 bits for the backward
// pass, and the gradients from the kept values.
//
// With s = sigma(g):  h = g s u,   du = dh g s,   dg = dh u s (1 + g (1 - s)).
// The kept copy of 32 values is their e4m3 codes at one power-of-two scale, the
// smallest that brings the largest magnitude to 448 or less (nothing
// saturates); scaling is exact, so the conversion instruction's rounding is the
// only one, at most 2^-4 of the value or 2^-10 of the scale.
//
// Bound: HBM.  One pass each way: forward reads g, u and writes h and 2 * 33/32
// bytes per element; backward reads those and dh and writes dg, du.  A lane
// holds eight values (16-byte accesses in bf16), four lanes a block.
#include <cuda_runtime.h>

#include <algorithm>

#include "k3_launch.cuh"
#include "k3_operand.cuh"

namespace k3 {
namespace {

constexpr int SW_THREADS = 256;
// Runs of chunks per SM, one CTA each.  At 65536 x 1536 bf16 forward + backward took
// 263, 269, 271, 255, 253 and 257 us with 4, 8, 16, 32, 48 and 96, and 270 with the
// CTAs' chunks interleaved over the whole grid.
constexpr int SW_RUNS = 48;

struct SwigluArgs {
    const void *g, *u, *dh;
    void *h, *dg, *du;
    long ldg, ldu, ldh, lddg, lddu, lddh;
    uint8_t *cg, *cu, *sg, *su;  // codes [T][fp] and scale bytes [T][fp / 32] of g and u
    uint32_t n;                  // eight-value chunks of this launch (rows x fp / 8), below 2^31
    uint32_t run;                // chunks of a CTA, a multiple of its threads
    int f;
    FastDiv cpr;                 // chunks per row (fp / 8)
};

// Eight values of a row as loaded.
template <typename T>
struct Raw {
    uint32_t w[2 * sizeof(T)];
};
// The values from column c, zero past f.  VEC: every row of every matrix is
// 16-byte aligned and f a multiple of 8, so a chunk is whole or not there.
template <typename T, bool VEC>
K3_DEV Raw<T> load8(const void *base, long ld, int t, int c, int f)
{
    Raw<T> r;
    constexpr int NW = 2 * sizeof(T);
#pragma unroll
    for (int i = 0; i < NW; i++) r.w[i] = 0u;
    const T *p = (const T *)base + (long)t * ld + c;
    if constexpr (VEC) {
        if (c < f)
#pragma unroll
            for (int i = 0; i < NW / 4; i++)
                asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(r.w[4 * i]), "=r"(r.w[4 * i + 1]), "=r"(r.w[4 * i + 2]), "=r"(r.w[4 * i + 3])
                             : "l"((const uint4 *)p + i));
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (c + i < f) {
                if constexpr (sizeof(T) == 2)
                    r.w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
                else
                    r.w[i] = p[i];
            }
    }
    return r;
}
template <typename T>
K3_DEV float value(const Raw<T> &r, int i)
{
    if constexpr (sizeof(T) == 2)
        return __uint_as_float((i & 1) ? (r.w[i >> 1] & 0xffff0000u) : (r.w[i >> 1] << 16));
    else
        return __uint_as_float(r.w[i]);
}
template <typename T, bool VEC>
K3_DEV void store8(void *base, long ld, int t, int c, int f, const float (&v)[8])
{
    T *p = (T *)base + (long)t * ld + c;
    if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *(const uint32_t *)&b;
        }
        if constexpr (VEC) {
            if (c < f) *(uint4 *)p = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (c + i < f) p[i] = (T)(w[i >> 1] >> (16 * (i & 1)));
        }
    } else {
        if constexpr (VEC) {
            if (c < f) {
                ((float4 *)p)[0] = make_float4(v[0], v[1], v[2], v[3]);
                ((float4 *)p)[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (c + i < f) p[i] = __float_as_uint(v[i]);
        }
    }
}

// The scale byte of the block whose eight values this lane and the three next
// to it hold, and the lane's codes.
template <typename T>
K3_DEV uint2 e4m3x8(const Raw<T> &v, uint32_t &e)
{
    uint32_t mb = absmax8(v.w);
    mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
    mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
    if (mb >= 0x7f800000u) {
        e = 255u;
        return make_uint2(0u, 0u);
    }
    // max = 1.m * 2^(E-127): 2^(E-8-127) holds it up to 1.75 * 2^8 = 448
    e = (uint32_t)max((int)(mb >> 23) - 8 + ((mb & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
    const float inv = __uint_as_float((254u - e) << 23);
    float a[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        a[i] = value(v, i), a[i + 1] = value(v, i + 1);
        scale2(a[i], a[i + 1], inv);
    }
    if (e == 247u)  // at 2^120 a code of 256 would read back as infinity
#pragma unroll
        for (int i = 0; i < 8; i++) a[i] = fminf(fmaxf(a[i], -240.f), 240.f);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        uint16_t q;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(q) : "f"(a[2 * i + 1]), "f"(a[2 * i]));
        w[i] = q;
    }
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}
K3_DEV void from_e4m3x8(uint2 q, uint32_t e, float (&v)[8])
{
    const float s = op_scale(e);
    const uint32_t w[4] = {q.x & 0xffffu, q.x >> 16, q.y & 0xffffu, q.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)w[i]));
        const float2 f = h2f2(h2);
        v[2 * i] = f.x * s;
        v[2 * i + 1] = f.y * s;
    }
}
// sigma(g) for |g| <= 56 (near() below).  bf16 data (2^-8) takes the fast
// exponential: its argument is rounded to 2^-24 of itself, 2^-18 of sigma at -56 and
// 2^-21 at -8; with the full one the forward pass was bound by issue.
template <typename T>
K3_DEV float sigmoid(float g)
{
    return rcp_fast(1.f + (sizeof(T) == 2 ? exp2_fast(-LOG2E * g) : expf(-g)));
}
// Does a block's scale byte say that its gates are at most 448 * 2^-3 = 56?
K3_DEV bool near(uint32_t eg) { return eg <= 124u; }
// Any gate: sigma = q f^2 and 1 - sigma = r with f = e^(-|g|/2) for g < 0 and 1 for
// g >= 0, q = 1 / (1 + e^-|g|).  sigma leaves the normal fp32 numbers below -87 while
// its products with g, u and dh need not, so each factor f goes to one of them.
// Blocks of such gates are rare, and one branch on their scale byte leaves the
// others their time.
struct Sigma {
    float f, q, r;
};
K3_DEV Sigma sigma_far(float g)
{
    const float e = expf(-0.5f * fabsf(g)), q = rcp_fast(1.f + e * e);
    return g < 0.f ? Sigma{e, q, q} : Sigma{1.f, q, e * e * q};
}

// Chunk i of a launch as (row, column); from `end` on the column is f.
struct Place {
    int t, c;
};
K3_DEV Place place(const SwigluArgs &a, uint32_t i, uint32_t end)
{
    const uint32_t t = a.cpr.div(i);
    return {(int)t, i < end ? (int)(i - t * a.cpr.d) * 8 : a.f};
}

// A lane works on one chunk while the next one's loads are in flight.
template <typename T, bool VEC>
__global__ void __launch_bounds__(SW_THREADS) k3_swiglu_forward(const SwigluArgs a)
{
    griddep_wait();
    griddep_launch_dependents();
    // each CTA takes one run of chunks, in steps of its threads
    const uint32_t end = min(a.n, (blockIdx.x + 1) * a.run), step = SW_THREADS;
    // n is a multiple of 4, so the four lanes of a block stay together; lanes
    // past the end take part in the shuffles
    uint32_t i = blockIdx.x * a.run + threadIdx.x;
    Place pl = place(a, i, end);
    Raw<T> g = load8<T, VEC>(a.g, a.ldg, pl.t, pl.c, a.f), u = load8<T, VEC>(a.u, a.ldu, pl.t, pl.c, a.f);
    while ((i & ~31u) < end) {
        const uint32_t in = i + step;
        const Place pn = place(a, in, end);
        const Raw<T> gn = load8<T, VEC>(a.g, a.ldg, pn.t, pn.c, a.f), un = load8<T, VEC>(a.u, a.ldu, pn.t, pn.c, a.f);
        uint32_t eg, eu;
        const uint2 qg = e4m3x8(g, eg), qu = e4m3x8(u, eu);
        if (i < end) {
            float h[8];
            if (near(eg)) {
#pragma unroll
                for (int j = 0; j < 8; j++) h[j] = value(g, j) * sigmoid<T>(value(g, j)) * value(u, j);
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const Sigma s = sigma_far(value(g, j));
                    h[j] = value(g, j) * s.f * s.q * (value(u, j) * s.f);
                }
            }
            store8<T, VEC>(a.h, a.ldh, pl.t, pl.c, a.f, h);
            *(uint2 *)(a.cg + 8 * (size_t)i) = qg;
            *(uint2 *)(a.cu + 8 * (size_t)i) = qu;
            if ((i & 3) == 0) {
                a.sg[i >> 2] = (uint8_t)eg;
                a.su[i >> 2] = (uint8_t)eu;
            }
        }
        i = in, pl = pn, g = gn, u = un;
    }
}

// What the backward pass reads of a chunk.
template <typename T>
struct Kept {
    Raw<T> dh;
    uint2 qg, qu;
    uint32_t eg, eu;
};
template <typename T, bool VEC>
K3_DEV Kept<T> load_kept(const SwigluArgs &a, uint32_t i, uint32_t end, const Place &p)
{
    Kept<T> k;
    k.dh = load8<T, VEC>(a.dh, a.lddh, p.t, p.c, a.f);
    if (i < end) {
        k.qg = *(const uint2 *)(a.cg + 8 * (size_t)i);
        k.qu = *(const uint2 *)(a.cu + 8 * (size_t)i);
        k.eg = a.sg[i >> 2];
        k.eu = a.su[i >> 2];
    } else {
        k.qg = k.qu = make_uint2(0u, 0u);
        k.eg = k.eu = 0u;
    }
    return k;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(SW_THREADS) k3_swiglu_backward(const SwigluArgs a)
{
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t end = min(a.n, (blockIdx.x + 1) * a.run), step = SW_THREADS;
    uint32_t i = blockIdx.x * a.run + threadIdx.x;
    Place pl = place(a, i, end);
    Kept<T> k = load_kept<T, VEC>(a, i, end, pl);
    while (i < end) {
        const uint32_t in = i + step;
        const Place pn = place(a, in, end);
        const Kept<T> kn = load_kept<T, VEC>(a, in, end, pn);
        float g[8], u[8];
        from_e4m3x8(k.qg, k.eg, g);
        from_e4m3x8(k.qu, k.eu, u);
        if (near(k.eg)) {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float s = sigmoid<T>(g[j]), d = value(k.dh, j) * s, gj = g[j];
                g[j] = d * u[j] * (1.f + gj * (1.f - s));
                u[j] = d * gj;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const Sigma s = sigma_far(g[j]);
                const float d = value(k.dh, j) * s.f * s.q, gj = g[j];
                g[j] = d * (u[j] * s.f) * (1.f + gj * s.r);
                u[j] = d * (gj * s.f);
            }
        }
        store8<T, VEC>(a.dg, a.lddg, pl.t, pl.c, a.f, g);
        store8<T, VEC>(a.du, a.lddu, pl.t, pl.c, a.f, u);
        i = in, pl = pn, k = kn;
    }
}

template <typename T, bool VEC>
constexpr auto pick(bool backward)
{
    return backward ? k3_swiglu_backward<T, VEC> : k3_swiglu_forward<T, VEC>;
}

// One launch per 2^31 / 8 chunks (32-bit chunk indices), each a block of rows.
int launch(SwigluArgs a, void *ckpt, int dtype, int T, bool vec, bool backward, cudaStream_t s)
{
    const int fp = op_in_padded(a.f), es = dtype == K3MOE_BF16 ? 2 : 4;
    const uint32_t cpr = (uint32_t)fp / 8;
    a.cpr = FastDiv(cpr);
    a.cg = (uint8_t *)ckpt;
    a.cu = a.cg + (size_t)T * fp;
    a.sg = a.cu + (size_t)T * fp;
    a.su = a.sg + (size_t)T * fp / 32;
    vec = vec && a.f % 8 == 0;
    void (*const kernel)(SwigluArgs) =
        dtype == K3MOE_BF16 ? (vec ? pick<uint16_t, true>(backward) : pick<uint16_t, false>(backward))
                            : (vec ? pick<uint32_t, true>(backward) : pick<uint32_t, false>(backward));
    const int rows = (int)std::min<long>(T, std::max<long>(1, (1L << 28) / cpr));
    for (int t = 0; t < T; t += rows) {
        const int r = std::min(rows, T - t);
        a.n = (uint32_t)r * cpr;
        const uint32_t steps = (a.n + SW_THREADS - 1) / SW_THREADS, ctas = (uint32_t)num_sms() * SW_RUNS;
        a.run = (steps + ctas - 1) / ctas * SW_THREADS;
        const dim3 grid((a.n + a.run - 1) / a.run);
        if (launch_pdl(kernel, grid, dim3(SW_THREADS), 0, s, a) != cudaSuccess) {
            cudaGetLastError();
            return K3MOE_ECUDA;
        }
        auto skip = [&](auto &p, long ld) { p = (decltype(+p))((const char *)p + (size_t)r * ld * es); };
        skip(a.g, a.ldg), skip(a.u, a.ldu), skip(a.dh, a.lddh);
        skip(a.h, a.ldh), skip(a.dg, a.lddg), skip(a.du, a.lddu);
        a.cg += (size_t)r * fp, a.cu += (size_t)r * fp;
        a.sg += (size_t)r * fp / 32, a.su += (size_t)r * fp / 32;
    }
    return K3MOE_OK;
}
bool rows16(const void *p, long ld, int dtype)
{
    return ((uintptr_t)p & 15u) == 0 && ld % (dtype == K3MOE_BF16 ? 8 : 4) == 0;
}

}  // namespace

int launch_swiglu_forward(void *h, long ldh, void *ckpt, const void *g, long ldg, const void *u, long ldu, int dtype,
                          int T, int f, cudaStream_t s)
{
    SwigluArgs a = {};
    a.g = g, a.u = u, a.h = h;
    a.ldg = ldg, a.ldu = ldu, a.ldh = ldh;
    a.f = f;
    const bool vec = rows16(g, ldg, dtype) && rows16(u, ldu, dtype) && rows16(h, ldh, dtype);
    return launch(a, ckpt, dtype, T, vec, false, s);
}
int launch_swiglu_backward(void *dg, long lddg, void *du, long lddu, const void *dh, long lddh, const void *ckpt,
                           int dtype, int T, int f, cudaStream_t s)
{
    SwigluArgs a = {};
    a.dg = dg, a.du = du, a.dh = dh;
    a.lddg = lddg, a.lddu = lddu, a.lddh = lddh;
    a.f = f;
    const bool vec = rows16(dg, lddg, dtype) && rows16(du, lddu, dtype) && rows16(dh, lddh, dtype);
    return launch(a, (void *)ckpt, dtype, T, vec, true, s);
}

}  // namespace k3
