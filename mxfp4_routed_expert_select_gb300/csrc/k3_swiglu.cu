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

struct SwigluArgs {
    const void *g, *u, *dh;
    void *h, *dg, *du;
    long ldg, ldu, ldh, lddg, lddu, lddh;
    uint8_t *cg, *cu, *sg, *su;  // codes [T][fp] and scale bytes [T][fp / 32] of g and u
    uint32_t n;                  // eight-value chunks of this launch (rows x fp / 8), below 2^31
    int f;
    FastDiv cpr;                 // chunks per row (fp / 8)
    bool vec;                    // every row of every matrix 16-byte aligned
};

// Eight values of a row from column c, zero past f.
template <typename T>
K3_DEV void load8(const void *base, long ld, int t, int c, int f, bool vec, float (&v)[8])
{
    const T *p = (const T *)base + (long)t * ld + c;
    if (vec && c + 8 <= f) {
        uint32_t w[2 * sizeof(T)];
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; i++) {
            uint4 q;
            asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                         : "l"((const uint4 *)p + i));
            w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
        }
#pragma unroll
        for (int i = 0; i < 8; i++) {
            if constexpr (sizeof(T) == 2)
                v[i] = __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
            else
                v[i] = __uint_as_float(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            v[i] = 0.f;
            if (c + i < f) {
                if constexpr (sizeof(T) == 2)
                    v[i] = __uint_as_float((uint32_t)p[i] << 16);
                else
                    v[i] = p[i];
            }
        }
    }
}
template <typename T>
K3_DEV void store8(void *base, long ld, int t, int c, int f, bool vec, const float (&v)[8])
{
    T *p = (T *)base + (long)t * ld + c;
    if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *(const uint32_t *)&b;
        }
        if (vec && c + 8 <= f)
            *(uint4 *)p = make_uint4(w[0], w[1], w[2], w[3]);
        else
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (c + i < f) p[i] = (T)(w[i >> 1] >> (16 * (i & 1)));
    } else {
        if (vec && c + 8 <= f) {
            ((float4 *)p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            ((float4 *)p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (c + i < f) p[i] = v[i];
    }
}

// The scale byte of the block whose eight values this lane and the three next
// to it hold, and the lane's codes.
K3_DEV uint2 e4m3x8(const float (&v)[8], uint32_t &e)
{
    uint32_t mb = 0u;
#pragma unroll
    for (int i = 0; i < 8; i++) mb = max(mb, __float_as_uint(v[i]) & 0x7fffffffu);
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
    for (int i = 0; i < 8; i++) a[i] = v[i] * inv;
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
K3_DEV float sigmoid(float g) { return __fdividef(1.f, 1.f + expf(-g)); }  // 0 where e^-g overflows

// Two chunks per lane in flight: chunk i and the one a block's threads further.
template <typename T>
__global__ void __launch_bounds__(SW_THREADS) k3_swiglu_forward(const SwigluArgs a)
{
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t step = gridDim.x * 2 * SW_THREADS;
    // n is a multiple of 4, so the four lanes of a block stay together; lanes
    // past the end take part in the shuffles
    for (uint32_t i0 = blockIdx.x * 2 * SW_THREADS + (threadIdx.x & ~31u); i0 < a.n; i0 += step) {
        float g[2][8], u[2][8];
        uint32_t i[2];
        int t[2], c[2];
#pragma unroll
        for (int k = 0; k < 2; k++) {
            i[k] = i0 + k * SW_THREADS + (threadIdx.x & 31);
            t[k] = (int)a.cpr.div(i[k]);
            c[k] = i[k] < a.n ? (int)(i[k] - (uint32_t)t[k] * a.cpr.d) * 8 : a.f;
            load8<T>(a.g, a.ldg, t[k], c[k], a.f, a.vec, g[k]);
            load8<T>(a.u, a.ldu, t[k], c[k], a.f, a.vec, u[k]);
        }
#pragma unroll
        for (int k = 0; k < 2; k++) {
            uint32_t eg, eu;
            const uint2 qg = e4m3x8(g[k], eg), qu = e4m3x8(u[k], eu);
            if (i[k] >= a.n) continue;
#pragma unroll
            for (int j = 0; j < 8; j++) g[k][j] = g[k][j] * sigmoid(g[k][j]) * u[k][j];
            store8<T>(a.h, a.ldh, t[k], c[k], a.f, a.vec, g[k]);
            *(uint2 *)(a.cg + 8 * (size_t)i[k]) = qg;
            *(uint2 *)(a.cu + 8 * (size_t)i[k]) = qu;
            if ((i[k] & 3) == 0) {
                a.sg[i[k] >> 2] = (uint8_t)eg;
                a.su[i[k] >> 2] = (uint8_t)eu;
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(SW_THREADS) k3_swiglu_backward(const SwigluArgs a)
{
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t step = gridDim.x * 2 * SW_THREADS;
    for (uint32_t i0 = blockIdx.x * 2 * SW_THREADS + threadIdx.x; i0 < a.n; i0 += step) {
        float dh[2][8];
        uint2 qg[2], qu[2];
        uint32_t eg[2], eu[2], i[2];
        int t[2], c[2];
#pragma unroll
        for (int k = 0; k < 2; k++) {
            i[k] = i0 + k * SW_THREADS;
            t[k] = (int)a.cpr.div(i[k]);
            c[k] = i[k] < a.n ? (int)(i[k] - (uint32_t)t[k] * a.cpr.d) * 8 : a.f;
            load8<T>(a.dh, a.lddh, t[k], c[k], a.f, a.vec, dh[k]);
            if (i[k] < a.n) {
                qg[k] = *(const uint2 *)(a.cg + 8 * (size_t)i[k]);
                qu[k] = *(const uint2 *)(a.cu + 8 * (size_t)i[k]);
                eg[k] = a.sg[i[k] >> 2];
                eu[k] = a.su[i[k] >> 2];
            }
        }
#pragma unroll
        for (int k = 0; k < 2; k++) {
            if (i[k] >= a.n) continue;
            float g[8], u[8];
            from_e4m3x8(qg[k], eg[k], g);
            from_e4m3x8(qu[k], eu[k], u);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float s = sigmoid(g[j]), d = dh[k][j] * s;
                dh[k][j] = d * g[j];
                g[j] = d * u[j] * (1.f + g[j] * (1.f - s));
            }
            store8<T>(a.dg, a.lddg, t[k], c[k], a.f, a.vec, g);
            store8<T>(a.du, a.lddu, t[k], c[k], a.f, a.vec, dh[k]);
        }
    }
}

// One launch per 2^31 / 8 chunks (32-bit chunk indices), each a block of rows.
int launch(SwigluArgs a, void *ckpt, int dtype, int T, bool backward, cudaStream_t s)
{
    const int fp = op_in_padded(a.f), es = dtype == K3MOE_BF16 ? 2 : 4;
    const uint32_t cpr = (uint32_t)fp / 8;
    a.cpr = FastDiv(cpr);
    a.cg = (uint8_t *)ckpt;
    a.cu = a.cg + (size_t)T * fp;
    a.sg = a.cu + (size_t)T * fp;
    a.su = a.sg + (size_t)T * fp / 32;
    void (*const kernel)(SwigluArgs) = dtype == K3MOE_BF16
                                           ? (backward ? k3_swiglu_backward<uint16_t> : k3_swiglu_forward<uint16_t>)
                                           : (backward ? k3_swiglu_backward<float> : k3_swiglu_forward<float>);
    const int rows = (int)std::min<long>(T, std::max<long>(1, (1L << 28) / cpr));
    for (int t = 0; t < T; t += rows) {
        const int r = std::min(rows, T - t);
        a.n = (uint32_t)r * cpr;
        const dim3 grid((unsigned)std::min<long>(((long)a.n + 2 * SW_THREADS - 1) / (2 * SW_THREADS), 16L * num_sms()));
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
    a.vec = rows16(g, ldg, dtype) && rows16(u, ldu, dtype) && rows16(h, ldh, dtype);
    return launch(a, ckpt, dtype, T, false, s);
}
int launch_swiglu_backward(void *dg, long lddg, void *du, long lddu, const void *dh, long lddh, const void *ckpt,
                           int dtype, int T, int f, cudaStream_t s)
{
    SwigluArgs a = {};
    a.dg = dg, a.du = du, a.dh = dh;
    a.lddg = lddg, a.lddu = lddu, a.lddh = lddh;
    a.f = f;
    a.vec = rows16(dg, lddg, dtype) && rows16(du, lddu, dtype) && rows16(dh, lddh, dtype);
    return launch(a, (void *)ckpt, dtype, T, true, s);
}

}  // namespace k3
