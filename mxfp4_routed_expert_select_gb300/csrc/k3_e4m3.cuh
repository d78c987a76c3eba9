// k3_e4m3.cuh -- rows of fp32 or bf16 values eight at a time, and blocks of 32 of
// them as e4m3 codes with one power-of-two scale (the SwiGLU checkpoint, the 8-bit
// rows of the grouped products).
#pragma once
#include "k3_operand.cuh"

namespace k3 {

// Rows that are all 16-byte aligned.
inline bool rows16(const void *p, long ld, int dtype)
{
    return ((uintptr_t)p & 15u) == 0 && ld % (dtype == K3MOE_BF16 ? 8 : 4) == 0;
}

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

// The scale byte of a block by its largest magnitude (finite), and 1 / scale.
K3_DEV float scale_of_block(uint32_t mb, uint32_t &e)
{
    // max = 1.m * 2^(E-127): 2^(E-8-127) holds it up to 1.75 * 2^8 = 448
    e = (uint32_t)max((int)(mb >> 23) - 8 + ((mb & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
    return __uint_as_float((254u - e) << 23);
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
    const float inv = scale_of_block(mb, e);
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

// An 8-bit row matrix (k3moe_mx8_rows): codes [rows][ceil32(in)], scale bytes
// [rows][4 ceil(in / 128)], so that the four bytes of 128 values are one word; the
// codes and bytes past `in` are zero.
__host__ __device__ inline int mx8_scale_stride(int in) { return 4 * ((in + 127) / 128); }

// Eight values of row t from column c (zero past `in`) into such a matrix.  Called by
// a whole warp whose lanes hold consecutive chunks, the first of a 128-value run in
// lane 0 or 16; columns past the matrix store nothing.
template <typename T>
K3_DEV void store_mx8(uint8_t *codes, uint8_t *scales, int in, int t, int c, const Raw<T> &v)
{
    uint32_t e;
    const uint2 q = e4m3x8(v, e);
    const int fp = op_in_padded(in), ss = mx8_scale_stride(in);
    if (c < fp) *(uint2 *)(codes + (long)t * fp + c) = q;
    const int lane = threadIdx.x & 31;
    uint32_t w = e << (8 * ((lane >> 2) & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    w |= __shfl_xor_sync(0xffffffffu, w, 8);
    if ((lane & 15) == 0 && c / 32 < ss) *(uint32_t *)(scales + (long)t * ss + c / 32) = w;
}

// One value a lane, a whole warp on one block of 32: lane 0's column is a multiple of 32.
K3_DEV void store_mx8_block(uint8_t *codes, uint8_t *scales, int in, int t, int c, float v)
{
    const uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu);
    const int fp = op_in_padded(in), ss = mx8_scale_stride(in);
    uint32_t e = 255u;
    uint16_t q = 0;
    if (mb < 0x7f800000u) {
        float a = scale_of_block(mb, e) * v;
        if (e == 247u) a = fminf(fmaxf(a, -240.f), 240.f);
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(q) : "f"(0.f), "f"(a));
    }
    if (c < fp) codes[(long)t * fp + c] = (uint8_t)q;
    if ((c & 31) == 0 && c / 32 < ss) scales[(long)t * ss + c / 32] = (uint8_t)e;
}

}  // namespace k3
