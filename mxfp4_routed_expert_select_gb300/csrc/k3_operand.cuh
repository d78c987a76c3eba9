// k3_operand.cuh -- layout of an MXFP4 product operand (k3moe_mx_operand).
#pragma once
#include "k3_device.cuh"

namespace k3 {

// Programmatic dependent launches of the kernels that use this header: all start
// as dependents and wait (griddep_wait) before they touch global memory.  Kernels
// that load weights before their own wait (GEMV, shared experts, the batch-1 layer)
// are ordered behind them on the host: each entry point here notes its writes
// (note_weight_writes), and such a kernel is then launched without the attribute.

// Codes: [rows][ceil32(in) / 2] bytes.  Scale bytes: 512-byte atoms of 128
// rows x 4 blocks (128 of the reduction), atom (row tile, k) at
// (row tile) * n_k + k, with n_k even so that a 256-long step always has two;
// byte 16 (r mod 32) + 4 (r / 32 mod 4) + (block mod 4) of its atom, the order
// in which tcgen05.cp takes scales to tensor memory.
__host__ __device__ inline int op_in_padded(int in) { return (in + 31) & ~31; }
__host__ __device__ inline int op_row_tiles(int rows) { return (rows + 127) / 128; }
__host__ __device__ inline int op_k_atoms(int in) { return 2 * ((in + 255) / 256); }
K3_DEV int op_atom_byte(int r, int b) { return 16 * (r & 31) + 4 * ((r >> 5) & 3) + (b & 3); }

// 2^(e-127) of a scale byte; NaN for byte 255 (a block that held a non-finite
// value).
K3_DEV float op_scale(uint32_t e)
{
    return __uint_as_float(e == 255u ? 0x7fc00000u : e == 0u ? 0x00400000u : e << 23);
}

// 2^x (relative error 2^-22) and 1 / x (2^-23), results below 2^-126 as 0: one
// instruction each, where the forms that keep such results take four.
K3_DEV float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
K3_DEV float rcp_fast(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float LOG2E = 1.44269504088896340736f;

// The larger magnitude (its sign is not meaningful); NaN if either is.
K3_DEV uint32_t absmax(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
K3_DEV uint32_t absmax2(uint32_t a, uint32_t b)  // two bf16 values
{
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Bits of the largest magnitude of eight values held as NW words (4: bf16 pairs,
// 8: fp32); 0x7f800000 and above if one is not finite.
template <int NW>
K3_DEV uint32_t absmax8(const uint32_t (&w)[NW])
{
    if constexpr (NW == 4) {
        const uint32_t m = absmax2(absmax2(w[0], w[1]), absmax2(w[2], w[3])) & 0x7fff7fffu;
        return max(m & 0xffff0000u, m << 16);
    } else {
        return absmax(absmax(absmax(w[0], w[1]), absmax(w[2], w[3])), absmax(absmax(w[4], w[5]), absmax(w[6], w[7]))) &
               0x7fffffffu;
    }
}
// (x, y) * s, one instruction.
K3_DEV void scale2(float &x, float &y, float s)
{
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmul.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(s));
}

// Division of n < 2^31 by a divisor fixed per launch: floor(n / d) =
// (n m) >> (32 + s) with m = ceil(2^(32+s) / d), 2^s >= d (m < 2^33: its top bit
// is the addition of n; Granlund and Montgomery, "Division by invariant
// integers using multiplication", 1994).
struct FastDiv {
    uint32_t d, m, s;
    FastDiv() = default;
    explicit FastDiv(uint32_t div) : d(div), m(0), s(0)
    {
        while ((1ull << s) < d) s++;
        m = (uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1);
    }
    K3_DEV uint32_t div(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
};

}  // namespace k3
