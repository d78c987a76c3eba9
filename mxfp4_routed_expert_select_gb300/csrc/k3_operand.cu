// k3_operand.cu -- MXFP4 product operands: quantisation along the rows and
// along the columns of a matrix from one read, scale atoms of a stored
// matrix, and the values an operand stands for.
//
// A block of 32 values along the reduction axis gets the E8M0 byte
// e = clamp(floor(log2 max|x|) - 2 + 127, 0, 254) and each value the nearest
// E2M1 magnitude of |x| 2^(127-e), ties to the even code, saturating at 6 (the
// OCP Microscaling v1.0 conversion, as k3moe_mx_quantize).  The scaling is a
// power of two, so the conversion instruction's rounding is the only one.
//
// Bound: HBM, and close behind it issue (about ten instructions per value for both
// forms).  A 128 x 128 tile is copied once into shared memory (cp.async, zero past
// the matrix) and converted from there along its rows and along its columns; a
// thread holds a whole block of 32, so that its maximum needs no exchange and its
// codes leave as 16 bytes.  Row pitches and the order of a thread's reads keep the
// banks apart.  Both forms' codes leave in 64-byte runs and their scale bytes as
// whole 512-byte atoms.  4096 x 7168 bf16 both ways: 14.4 us, 6.2 TB/s; four lanes
// per block from registers took 18 to 22.
#include <cuda_runtime.h>

#include <algorithm>

#include "k3_launch.cuh"
#include "k3_operand.cuh"

namespace k3 {
namespace {

constexpr int QT = 128;        // tile rows and columns
// Threads of a CTA: four CTAs of 256 share an SM on bf16 tiles, two of 512 on fp32
// tiles, whose shared memory is twice as large.
template <typename XT>
constexpr int q_threads() { return sizeof(XT) == 2 ? 256 : 512; }

struct QuantArgs {
    const void *x;
    long ld;
    int rows, cols;
    FastDiv tiles_x;
    uint8_t *rcodes, *ratoms;      // row form, or null
    uint8_t *ccodes, *catoms;      // column form, or null
};

// The E8M0 byte of a block whose largest magnitude has bits mb, and the
// factor 2^(127-e) that its values are converted with.
K3_DEV uint32_t block_byte(uint32_t mb, float &inv)
{
    const uint32_t e = (uint32_t)max((int)(mb >> 23) - 2, 0);
    inv = __uint_as_float((254u - e) << 23);
    return mb >= 0x7f800000u ? 255u : e;
}
// Eight scaled values to eight codes, value i in nibble i.
K3_DEV uint32_t codes8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
K3_DEV uint32_t convert8(const float (&v)[8], float inv, uint32_t e)
{
    float a[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        a[i] = v[i], a[i + 1] = v[i + 1];
        scale2(a[i], a[i + 1], inv);
    }
    return e == 255u ? 0u : codes8(a);  // a non-finite block: codes 0
}

// 16 bytes to shared memory.
K3_DEV void copy16(uint32_t dst, const void *p)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(p) : "memory");
}
// The first n of them from p, zero past those.
K3_DEV void copy16(uint32_t dst, const void *p, int n)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(p), "r"(n) : "memory");
}

// Words per tile row in shared memory: 64 words of two bf16 columns or 128 of one
// fp32 column, and 4 that move each row on by 16 bytes of banks.
template <typename XT>
constexpr int tile_pitch() { return QT * (int)sizeof(XT) / 4 + 4; }
constexpr int DQ_U = 2;       // dequantise: 16-value units of a thread in flight
constexpr int CODE_PITCH = 80;  // bytes of one column's staged codes (64, and 16 to spread the banks)
template <typename XT>
constexpr int quant_smem() { return QT * tile_pitch<XT>() * 4 + QT * CODE_PITCH; }

// XT: uint16_t (bf16 bits) or uint32_t (fp32 bits).  VEC: rows are 16-byte
// aligned; else the tile comes in by single elements, neighbouring lanes on
// neighbouring columns.
template <typename XT, bool VEC>
__global__ void __launch_bounds__(q_threads<XT>(), sizeof(XT) == 2 ? 4 : 2) k3_mx_quantize_operand(const QuantArgs a)
{
    constexpr int Q_THREADS = q_threads<XT>();
    extern __shared__ __align__(16) uint32_t tile[];
    __shared__ __align__(16) uint8_t ratom[512], catom[512];
    constexpr int PITCH = tile_pitch<XT>(), ES = (int)sizeof(XT);
    uint8_t *stage = (uint8_t *)(tile + QT * PITCH);
    const int tid = threadIdx.x;
    const int ty = (int)a.tiles_x.div(blockIdx.x), tx = (int)blockIdx.x - ty * (int)a.tiles_x.d;
    const int r0 = ty * QT, c0 = tx * QT;
    const bool do_row = a.rcodes && ty < op_row_tiles(a.rows), do_col = a.ccodes && tx < op_row_tiles(a.cols);
    griddep_wait();
    if (!do_row && !do_col) return;

    if constexpr (VEC) {
        constexpr int CPR = QT * ES / 16, RS = Q_THREADS / CPR;  // 16-byte units per row, rows per pass
        const int u = tid % CPR, r = tid / CPR;
        const XT *p = (const XT *)a.x + (long)(r0 + r) * a.ld + c0 + u * (16 / ES);
        const uint32_t dst = smem_u32(tile + r * PITCH + 4 * u);
        const long pass = RS * a.ld;
        if (r0 + QT <= a.rows && c0 + QT <= a.cols) {
#pragma unroll
            for (int i = 0; i < QT / RS; i++, p += pass) copy16(dst + (uint32_t)(i * RS * PITCH * 4), p);
        } else {
            // counted in elements up to a unit's: the bytes of a row do not fit 32 bits
            const int bytes = min(max(a.cols - c0 - u * (16 / ES), 0), 16 / ES) * ES;
#pragma unroll
            for (int i = 0; i < QT / RS; i++, p += pass) {
                const bool in = bytes > 0 && r0 + r + i * RS < a.rows;
                copy16(dst + (uint32_t)(i * RS * PITCH * 4), in ? p : (const XT *)a.x, in ? bytes : 0);
            }
        }
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    } else {
        const int c = tid & 127, rows = min(QT, a.rows - r0);
        const XT *p = (const XT *)a.x + (long)r0 * a.ld + c0 + c;
        const bool in = c0 + c < a.cols;
#pragma unroll 16
        for (int r = tid >> 7; r < QT; r += Q_THREADS / QT)
            ((XT *)(tile + r * PITCH))[c] = in && r < rows ? p[(long)r * a.ld] : (XT)0;
    }
    __syncthreads();

    if (do_row) {
        // a task is a row's block; four lanes take a row's four.  Their reads go
        // round the block from a quarter that differs between them (ROT words of
        // codes on), so that eight lanes' 16-byte reads fall on distinct banks.
        const long rpitch = op_in_padded(a.cols) / 2;
        const int b = tid & 3, rot = ES == 2 ? 2 * (b >> 1) : b;
        const bool block = c0 + 32 * b < op_in_padded(a.cols);
#pragma unroll
        for (int i = 0; i < QT * 4 / Q_THREADS; i++) {
            const int r = i * (Q_THREADS / 4) + (tid >> 2);
            constexpr int NW = 32 * ES / 4;  // words of a block
            uint32_t q[NW];
            const uint32_t *p = tile + r * PITCH + NW * b;
#pragma unroll
            for (int k = 0; k < NW / 4; k++) {
                // quarters of the block (8 values: ES / 2 reads each), rotated
                const uint4 v = *(const uint4 *)(p + 4 * ((k + rot * (ES / 2)) & (NW / 4 - 1)));
                q[4 * k] = v.x, q[4 * k + 1] = v.y, q[4 * k + 2] = v.z, q[4 * k + 3] = v.w;
            }
            uint32_t top = q[0];
#pragma unroll
            for (int k = 1; k < NW; k++) top = ES == 2 ? absmax2(top, q[k]) : absmax(top, q[k]);
            top = ES == 2 ? max(top & 0x7fff0000u, (top & 0x7fffu) << 16) : top & 0x7fffffffu;
            float inv;
            const uint32_t e = block_byte(top, inv);
            uint32_t w[4];
#pragma unroll
            for (int g = 0; g < 4; g++) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; k++)
                    v[k] = __uint_as_float(ES == 4            ? q[8 * g + k]
                                           : (k & 1) ? (q[4 * g + (k >> 1)] & 0xffff0000u)
                                                     : (q[4 * g + (k >> 1)] << 16));
                w[g] = convert8(v, inv, e);
            }
            // back to the block's order: word g holds quarter (g + rot) mod 4
            const uint4 out = rot == 0   ? make_uint4(w[0], w[1], w[2], w[3])
                              : rot == 1 ? make_uint4(w[3], w[0], w[1], w[2])
                              : rot == 2 ? make_uint4(w[2], w[3], w[0], w[1])
                                         : make_uint4(w[1], w[2], w[3], w[0]);
            const bool in = block && r0 + r < a.rows;
            if (in) *(uint4 *)(a.rcodes + (long)(r0 + r) * rpitch + c0 / 2 + 16 * b) = out;
            ratom[op_atom_byte(r, b)] = in ? (uint8_t)e : 0u;
        }
    }
    if (do_col) {
        // a task is one column's (fp32) or column pair's (bf16) 32 rows
        const int rpad = op_in_padded(a.rows);
        constexpr int COLS = 4 / ES, WPR = QT / COLS;  // columns per task, tasks per row block
#pragma unroll 1
        for (int i = 0; i < 4 * WPR / Q_THREADS; i++) {
            const int task = i * Q_THREADS + tid, wc = task % WPR, rb = task / WPR;  // word column, row block
            uint32_t raw[32], top = 0u;
#pragma unroll
            for (int k = 0; k < 32; k++) {
                raw[k] = tile[(32 * rb + k) * PITCH + wc];
                top = ES == 2 ? absmax2(top, raw[k]) : absmax(top, raw[k]);
            }
#pragma unroll
            for (int h = 0; h < COLS; h++) {
                const int c = COLS * wc + h;
                float inv;
                const uint32_t e = block_byte(
                    ES == 4 ? top & 0x7fffffffu : h ? top & 0x7fff0000u : (top & 0x7fffu) << 16, inv);
                uint32_t w[4];
#pragma unroll
                for (int g = 0; g < 4; g++) {
                    float v[8];
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        const uint32_t x = raw[8 * g + k];
                        v[k] = __uint_as_float(ES == 4 ? x : h ? (x & 0xffff0000u) : (x << 16));
                    }
                    w[g] = convert8(v, inv, e);
                }
                *(uint4 *)(stage + c * CODE_PITCH + 16 * rb) = make_uint4(w[0], w[1], w[2], w[3]);
                catom[op_atom_byte(c, rb)] = c0 + c < a.cols && r0 + 32 * rb < rpad ? (uint8_t)e : 0u;
            }
        }
    }
    __syncthreads();
    if (do_row && tid < 128)
        ((uint32_t *)(a.ratoms + ((long)ty * op_k_atoms(a.cols) + tx) * 512))[tid] = ((const uint32_t *)ratom)[tid];
    if (!do_col) return;
    if (tid >= 128 && tid < 256)
        ((uint32_t *)(a.catoms + ((long)tx * op_k_atoms(a.rows) + ty) * 512))[tid - 128] =
            ((const uint32_t *)catom)[tid - 128];
    const long cpitch = op_in_padded(a.rows) / 2;
#pragma unroll
    for (int i = 0; i < QT * 4 / Q_THREADS; i++) {
        const int k = i * Q_THREADS + tid, c = k >> 2, rb = k & 3;  // four blocks of 16 bytes per column
        if (c0 + c < a.cols && r0 + 32 * rb < op_in_padded(a.rows))
            *(uint4 *)(a.ccodes + (long)(c0 + c) * cpitch + r0 / 2 + 16 * rb) =
                *(const uint4 *)(stage + c * CODE_PITCH + 16 * rb);
    }
}

// Scale atoms of a stored matrix (scales [rows][nb], nb blocks per row): byte
// 255 (a dropped group) becomes 0, so that the group adds at most 6 * 2^-127
// of the other operand's block.  One CTA per atom.
__global__ void __launch_bounds__(128) k3_mx_scale_atoms(const uint8_t *scales, int rows, int nb, int nk, uint8_t *atoms)
{
    griddep_wait();
    const int r = (int)(blockIdx.x / nk) * 128 + threadIdx.x, b0 = 4 * (int)(blockIdx.x % nk);
    uint32_t w = 0u;
    if (r < rows)
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (b0 + i < nb) {
                const uint32_t e = scales[(long)r * nb + b0 + i];
                w |= (e == 255u ? 0u : e) << (8 * i);
            }
    *(uint32_t *)(atoms + (long)blockIdx.x * 512 + op_atom_byte(threadIdx.x, 0)) = w;
}

// 32 bytes to an address of that alignment.
K3_DEV void st32(void *p, const uint32_t *w)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// The values of an operand: units of 16 per thread (two code words, half a block)
// where the rows of y are 16-byte aligned, stored 32 bytes at a time where they are
// 32-byte aligned (wide), else two values per thread, so that a warp's stores stay
// next to each other.  HBM writes bound it, and with units of eight values the
// addresses' instructions did: 4096 x 7168 to bf16 took 10.6 us, 9.2 so (9.7 and 9.5
// with four and one units in flight).
template <typename YT, bool VEC>
__global__ void __launch_bounds__(256) k3_mx_dequantize(const uint8_t *codes, const uint8_t *atoms, int r0,
                                                        uint32_t n, FastDiv upr, int nk, int in, YT *y, long ld,
                                                        bool spread, bool wide)
{
    griddep_wait();
    constexpr int UV = VEC ? 16 : 2, U = VEC ? DQ_U : 4;  // values of a unit, units of a thread in flight
    // a thread's units lie 256 apart (a CTA's are then one run), or, when that would
    // leave SMs idle, a grid apart
    const uint32_t gap = spread ? gridDim.x * 256 : 256;
    for (uint32_t i0 = blockIdx.x * (spread ? 256 : U * 256) + threadIdx.x; i0 < n; i0 += gridDim.x * U * 256) {
        uint2 word[U];
        uint32_t scale[U];
        int r[U], c[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uint32_t i = min(i0 + u * gap, n - 1), q = upr.div(i);
            r[u] = r0 + (int)q, c[u] = (int)(i - q * upr.d) * UV;
            const int b = c[u] >> 5;
            if constexpr (VEC)
                word[u] = ((const uint2 *)codes)[i];
            else
                word[u].x = codes[i];
            scale[u] = atoms[((size_t)(r[u] >> 7) * nk + (b >> 2)) * 512 + op_atom_byte(r[u], b)];
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (i0 + u * gap >= n) break;
            const float s = op_scale(scale[u]);
            YT *o = y + (long)r[u] * ld + c[u];
            const int left = in - c[u];
            if constexpr (VEC) {
                uint32_t h[8], w[16 * sizeof(YT) / 4];
                e2m1x8_to_half2x4(word[u].x, h[0], h[1], h[2], h[3]);
                e2m1x8_to_half2x4(word[u].y, h[4], h[5], h[6], h[7]);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    float2 f = h2f2(h[j]);
                    scale2(f.x, f.y, s);
                    if constexpr (sizeof(YT) == 2) {  // an E2M1 value times a power of two is exact in bf16
                        const __nv_bfloat162 t = __floats2bfloat162_rn(f.x, f.y);
                        w[j] = *(const uint32_t *)&t;
                    } else {
                        w[2 * j] = __float_as_uint(f.x), w[2 * j + 1] = __float_as_uint(f.y);
                    }
                }
                constexpr int NW = sizeof(w) / 4;
                if (left >= 16 && wide) {
#pragma unroll
                    for (int j = 0; j < NW; j += 8) st32((uint32_t *)o + j, w + j);
                } else if (left >= 16) {
#pragma unroll
                    for (int j = 0; j < NW; j += 4) ((uint4 *)o)[j / 4] = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
                } else {
#pragma unroll
                    for (int j = 0; j < 15; j++)
                        if (j < left) {
                            if constexpr (sizeof(YT) == 2)
                                o[j] = (YT)(w[j >> 1] >> (16 * (j & 1)));
                            else
                                o[j] = __uint_as_float(w[j]);
                        }
                }
            } else {
                const float2 f = e2m1x2_to_float2(word[u].x);
#pragma unroll
                for (int j = 0; j < 2; j++)
                    if (j < left) {
                        const float v = (j ? f.y : f.x) * s;
                        if constexpr (sizeof(YT) == 2)
                            o[j] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
                        else
                            o[j] = v;
                    }
            }
        }
    }
}

bool rows_aligned(const void *p, long ld, int es, int n) { return (uintptr_t)p % n == 0 && (ld * es) % n == 0; }

}  // namespace

// x [rows][cols] (row stride ld elements) to the row form (row: rows x cols)
// and / or the column form (col: cols x rows).
int launch_mx_quantize_operand(const void *x, int xdt, int rows, int cols, long ld, const k3moe_mx_operand *row,
                               const k3moe_mx_operand *col, cudaStream_t s)
{
    QuantArgs a = {};
    a.x = x;
    a.ld = ld;
    a.rows = rows;
    a.cols = cols;
    if (row) a.rcodes = row->codes, a.ratoms = row->atoms;
    if (col) a.ccodes = col->codes, a.catoms = col->atoms;
    // the tiles cover every scale atom, the padding ones included
    const int tiles_x = row ? op_k_atoms(cols) : op_row_tiles(cols);
    a.tiles_x = FastDiv((uint32_t)tiles_x);
    const long tiles = (long)tiles_x * (col ? op_k_atoms(rows) : op_row_tiles(rows));
    if (tiles > 0x3fffffffL) return K3MOE_EINVAL;
    const bool vec = rows_aligned(x, ld, xdt == K3MOE_BF16 ? 2 : 4, 16);
    const size_t sm = xdt == K3MOE_BF16 ? quant_smem<uint16_t>() : quant_smem<uint32_t>();
    void (*const kernel)(QuantArgs) =
        xdt == K3MOE_BF16 ? (vec ? k3_mx_quantize_operand<uint16_t, true> : k3_mx_quantize_operand<uint16_t, false>)
                          : (vec ? k3_mx_quantize_operand<uint32_t, true> : k3_mx_quantize_operand<uint32_t, false>);
    if (ensure_smem((const void *)kernel, sm) != K3MOE_OK) return K3MOE_ECUDA;
    return launch_pdl(kernel, dim3((unsigned)tiles), dim3((unsigned)(xdt == K3MOE_BF16 ? q_threads<uint16_t>() : q_threads<uint32_t>())), sm, s, a) == cudaSuccess
               ? K3MOE_OK
               : (cudaGetLastError(), K3MOE_ECUDA);
}

int launch_mx_scale_atoms(const uint8_t *scales, int rows, int in, uint8_t *atoms, cudaStream_t s)
{
    const long n = (long)op_row_tiles(rows) * op_k_atoms(in);
    if (n > 0x7fffffffL) return K3MOE_EINVAL;
    const cudaError_t e = launch_pdl(k3_mx_scale_atoms, dim3((unsigned)n), dim3(128), 0, s, scales, rows,
                                     op_in_padded(in) / 32, op_k_atoms(in), atoms);
    return e == cudaSuccess ? K3MOE_OK : (cudaGetLastError(), K3MOE_ECUDA);
}

template <typename YT, bool VEC>
static int launch_dequantize(const k3moe_mx_operand *op, YT *y, long ld, cudaStream_t s)
{
    // one launch per block of rows whose units fit 31 bits
    const uint32_t upr = (uint32_t)op_in_padded(op->in) / (VEC ? 16 : 2);
    const int rows = (int)std::min<long>(op->rows, std::max<long>(1, (1L << 30) / upr));
    for (int r = 0; r < op->rows; r += rows) {
        const uint32_t n = (uint32_t)std::min(rows, op->rows - r) * upr;
        constexpr uint32_t CTA = 256 * (VEC ? DQ_U : 4);
        const bool spread = n < CTA * (unsigned)num_sms();
        const unsigned grid = (unsigned)std::min<long>(spread ? (n + 255) / 256 : (n + CTA - 1) / CTA, 16L * num_sms());
        if (launch_pdl(k3_mx_dequantize<YT, VEC>, dim3(grid), dim3(256), 0, s,
                       (const uint8_t *)op->codes + (size_t)r * (op_in_padded(op->in) / 2), (const uint8_t *)op->atoms,
                       r, n, FastDiv(upr), op_k_atoms(op->in), op->in, y, ld, spread,
                       rows_aligned(y, ld, (int)sizeof(YT), 32)) != cudaSuccess) {
            cudaGetLastError();
            return K3MOE_ECUDA;
        }
    }
    return K3MOE_OK;
}

int launch_mx_dequantize(const k3moe_mx_operand *op, void *y, int ydt, long ld, cudaStream_t s)
{
    const bool vec = rows_aligned(y, ld, ydt == K3MOE_BF16 ? 2 : 4, 16);
    if (ydt == K3MOE_BF16)
        return vec ? launch_dequantize<uint16_t, true>(op, (uint16_t *)y, ld, s)
                   : launch_dequantize<uint16_t, false>(op, (uint16_t *)y, ld, s);
    return vec ? launch_dequantize<float, true>(op, (float *)y, ld, s)
               : launch_dequantize<float, false>(op, (float *)y, ld, s);
}

}  // namespace k3
