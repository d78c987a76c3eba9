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
// Bound: HBM.  A 128 x 128 tile is read once, converted along its rows from
// registers (four lanes hold a block; two shuffles find its maximum) and, for
// the column form, along its columns from shared memory, where a lane walks
// the 32 values of a block without bank conflicts.  Both forms' codes leave as
// 64-byte runs and their scale bytes as whole 512-byte atoms.
#include <cuda_runtime.h>

#include <algorithm>

#include "k3_launch.cuh"
#include "k3_operand.cuh"

namespace k3 {
namespace {

constexpr int QT = 128;        // tile rows and columns
constexpr int Q_THREADS = 256;

struct QuantArgs {
    const void *x;
    long ld;
    int rows, cols, tiles_x, tiles;
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

// Sixteen bytes that this kernel reads once.  Not the read-only (nc) path: as
// a programmatic dependent the kernel may have started before its input was
// written.
K3_DEV uint4 ld_once16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Eight values of a row.
template <typename XT>
struct alignas(16) Chunk {
    uint32_t w[2 * sizeof(XT)];
};
// From p (16-byte aligned if whole), the first `cols` of them, zero past those.
template <typename XT>
K3_DEV Chunk<XT> load_chunk(const XT *p, bool whole, int cols)
{
    Chunk<XT> o;
    constexpr int NW = 2 * sizeof(XT);
    if (whole) {
#pragma unroll
        for (int i = 0; i < NW / 4; i++) {
            const uint4 q = ld_once16((const uint4 *)p + i);
            o.w[4 * i] = q.x, o.w[4 * i + 1] = q.y, o.w[4 * i + 2] = q.z, o.w[4 * i + 3] = q.w;
        }
        return o;
    }
#pragma unroll
    for (int i = 0; i < NW; i++) o.w[i] = 0u;
    if (cols > 0) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < cols) {
                if constexpr (sizeof(XT) == 2)
                    o.w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
                else
                    o.w[i] = p[i];
            }
    }
    return o;
}
template <typename XT>
K3_DEV void chunk_values(const Chunk<XT> &q, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i++) {
        if constexpr (sizeof(XT) == 2)
            v[i] = __uint_as_float((i & 1) ? (q.w[i >> 1] & 0xffff0000u) : (q.w[i >> 1] << 16));
        else
            v[i] = __uint_as_float(q.w[i]);
    }
}

// Words per tile row in shared memory.  bf16: 64 words of two columns; fp32:
// 128 words.  The column pass reads 32 consecutive words of one row per warp,
// and the 16-byte stores of the first pass fall on distinct banks too.
template <typename XT>
constexpr int tile_pitch() { return sizeof(XT) == 2 ? 64 : 128; }
constexpr int CODE_PITCH = 80;  // bytes of one column's staged codes (64, and 16 to spread the banks)
template <typename XT>
constexpr int quant_smem() { return QT * tile_pitch<XT>() * 4 + QT * CODE_PITCH; }

// XT: uint16_t (bf16 bits) or uint32_t (fp32 bits).  VEC: rows are 16-byte
// aligned; else the tile comes in by single elements, neighbouring lanes on
// neighbouring columns, through shared memory.
template <typename XT, bool VEC>
__global__ void __launch_bounds__(Q_THREADS, 3) k3_mx_quantize_operand(const QuantArgs a)
{
    extern __shared__ __align__(16) uint32_t tile[];
    __shared__ __align__(16) uint8_t ratom[512], catom[512];
    constexpr int PITCH = tile_pitch<XT>();
    constexpr int NIT = QT * (QT / 8) / Q_THREADS;       // chunks per thread
    constexpr int NB = sizeof(XT) == 2 ? NIT : NIT / 2;  // of them in flight at a time
    uint8_t *stage = (uint8_t *)(tile + QT * PITCH);
    const int tid = threadIdx.x, rt = tid >> 4, cc = tid & 15;  // chunk j: row rt + 16 j, columns 8 cc ..
    uint32_t *pt = tile + rt * PITCH + cc * 2 * (int)sizeof(XT);
    const long rpitch = op_in_padded(a.cols) / 2;
    const int rpad = op_in_padded(a.rows);
    Chunk<XT> q[NB];
    // chunks j0 .. j0 + NB - 1 of tile t
    auto load = [&](int t, int j0) {
        const int r = (t / a.tiles_x) * QT + rt + 16 * j0, c = (t % a.tiles_x) * QT + 8 * cc;
        const int rows_left = a.rows - r, cols_left = a.cols - c;
        const XT *px = (const XT *)a.x + (long)r * a.ld + c;
#pragma unroll
        for (int j = 0; j < NB; j++, px += 16 * a.ld) {
            const bool row = 16 * j < rows_left;
            q[j] = load_chunk<XT>(px, row && cols_left >= 8, row ? cols_left : 0);
        }
    };
    griddep_launch_dependents();
    griddep_wait();

    if (VEC) load(blockIdx.x, 0);
    for (int t = blockIdx.x; t < a.tiles; t += gridDim.x) {
        const int tx = t % a.tiles_x, ty = t / a.tiles_x, r0 = ty * QT, c0 = tx * QT;
        const bool do_row = a.rcodes && ty < op_row_tiles(a.rows), do_col = a.ccodes && tx < op_row_tiles(a.cols);
        if constexpr (!VEC) {
            const int c = tid & 127, rows = min(QT, a.rows - r0);
            const XT *p = (const XT *)a.x + (long)r0 * a.ld + c0 + c;
            const bool in = c0 + c < a.cols;
#pragma unroll 16
            for (int r = tid >> 7; r < QT; r += Q_THREADS / QT)
                ((XT *)(tile + r * PITCH))[c] = in && r < rows ? p[(long)r * a.ld] : (XT)0;
            __syncthreads();
        }
        const int rows_left = a.rows - r0 - rt;
        const bool code_cols = c0 + 8 * cc < op_in_padded(a.cols);
        uint8_t *pc = a.rcodes + (long)(r0 + rt) * rpitch + c0 / 2 + 4 * cc;
#pragma unroll
        for (int it0 = 0; it0 < NIT; it0 += NB) {
            if constexpr (VEC) {
                if (it0) load(t, it0);
            } else if (do_row) {
#pragma unroll
                for (int j = 0; j < NB; j++) q[j] = *(const Chunk<XT> *)(pt + 16 * (it0 + j) * PITCH);
            }
#pragma unroll
            for (int j = 0; j < NB; j++, pc += 16 * rpitch) {
                const int i16 = it0 + j;  // row rt + 16 i16
                if (VEC && do_col) {
#pragma unroll
                    for (int i = 0; i < (int)sizeof(XT) / 2; i++)
                        *(uint4 *)(pt + 16 * i16 * PITCH + 4 * i) =
                            make_uint4(q[j].w[4 * i], q[j].w[4 * i + 1], q[j].w[4 * i + 2], q[j].w[4 * i + 3]);
                }
                if (do_row) {
                    float v[8];
                    chunk_values<XT>(q[j], v);
                    uint32_t mb = absmax8(q[j].w);
                    mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
                    mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
                    float inv;
                    const uint32_t e = block_byte(mb, inv);
                    const uint32_t w = convert8(v, inv, e);
                    const bool in = 16 * i16 < rows_left && code_cols;
                    if (in) *(uint32_t *)pc = w;
                    if ((cc & 3) == 0) ratom[16 * rt + (cc >> 2) + op_atom_byte(16 * i16, 0)] = in ? (uint8_t)e : 0u;
                }
            }
        }
        // the next tile's loads are in flight during this one's column pass
        if (VEC && t + (int)gridDim.x < a.tiles) load(t + gridDim.x, 0);
        __syncthreads();
        if (do_row && tid < 128)
            ((uint32_t *)(a.ratoms + ((long)ty * op_k_atoms(a.cols) + tx) * 512))[tid] = ((const uint32_t *)ratom)[tid];
        if (do_col) {
            // a task is one column's (fp32) or column pair's (bf16) 32 rows
            constexpr int COLS = sizeof(XT) == 2 ? 2 : 1;   // columns per task
            constexpr int WPR = QT / COLS;                  // tasks per row block
#pragma unroll
            for (int i = 0; i < 4 * WPR / Q_THREADS; i++) {
                const int task = i * Q_THREADS + tid, wc = task % WPR, rb = task / WPR;  // word column, row block
                uint32_t raw[32], top = 0u;
#pragma unroll
                for (int k = 0; k < 32; k++) {
                    raw[k] = tile[(32 * rb + k) * PITCH + wc];
                    top = sizeof(XT) == 2 ? absmax2(top, raw[k]) : absmax(top, raw[k]);
                }
#pragma unroll
                for (int h = 0; h < COLS; h++) {
                    const int c = COLS * wc + h;
                    const uint32_t mb =
                        sizeof(XT) == 4 ? top & 0x7fffffffu : h ? top & 0x7fff0000u : (top & 0x7fffu) << 16;
                    float inv;
                    const uint32_t e = block_byte(mb, inv);
                    uint32_t w[4];
#pragma unroll
                    for (int g = 0; g < 4; g++) {
                        float v[8];
#pragma unroll
                        for (int k = 0; k < 8; k++) {
                            const uint32_t x = raw[8 * g + k];
                            v[k] = __uint_as_float(sizeof(XT) == 4 ? x : h ? (x & 0xffff0000u) : (x << 16));
                        }
                        w[g] = convert8(v, inv, e);
                    }
                    *(uint4 *)(stage + c * CODE_PITCH + 16 * rb) = make_uint4(w[0], w[1], w[2], w[3]);
                    catom[op_atom_byte(c, rb)] = c0 + c < a.cols && r0 + 32 * rb < rpad ? (uint8_t)e : 0u;
                }
            }
            __syncthreads();
            if (tid < 128)
                ((uint32_t *)(a.catoms + ((long)tx * op_k_atoms(a.rows) + ty) * 512))[tid] =
                    ((const uint32_t *)catom)[tid];
            const long cpitch = rpad / 2;
#pragma unroll
            for (int i = 0; i < QT * 4 / Q_THREADS; i++) {
                const int k = i * Q_THREADS + tid, c = k >> 2, rb = k & 3;  // four blocks of 16 bytes per column
                if (c0 + c < a.cols && r0 + 32 * rb < rpad)
                    *(uint4 *)(a.ccodes + (long)(c0 + c) * cpitch + r0 / 2 + 16 * rb) =
                        *(const uint4 *)(stage + c * CODE_PITCH + 16 * rb);
            }
        }
        __syncthreads();  // the tile, its codes and atoms in shared memory are free
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

// The values of an operand: eight per thread (one code word) where the rows of
// y are 16-byte aligned, else two per thread, so that a warp's stores stay next
// to each other.
template <typename YT, bool VEC>
__global__ void __launch_bounds__(256) k3_mx_dequantize(const uint8_t *codes, const uint8_t *atoms, int r0,
                                                        uint32_t n, FastDiv upr, int nk, int in, YT *y, long ld)
{
    griddep_launch_dependents();
    griddep_wait();
    constexpr int UB = VEC ? 4 : 1;  // code bytes of a unit
    for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
        const uint32_t q = upr.div(i);
        const int r = r0 + (int)q, c = (int)(i - q * upr.d) * 2 * UB, b = c >> 5;
        const float s = op_scale(atoms[((size_t)(r >> 7) * nk + (b >> 2)) * 512 + op_atom_byte(r, b)]);
        YT *o = y + (long)r * ld + c;
        if constexpr (VEC) {
            uint32_t h[4];
            e2m1x8_to_half2x4(*(const uint32_t *)(codes + 4 * (size_t)i), h[0], h[1], h[2], h[3]);
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float2 f = h2f2(h[j]);
                v[2 * j] = f.x * s;
                v[2 * j + 1] = f.y * s;
            }
            if constexpr (sizeof(YT) == 2) {
                uint32_t p[4];  // an E2M1 value times a power of two is exact in bf16
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                    p[j] = *(const uint32_t *)&t;
                }
                if (c + 8 <= in)
                    *(uint4 *)o = make_uint4(p[0], p[1], p[2], p[3]);
                else
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        if (c + j < in) o[j] = (YT)(p[j >> 1] >> (16 * (j & 1)));
            } else {
                if (c + 8 <= in) {
                    ((float4 *)o)[0] = make_float4(v[0], v[1], v[2], v[3]);
                    ((float4 *)o)[1] = make_float4(v[4], v[5], v[6], v[7]);
                } else
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        if (c + j < in) o[j] = v[j];
            }
        } else {
            const float2 f = e2m1x2_to_float2(codes[i]);
#pragma unroll
            for (int j = 0; j < 2; j++)
                if (c + j < in) {
                    const float v = (j ? f.y : f.x) * s;
                    if constexpr (sizeof(YT) == 2)
                        o[j] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
                    else
                        o[j] = v;
                }
        }
    }
}

bool rows_aligned16(const void *p, long ld, int es) { return ((uintptr_t)p & 15u) == 0 && (ld * es) % 16 == 0; }

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
    a.tiles_x = row ? op_k_atoms(cols) : op_row_tiles(cols);
    const long tiles = (long)a.tiles_x * (col ? op_k_atoms(rows) : op_row_tiles(rows));
    if (tiles > 0x3fffffffL) return K3MOE_EINVAL;
    a.tiles = (int)tiles;
    const bool vec = rows_aligned16(x, ld, xdt == K3MOE_BF16 ? 2 : 4);
    const size_t sm = !col && vec ? 0 : xdt == K3MOE_BF16 ? quant_smem<uint16_t>() : quant_smem<uint32_t>();
    void (*const kernel)(QuantArgs) =
        xdt == K3MOE_BF16 ? (vec ? k3_mx_quantize_operand<uint16_t, true> : k3_mx_quantize_operand<uint16_t, false>)
                          : (vec ? k3_mx_quantize_operand<uint32_t, true> : k3_mx_quantize_operand<uint32_t, false>);
    if (ensure_smem((const void *)kernel, sm) != K3MOE_OK) return K3MOE_ECUDA;
    return launch_pdl(kernel, dim3((unsigned)std::min<long>(tiles, 3L * num_sms())), dim3(Q_THREADS), sm, s, a) == cudaSuccess
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
    const uint32_t upr = (uint32_t)op_in_padded(op->in) / (VEC ? 8 : 2);
    const int rows = (int)std::min<long>(op->rows, std::max<long>(1, (1L << 30) / upr));
    for (int r = 0; r < op->rows; r += rows) {
        const uint32_t n = (uint32_t)std::min(rows, op->rows - r) * upr;
        const unsigned grid = (unsigned)std::min<long>(((long)n + 255) / 256, 32L * num_sms());
        if (launch_pdl(k3_mx_dequantize<YT, VEC>, dim3(grid), dim3(256), 0, s,
                       (const uint8_t *)op->codes + (size_t)r * (op_in_padded(op->in) / 2), (const uint8_t *)op->atoms,
                       r, n, FastDiv(upr), op_k_atoms(op->in), op->in, y, ld) != cudaSuccess) {
            cudaGetLastError();
            return K3MOE_ECUDA;
        }
    }
    return K3MOE_OK;
}

int launch_mx_dequantize(const k3moe_mx_operand *op, void *y, int ydt, long ld, cudaStream_t s)
{
    const bool vec = rows_aligned16(y, ld, ydt == K3MOE_BF16 ? 2 : 4);
    if (ydt == K3MOE_BF16)
        return vec ? launch_dequantize<uint16_t, true>(op, (uint16_t *)y, ld, s)
                   : launch_dequantize<uint16_t, false>(op, (uint16_t *)y, ld, s);
    return vec ? launch_dequantize<float, true>(op, (float *)y, ld, s)
               : launch_dequantize<float, false>(op, (float *)y, ld, s);
}

}  // namespace k3
