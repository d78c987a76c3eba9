// k3_capi_train.cu -- the extern "C" entry points around training and making
// MXFP4 layers: operands and their product, the SwiGLU checkpoint, the balance
// loss.  Argument checks and one launch each.
#include <cuda_runtime.h>

#include "k3_operand.cuh"

namespace k3 {
int launch_mx_quantize_operand(const void *x, int xdt, int rows, int cols, long ld, const k3moe_mx_operand *row,
                               const k3moe_mx_operand *col, cudaStream_t s);
int launch_mx_scale_atoms(const uint8_t *scales, int rows, int in, uint8_t *atoms, cudaStream_t s);
int launch_mx_dequantize(const k3moe_mx_operand *op, void *y, int ydt, long ld, cudaStream_t s);
int launch_mx_matmul(void *C, int cdt, long ldc, const k3moe_mx_operand *A, const k3moe_mx_operand *B, int accumulate,
                     int *err, cudaStream_t s);
void mx_matmul_form(int M, int N, int in, int cdt, int *pair, int *columns, int *ranks);
int launch_swiglu_forward(void *h, long ldh, void *ckpt, const void *g, long ldg, const void *u, long ldu, int dtype,
                          int T, int f, cudaStream_t s);
int launch_swiglu_backward(void *dg, long lddg, void *du, long lddu, const void *dh, long lddh, const void *ckpt,
                           int dtype, int T, int f, cudaStream_t s);
size_t balance_workspace_bytes(int E);
int launch_balance_forward(float *loss, int32_t *counts, int32_t *n_valid, const void *logits, int dtype, long ld,
                           const int32_t *ids, const uint8_t *mask, int T, int E, int k, float alpha, int rule,
                           void *ws, cudaStream_t s);
int launch_balance_backward(void *dlogits, long ldd, const void *logits, int dtype, long ld, const int32_t *ids,
                            const uint8_t *mask, const int32_t *counts, const int32_t *n_valid, const float *dloss,
                            const float *w, const float *dw, int T, int E, int k, float alpha, int rule,
                            cudaStream_t s);
}  // namespace k3

namespace {

cudaStream_t cs(k3moe_stream s) { return reinterpret_cast<cudaStream_t>(s); }
bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool valid_dtype(int dt) { return dt == K3MOE_F32 || dt == K3MOE_BF16; }
int esize(int dt) { return dt == K3MOE_BF16 ? 2 : 4; }
constexpr int32_t kMaxDim = 1 << 30;  // byte and tile indices of a row stay in 32 bits

// A [rows][cols] matrix of a caller: pointer, element alignment, row stride.
bool valid_rows(const void *p, int dt, int64_t ld, int32_t cols)
{
    return p && aligned(p, esize(dt)) && ld >= cols && ld <= ((int64_t)1 << 40);
}
bool valid_operand(const k3moe_mx_operand *o)
{
    return o && o->codes && o->atoms && aligned(o->codes, 16) && aligned(o->atoms, 16) && o->rows >= 1 &&
           o->rows <= kMaxDim && o->in >= 1 && o->in <= kMaxDim;
}
bool valid_operand(const k3moe_mx_operand *o, int32_t rows, int32_t in)
{
    return valid_operand(o) && o->rows == rows && o->in == in;
}
// A launch that writes what a later call may read as weights.  The launches allocate
// no memory of their own, but the library's table of raised shared-memory limits may
// grow: no exception leaves an entry point.
template <typename F>
int writing(k3moe_stream s, F launch)
{
    try {
        k3::note_weight_writes(cs(s));
        return launch();
    } catch (...) {
        return K3MOE_ENOMEM;
    }
}

}  // namespace

extern "C" {

int64_t k3moe_mx_operand_codes_bytes(int32_t rows, int32_t in)
{
    if (rows < 1 || in < 1 || rows > kMaxDim || in > kMaxDim) return -1;
    return (int64_t)rows * (k3::op_in_padded(in) / 2);
}

int64_t k3moe_mx_operand_atoms_bytes(int32_t rows, int32_t in)
{
    if (rows < 1 || in < 1 || rows > kMaxDim || in > kMaxDim) return -1;
    return (int64_t)k3::op_row_tiles(rows) * k3::op_k_atoms(in) * 512;
}

int k3moe_mx_quantize_operand(const k3moe_mx_operand *row, const k3moe_mx_operand *col, const void *x, int x_dtype,
                              int32_t rows, int32_t cols, int64_t ld, k3moe_stream s)
{
    if (rows < 1 || cols < 1 || rows > kMaxDim || cols > kMaxDim || !valid_dtype(x_dtype) || (!row && !col) ||
        !valid_rows(x, x_dtype, ld, cols) || (row && !valid_operand(row, rows, cols)) ||
        (col && !valid_operand(col, cols, rows)))
        return K3MOE_EINVAL;
    return writing(s, [&] { return k3::launch_mx_quantize_operand(x, x_dtype, rows, cols, (long)ld, row, col, cs(s)); });
}

int k3moe_mx_operand_from_matrix(const k3moe_mx_operand *op, const k3moe_mat *W, k3moe_stream s)
{
    if (!valid_operand(op) || !W || !W->packed || !W->scales || op->codes != W->packed || op->rows != W->rows ||
        W->in % 32 || k3::op_in_padded(op->in) != W->in || !aligned(W->scales, 16))
        return K3MOE_EINVAL;
    return writing(s, [&] { return k3::launch_mx_scale_atoms(W->scales, op->rows, op->in, op->atoms, cs(s)); });
}

int k3moe_mx_dequantize(void *y, int y_dtype, int64_t ld, const k3moe_mx_operand *op, k3moe_stream s)
{
    if (!valid_operand(op) || !valid_dtype(y_dtype) || !valid_rows(y, y_dtype, ld, op->in)) return K3MOE_EINVAL;
    return writing(s, [&] { return k3::launch_mx_dequantize(op, y, y_dtype, (long)ld, cs(s)); });
}

int k3moe_mx_matmul(void *C, int c_dtype, int64_t ldc, const k3moe_mx_operand *A, const k3moe_mx_operand *B,
                    int32_t accumulate, k3moe_stream s)
{
    if (!valid_operand(A) || !valid_operand(B) || A->in != B->in || !valid_dtype(c_dtype) ||
        !valid_rows(C, c_dtype, ldc, B->rows) || (accumulate && c_dtype != K3MOE_F32))
        return K3MOE_EINVAL;
    return writing(s, [&] {
        int *err = k3::device_error_word();
        if (!err) return (int)K3MOE_ECUDA;
        return k3::launch_mx_matmul(C, c_dtype, (long)ldc, A, B, accumulate ? 1 : 0, err, cs(s));
    });
}

int k3moe_mx_matmul_form(int32_t M, int32_t N, int32_t in, int c_dtype, int32_t *pair, int32_t *columns,
                         int32_t *ranks)
{
    if (M < 1 || N < 1 || in < 1 || M > kMaxDim || N > kMaxDim || in > kMaxDim || !valid_dtype(c_dtype) || !pair ||
        !columns || !ranks)
        return K3MOE_EINVAL;
    k3::mx_matmul_form(M, N, in, c_dtype, pair, columns, ranks);
    return K3MOE_OK;
}

int64_t k3moe_swiglu_ckpt_bytes(int32_t T, int32_t f)
{
    if (T < 1 || T > kMaxDim || f < 1 || f > kMaxDim) return -1;
    return 2 * (int64_t)T * (k3::op_in_padded(f) + k3::op_in_padded(f) / 32);
}

int k3moe_swiglu_forward(void *h, int64_t ldh, void *ckpt, int64_t ckpt_bytes, const void *g, int64_t ldg,
                         const void *u, int64_t ldu, int dtype, int32_t T, int32_t f, k3moe_stream s)
{
    if (k3moe_swiglu_ckpt_bytes(T, f) < 0 || !valid_dtype(dtype) || !ckpt || !aligned(ckpt, 16) ||
        ckpt_bytes < k3moe_swiglu_ckpt_bytes(T, f) || !valid_rows(h, dtype, ldh, f) || !valid_rows(g, dtype, ldg, f) ||
        !valid_rows(u, dtype, ldu, f))
        return K3MOE_EINVAL;
    return writing(s, [&] {
        return k3::launch_swiglu_forward(h, (long)ldh, ckpt, g, (long)ldg, u, (long)ldu, dtype, T, f, cs(s));
    });
}

int k3moe_swiglu_backward(void *dg, int64_t lddg, void *du, int64_t lddu, const void *dh, int64_t lddh,
                          const void *ckpt, int64_t ckpt_bytes, int dtype, int32_t T, int32_t f, k3moe_stream s)
{
    if (k3moe_swiglu_ckpt_bytes(T, f) < 0 || !valid_dtype(dtype) || !ckpt || !aligned(ckpt, 16) ||
        ckpt_bytes < k3moe_swiglu_ckpt_bytes(T, f) || !valid_rows(dg, dtype, lddg, f) ||
        !valid_rows(du, dtype, lddu, f) || !valid_rows(dh, dtype, lddh, f) || dg == du)
        return K3MOE_EINVAL;
    // on top of dh with another stride a row would be written before it is read
    if (T > 1 && ((dg == dh && lddg != lddh) || (du == dh && lddu != lddh))) return K3MOE_EINVAL;
    return writing(s, [&] {
        return k3::launch_swiglu_backward(dg, (long)lddg, du, (long)lddu, dh, (long)lddh, ckpt, dtype, T, f, cs(s));
    });
}

size_t k3moe_balance_workspace(int32_t E) { return E < 1 || E > 1024 ? 0 : k3::balance_workspace_bytes(E); }

static bool valid_balance(const void *logits, int dtype, int64_t ld, const int32_t *ids, int32_t T, int32_t E,
                          int32_t k, int rule)
{
    return T >= 1 && T <= kMaxDim && E >= 1 && E <= 1024 && k >= 1 && k <= 32 && valid_dtype(dtype) &&
           valid_rows(logits, dtype, ld, E) && ids && aligned(ids, 4) && rule >= K3MOE_ROUTER_SOFTMAX &&
           rule <= K3MOE_ROUTER_SIGMOID_NORM;
}

int k3moe_balance_forward(float *loss, int32_t *counts, int32_t *n_valid, const void *logits, int dtype, int64_t ld,
                          const int32_t *ids, const uint8_t *mask, int32_t T, int32_t E, int32_t k, float alpha,
                          int rule, void *ws, size_t ws_bytes, k3moe_stream s)
{
    if (!valid_balance(logits, dtype, ld, ids, T, E, k, rule) || !loss || !counts || !n_valid || !aligned(loss, 4) ||
        !aligned(counts, 4) || !aligned(n_valid, 4) || !ws || !aligned(ws, 16) ||
        ws_bytes < k3moe_balance_workspace(E))
        return K3MOE_EINVAL;
    return writing(s, [&] {
        return k3::launch_balance_forward(loss, counts, n_valid, logits, dtype, (long)ld, ids, mask, T, E, k, alpha,
                                          rule, ws, cs(s));
    });
}

int k3moe_balance_backward(void *dlogits, int64_t ldd, const void *logits, int dtype, int64_t ld, const int32_t *ids,
                           const uint8_t *mask, const int32_t *counts, const int32_t *n_valid, const float *dloss,
                           const float *w, const float *dw, int32_t T, int32_t E, int32_t k, float alpha, int rule,
                           k3moe_stream s)
{
    if (!valid_balance(logits, dtype, ld, ids, T, E, k, rule) || !valid_rows(dlogits, dtype, ldd, E) || !counts ||
        !n_valid || !dloss || !aligned(counts, 4) || !aligned(n_valid, 4) || !aligned(dloss, 4) || (!w != !dw) ||
        !aligned(w, 4) || !aligned(dw, 4) || (dlogits == logits && ldd != ld))
        return K3MOE_EINVAL;
    return writing(s, [&] {
        return k3::launch_balance_backward(dlogits, (long)ldd, logits, dtype, (long)ld, ids, mask, counts, n_valid,
                                           dloss, w, dw, T, E, k, alpha, rule, cs(s));
    });
}

}  // extern "C"
