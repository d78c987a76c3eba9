// k3_balance.cu -- the router's balance loss with per-expert counts, and the
// gradient of the logits (balance loss and combine weights together).
//
//   p = softmax(l) or sigma(l) / sum sigma(l);  c_e = slots that chose e
//   f_e = E c_e / (k N),  P_e = mean p_e,  loss = alpha sum f_e P_e
//   dl = dloss alpha / N * p (f - <f, p>)  [* (1 - sigma(l)) for the sigmoid rules]
//
// <f, p> is taken of f - 1 (sum p = 1), an integer difference over k N, so that a
// nearly even choice does not lose the gradient to cancellation.
//
// Bound: HBM for large batches (the logits are read once per direction),
// latency for small ones.  A warp holds a row in registers, expert
// 128 i + 4 lane + c (E <= 1024: at most 32 values a lane), while its next row is
// on the way into shared memory (cp.async; rows that are not made of aligned
// 16-byte units are loaded directly).  Forward: each warp sums its rows' p per
// expert in registers, a CTA adds its warps' sums in shared memory in warp order,
// and the CTAs meet in 64-bit fixed point (integer adds: the same result in any
// order); the last CTA to arrive forms the loss and clears the workspace.  One
// launch per direction.
#include <cuda_runtime.h>

#include <algorithm>

#include "k3_launch.cuh"
#include "k3_operand.cuh"

namespace k3 {
namespace {

// Backward: three CTAs per SM (16384 x 896 fp32, softmax, with combine weights 22.9 us,
// 5.3 TB/s read and written; the sigmoid rules 59 us, bound by the issue of their
// exponentials and divisions).
constexpr int BL_THREADS = 256, BL_WARPS = BL_THREADS / 32;
// Forward: one CTA per SM, so that half as many sums meet in global atomics as
// with two of 256 threads.  Its rows cost latency (two reductions each), so more
// warps help until the joining of their sums costs as much: 16384 x 896 fp32 takes
// 14.8 us with 16 warps, 13.2 with 20, 14.0 with 24 (a third row in flight per warp
// changed nothing); 13.6 since the row's maximum is subtracted first; the sigmoid rules
// 33.6.
constexpr int BF_THREADS = 640, BF_WARPS = BF_THREADS / 32;

// Workspace: fixed-point sums [E], counts [E], valid tokens, a flag for
// non-finite sums, the ticket.
struct BalanceWs {
    unsigned long long *sum;
    unsigned *count, *valid, *bad, *ticket;
};
__host__ __device__ inline BalanceWs balance_ws(void *p, int E)
{
    BalanceWs w;
    w.sum = (unsigned long long *)p;
    w.count = (unsigned *)(w.sum + E);
    w.valid = w.count + E;
    w.bad = w.valid + 1;
    w.ticket = w.valid + 2;
    return w;
}

struct BalanceArgs {
    const void *logits;
    long ld, ldd;
    const int32_t *ids;
    const uint8_t *mask;
    int T, E, k, rule;
    float alpha;
    bool vec, vec_out;  // rows of logits, of dlogits made of aligned 16-byte units
    // forward
    float *loss;
    int32_t *counts, *n_valid;
    void *ws;
    int shift;  // fixed-point sums in units of 2^-shift
    // backward
    void *dlogits;
    const float *dloss, *w, *dw;
};

template <typename T>
K3_DEV float load1(const void *p, long i)
{
    if constexpr (sizeof(T) == 2)
        return __uint_as_float((uint32_t)((const uint16_t *)p)[i] << 16);
    else
        return ((const float *)p)[i];
}

K3_DEV void put1(uint16_t *o, int e, float v) { o[e] = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
K3_DEV void put1(float *o, int e, float v) { o[e] = v; }

// Largest value, NaN if there is one.
K3_DEV float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// sigma(l) / e^m without overflow or a row of zeros, for m = min(largest l, 0).
K3_DEV float scaled_sigmoid(float l, float m)
{
    return l > 0.f ? 1.f / (1.f + expf(-l)) : expf(l - m) / (1.f + expf(l));
}

// Starts the copy of row t into a warp's buffer; one group per call.
template <typename T>
K3_DEV void fetch_row(const BalanceArgs &a, int t, bool on, uint8_t *buf, int lane)
{
    if (on) {
        const uint8_t *src = (const uint8_t *)a.logits + (long)t * a.ld * (int)sizeof(T);
        const int n16 = a.E * (int)sizeof(T) / 16;
        for (int i = lane; i < n16; i += 32)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(buf + 16 * i)), "l"(src + 16 * i)
                         : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// Row t into registers: v[4 i + c] = logit of expert 128 i + 4 lane + c, -inf past
// E; from the warp's buffer (a.vec) or from global memory.
template <typename T, int NV>
K3_DEV void read_row(const BalanceArgs &a, int t, const uint8_t *buf, int lane, float (&v)[4 * NV])
{
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int e = 128 * i + 4 * lane;
        if (a.vec) {
            if (e < a.E) {  // E is a multiple of 4
                if constexpr (sizeof(T) == 2) {
                    const uint2 q = *(const uint2 *)(buf + 2 * e);
                    v[4 * i] = __uint_as_float(q.x << 16);
                    v[4 * i + 1] = __uint_as_float(q.x & 0xffff0000u);
                    v[4 * i + 2] = __uint_as_float(q.y << 16);
                    v[4 * i + 3] = __uint_as_float(q.y & 0xffff0000u);
                } else {
                    const float4 q = *(const float4 *)(buf + 4 * e);
                    v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; c++) v[4 * i + c] = -INFINITY;
            }
        } else {
#pragma unroll
            for (int c = 0; c < 4; c++) v[4 * i + c] = e + c < a.E ? load1<T>(a.logits, (long)t * a.ld + e + c) : -INFINITY;
        }
    }
}

// Logits to unnormalised probabilities; inv makes them sum to 1.  False (and
// nothing done) for a row of -inf.  SIG: the sigmoid rules.
// Softmax: e^(l - m) as 2^((l - m) log2 e) by the one-instruction exponential
// (2^-22).  The difference comes first: the product of a large m alone is off by
// more than an exponent can hold (from about 2^31 on) or infinite.  The roundings
// of the difference t, of the constant and of the product cost p at most 3 t 2^-24
// of itself, so about 2^-24 of the row's largest p.
template <bool SIG>
K3_DEV float unnormalised(float l, float m)
{
    return SIG ? scaled_sigmoid(l, m) : exp2_fast((l - m) * LOG2E);
}
template <int NV, bool SIG>
K3_DEV bool row_probs(float (&v)[4 * NV], float &inv, float &m)
{
    m = v[0];
#pragma unroll
    for (int i = 1; i < 4 * NV; i++) m = max_nan(m, v[i]);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (m == -INFINITY) return false;
    if constexpr (SIG) m = fminf(m, 0.f);  // a NaN among the logits is still in the sum
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4 * NV; i++) s += v[i] = unnormalised<SIG>(v[i], m);
    inv = 1.f / warp_sum(s);
    return true;
}

// Bytes of a row's buffer.
__host__ __device__ inline int row_buf(int E, int es) { return (E * es + 15) / 16 * 16; }

template <typename T, int NV, bool SIG>
__global__ void __launch_bounds__(BF_THREADS, 1) k3_balance_forward(const BalanceArgs a)
{
    extern __shared__ __align__(16) uint8_t dyn[];  // two row buffers per warp; afterwards the warps' sums
    __shared__ unsigned cnt[128 * NV];
    __shared__ unsigned nval, last;
    __shared__ float red[BF_WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rb = row_buf(a.E, (int)sizeof(T));
    uint8_t *buf = dyn + warp * 2 * rb;
    for (int e = threadIdx.x; e < 128 * NV; e += BF_THREADS) cnt[e] = 0u;
    if (threadIdx.x == 0) nval = 0u;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();

    float acc[4 * NV];
#pragma unroll
    for (int i = 0; i < 4 * NV; i++) acc[i] = 0.f;
    unsigned mine = 0u;
    const int step = gridDim.x * BF_WARPS;
    int t = blockIdx.x * BF_WARPS + warp, b = 0;
    auto kept = [&](int r) { return r < a.T && (!a.mask || a.mask[r]); };
    auto slot = [&](int r) { return lane < a.k && r < a.T ? a.ids[(long)r * a.k + lane] : -1; };
    // the mask is read two rows ahead, the row and its ids one
    bool on = kept(t), on_next = kept(t + step);
    int id = slot(t);
    if (a.vec) fetch_row<T>(a, t, on, buf, lane);
    for (; t < a.T; t += step) {
        const bool on_later = kept(t + 2 * step);
        const int id_next = slot(t + step);
        if (a.vec) {
            fetch_row<T>(a, t + step, on_next, buf + (b ^ 1) * rb, lane);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
        }
        if (on) {
            float v[4 * NV], inv, m;
            read_row<T, NV>(a, t, buf + b * rb, lane, v);
            if (row_probs<NV, SIG>(v, inv, m)) {
                mine++;
                // a warp has at most T / 3040 + 1 rows: fp32 loses 2^-24 of the sum a row
#pragma unroll
                for (int i = 0; i < 4 * NV; i++) acc[i] += v[i] * inv;
                if (id >= 0 && id < a.E) atomicAdd(&cnt[id], 1u);
            }
        }
        __syncwarp();  // the buffer has been read before it is filled again
        on = on_next, on_next = on_later, id = id_next, b ^= 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float *part = (float *)dyn;  // [warp][128 NV]
#pragma unroll
    for (int i = 0; i < NV; i++)
        *(float4 *)(part + warp * 128 * NV + 128 * i + 4 * lane) =
            make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
    if (lane == 0 && mine) atomicAdd(&nval, mine);
    __syncthreads();
    const BalanceWs ws = balance_ws(a.ws, a.E);
    const float unit = __uint_as_float((uint32_t)(127 + a.shift) << 23);
    for (int e = threadIdx.x; e < a.E; e += BF_THREADS) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < BF_WARPS; w++) s += part[w * 128 * NV + e];
        // the sum is at most the CTA's tokens, the scaled one below 2^62
        if (s == s) {
            if (s != 0.f) atomicAdd(ws.sum + e, (unsigned long long)(s * unit));
        } else {
            atomicOr(ws.bad, 1u);
        }
        if (cnt[e]) atomicAdd(ws.count + e, cnt[e]);
    }
    if (threadIdx.x == 0 && nval) atomicAdd(ws.valid, nval);
    __syncthreads();
    if (threadIdx.x == 0) last = ticket_arrive(ws.ticket) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;

    // the last CTA: the loss from the whole batch's sums, the workspace cleared.
    // f_e P_e = E c_e / (k n) * sum / n in fp32, added in a fixed tree: a few 2^-24 of
    // the loss, which is of one sign throughout.
    const unsigned n = __ldcg(ws.valid);
    const float kn = (float)a.k * (float)n, pn = n ? 1.f / (unit * (float)n) : 0.f;
    float l = 0.f;
    for (int e = threadIdx.x; e < a.E; e += BF_THREADS) {
        const unsigned c = __ldcg(ws.count + e);
        l += (float)c * ((float)__ldcg(ws.sum + e) * pn);
        a.counts[e] = (int32_t)c;
        ws.sum[e] = 0ull;
        ws.count[e] = 0u;
    }
    l = warp_sum(l);
    if (lane == 0) red[warp] = l;
    __syncthreads();
    if (threadIdx.x == 0) {
        float s = 0.f;
        for (int w = 0; w < BF_WARPS; w++) s += red[w];
        float loss = n ? a.alpha * ((float)a.E * s / kn) : 0.f;
        if (__ldcg(ws.bad)) loss = __uint_as_float(0x7fc00000u);
        *a.loss = loss;
        *a.n_valid = (int32_t)n;
        *ws.valid = 0u;
        *ws.bad = 0u;
        *ws.ticket = 0u;
    }
}

template <typename T, int NV, bool SIG>
__global__ void __launch_bounds__(BL_THREADS, 3) k3_balance_backward(const BalanceArgs a)
{
    extern __shared__ __align__(16) uint8_t dyn[];  // two row buffers per warp
    __shared__ __align__(16) float f1[128 * NV];    // f_e - 1
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rb = row_buf(a.E, (int)sizeof(T));
    uint8_t *buf = dyn + warp * 2 * rb;
    griddep_wait();
    griddep_launch_dependents();
    const int step = gridDim.x * BL_WARPS;
    int t = blockIdx.x * BL_WARPS + warp, b = 0;
    auto kept = [&](int r) { return r < a.T && (!a.mask || a.mask[r]); };
    // a row's chosen experts, one per lane, with their weights and gradients
    struct Slot {
        int id;
        float w, dw;
    };
    auto slot = [&](int r) {
        Slot s = {-1, 0.f, 0.f};
        if (a.dw && lane < a.k && r < a.T) {
            const long i = (long)r * a.k + lane;
            s = {a.ids[i], a.w[i], a.dw[i]};
            if (s.id < 0 || s.id >= a.E) s.id = -1;
        }
        return s;
    };
    // the mask is read two rows ahead, the row and its slots one
    bool on = kept(t), on_next = kept(t + step);
    if (a.vec) fetch_row<T>(a, t, on, buf, lane);
    Slot sl = slot(t);
    const int n = *a.n_valid;
    const long kn = (long)a.k * n;
    for (int e = threadIdx.x; e < 128 * NV; e += BL_THREADS)
        f1[e] = e < a.E && n > 0 ? (float)((long)a.E * a.counts[e] - kn) / (float)kn : 0.f;
    __syncthreads();
    const float scale = n > 0 ? a.alpha * *a.dloss / (float)n : 0.f;

    for (; t < a.T; t += step) {
        const bool on_later = kept(t + 2 * step);
        const Slot next = slot(t + step);
        if (a.vec) {
            fetch_row<T>(a, t + step, on_next, buf + (b ^ 1) * rb, lane);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
        }
        T *o = (T *)a.dlogits + (long)t * a.ldd;
        float v[4 * NV], inv, m;
        bool valid = on, first = false;
        float at = 0.f;  // the whole gradient of this lane's chosen expert
        if (on) {
            // logit of the chosen expert, before another lane may write it (in place)
            float lj = 0.f;
            if (sl.id >= 0) lj = a.vec ? load1<T>(buf + b * rb, sl.id) : load1<T>(a.logits, (long)t * a.ld + sl.id);
            read_row<T, NV>(a, t, buf + b * rb, lane, v);
            __syncwarp();
            valid = row_probs<NV, SIG>(v, inv, m);
            if (valid) {
                float dot = 0.f;  // <f - 1, unnormalised p>
#pragma unroll
                for (int i = 0; i < NV; i++) {
                    const float4 f = *(const float4 *)(f1 + 128 * i + 4 * lane);
                    dot += v[4 * i] * f.x + v[4 * i + 1] * f.y + v[4 * i + 2] * f.z + v[4 * i + 3] * f.w;
                }
                // p scale (f - <f, p>)
                const float c1 = scale * inv, c0 = -warp_sum(dot) * inv * c1;
                if (a.dw) {
                    const float inner = warp_sum(sl.id >= 0 ? sl.w * sl.dw : 0.f);
                    float c;
                    if constexpr (SIG) {
                        const float r = 1.f / (1.f + expf(lj));  // 1 - sigma
                        c = a.rule == K3MOE_ROUTER_SIGMOID ? router_sigmoid(lj) * r * sl.dw
                                                           : sl.w * r * (sl.dw - inner);
                        at = r;
                    } else {
                        c = sl.w * (sl.dw - inner);
                        at = 1.f;
                    }
                    // slots with the same id are added in slot order by the first
                    const unsigned same = __match_any_sync(0xffffffffu, sl.id);
                    if (__any_sync(0xffffffffu, sl.id >= 0 && __popc(same) > 1)) {
                        float s = 0.f;
                        for (int j = 0; j < a.k; j++) {
                            const float cj = __shfl_sync(0xffffffffu, c, j);
                            if ((same >> j) & 1u) s += cj;
                        }
                        c = s;
                    }
                    first = sl.id >= 0 && (same & ((1u << lane) - 1u)) == 0u;
                    at = unnormalised<SIG>(lj, m) * (f1[max(sl.id, 0)] * c1 + c0) * at + c;
                }
#pragma unroll
                for (int i = 0; i < NV; i++) {
                    const float4 f = *(const float4 *)(f1 + 128 * i + 4 * lane);
                    v[4 * i] *= f.x * c1 + c0, v[4 * i + 1] *= f.y * c1 + c0;
                    v[4 * i + 2] *= f.z * c1 + c0, v[4 * i + 3] *= f.w * c1 + c0;
                }
                if constexpr (SIG) {
                    // 1 - sigma(l) as sigma(-l), which keeps its digits for large l
                    float l[4 * NV];
                    read_row<T, NV>(a, t, buf + b * rb, lane, l);
#pragma unroll
                    for (int i = 0; i < 4 * NV; i++) v[i] *= 1.f / (1.f + expf(l[i]));
                }
            }
        }
        if (!valid) {
#pragma unroll
            for (int i = 0; i < 4 * NV; i++) v[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int e = 128 * i + 4 * lane;
            if (a.vec_out) {
                if (e < a.E) {
                    if constexpr (sizeof(T) == 2) {
                        const __nv_bfloat162 lo = __floats2bfloat162_rn(v[4 * i], v[4 * i + 1]),
                                             hi = __floats2bfloat162_rn(v[4 * i + 2], v[4 * i + 3]);
                        *(uint2 *)(o + e) = make_uint2(*(const uint32_t *)&lo, *(const uint32_t *)&hi);
                    } else {
                        *(float4 *)(o + e) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; c++)
                    if (e + c < a.E) put1(o, e + c, v[4 * i + c]);
            }
        }
        // the row is stored (and the buffer read, before it is filled again); the
        // chosen experts' entries are stored over it
        __syncwarp();
        if (first) put1(o, sl.id, at);
        on = on_next, on_next = on_later, sl = next, b ^= 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename T, int NV, bool SIG>
int launch(const BalanceArgs &a, bool backward, cudaStream_t s)
{
    const int threads = backward ? BL_THREADS : BF_THREADS, warps = threads / 32;
    const dim3 grid((unsigned)std::max(1, std::min((a.T - 1) / warps + 1, (backward ? 3 : 1) * num_sms())));
    const size_t bufs = (size_t)warps * 2 * row_buf(a.E, (int)sizeof(T));
    const size_t smem = backward ? bufs : std::max(bufs, sizeof(float) * warps * 128 * NV);
    const auto kernel = backward ? k3_balance_backward<T, NV, SIG> : k3_balance_forward<T, NV, SIG>;
    // the static arrays count towards the limit too
    if (ensure_smem((const void *)kernel, smem + 8192) != K3MOE_OK) return K3MOE_ECUDA;
    return launch_pdl(kernel, grid, dim3((unsigned)threads), smem, s, a) == cudaSuccess ? K3MOE_OK
                                                                                 : (cudaGetLastError(), K3MOE_ECUDA);
}
// A lane holds four values per 128 experts.
template <typename T, bool SIG, int NV = 1>
int launch_e(const BalanceArgs &a, bool backward, cudaStream_t s)
{
    if constexpr (NV < 8)
        if (a.E > 128 * NV) return launch_e<T, SIG, NV + 1>(a, backward, s);
    return launch<T, NV, SIG>(a, backward, s);
}
template <typename T>
int launch_rule(const BalanceArgs &a, bool backward, cudaStream_t s)
{
    return a.rule == K3MOE_ROUTER_SOFTMAX ? launch_e<T, false>(a, backward, s) : launch_e<T, true>(a, backward, s);
}
// Rows made of aligned 16-byte units.
bool rows16(const void *p, long ld, int E, int es)
{
    return ((uintptr_t)p & 15u) == 0 && ld * es % 16 == 0 && E * es % 16 == 0;
}
int launch_dt(const BalanceArgs &a, int dtype, bool backward, cudaStream_t s)
{
    return dtype == K3MOE_BF16 ? launch_rule<uint16_t>(a, backward, s) : launch_rule<float>(a, backward, s);
}

}  // namespace

size_t balance_workspace_bytes(int E) { return (size_t)E * 12 + 16; }

int launch_balance_forward(float *loss, int32_t *counts, int32_t *n_valid, const void *logits, int dtype, long ld,
                           const int32_t *ids, const uint8_t *mask, int T, int E, int k, float alpha, int rule,
                           void *ws, cudaStream_t s)
{
    BalanceArgs a = {};
    a.logits = logits, a.ld = ld, a.ids = ids, a.mask = mask;
    a.T = T, a.E = E, a.k = k, a.rule = rule, a.alpha = alpha;
    a.loss = loss, a.counts = counts, a.n_valid = n_valid, a.ws = ws;
    a.vec = rows16(logits, ld, E, dtype == K3MOE_BF16 ? 2 : 4);
    a.shift = 61;  // T 2^shift < 2^62
    while (a.shift > 46 || ((long)T >> (62 - a.shift)) != 0) a.shift--;
    return launch_dt(a, dtype, false, s);
}
int launch_balance_backward(void *dlogits, long ldd, const void *logits, int dtype, long ld, const int32_t *ids,
                            const uint8_t *mask, const int32_t *counts, const int32_t *n_valid, const float *dloss,
                            const float *w, const float *dw, int T, int E, int k, float alpha, int rule, cudaStream_t s)
{
    BalanceArgs a = {};
    a.logits = logits, a.ld = ld, a.ldd = ldd, a.ids = ids, a.mask = mask;
    a.T = T, a.E = E, a.k = k, a.rule = rule, a.alpha = alpha;
    a.counts = (int32_t *)counts, a.n_valid = (int32_t *)n_valid;
    a.vec = rows16(logits, ld, E, dtype == K3MOE_BF16 ? 2 : 4);
    a.vec_out = rows16(dlogits, ldd, E, dtype == K3MOE_BF16 ? 2 : 4);
    a.dlogits = dlogits, a.dloss = dloss, a.w = w, a.dw = dw;
    return launch_dt(a, dtype, true, s);
}

}  // namespace k3
