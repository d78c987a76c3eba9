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
// latency for small ones.  A warp holds a row in registers (E <= 1024: at most 32
// values a lane).  Forward: each warp sums its rows' p per expert in registers,
// a CTA adds its warps' sums in shared memory in warp order, and the CTAs meet in
// 64-bit fixed point (integer adds: the same result in any order); the last CTA
// to arrive forms the loss and clears the workspace.  One launch per direction.
#include <cuda_runtime.h>

#include <algorithm>

#include "k3_launch.cuh"
#include "k3_device.cuh"

namespace k3 {
namespace {

constexpr int BL_THREADS = 256, BL_WARPS = BL_THREADS / 32;

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

K3_DEV float warp_max(float v)
{
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// sigma(l) / e^m without overflow or a row of zeros, for m = min(largest l, 0).
K3_DEV float scaled_sigmoid(float l, float m)
{
    return l > 0.f ? 1.f / (1.f + expf(-l)) : expf(l - m) / (1.f + expf(l));
}

// Row t of the logits, v[i] = logit of expert lane + 32 i (-inf past E).
// Returns whether the token is valid.  Afterwards v holds the unnormalised
// probabilities and inv the factor that makes them sum to 1.
template <typename T, int NC>
K3_DEV bool row_probs(const BalanceArgs &a, int t, int lane, float (&v)[NC], float &m, float &inv)
{
    if (a.mask && !a.mask[t]) return false;
    float mx = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < NC; i++) {
        const int e = lane + 32 * i;
        v[i] = e < a.E ? load1<T>(a.logits, (long)t * a.ld + e) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < NC; i++) {
        mx = fmaxf(mx, v[i]);
        nan |= v[i] != v[i];
    }
    mx = warp_max(mx);
    if (mx == -INFINITY && !__any_sync(0xffffffffu, nan)) return false;
    m = a.rule == K3MOE_ROUTER_SOFTMAX ? mx : fminf(mx, 0.f);
    float s = 0.f;
    if (a.rule == K3MOE_ROUTER_SOFTMAX) {
#pragma unroll
        for (int i = 0; i < NC; i++) s += v[i] = expf(v[i] - m);
    } else {
#pragma unroll
        for (int i = 0; i < NC; i++) s += v[i] = scaled_sigmoid(v[i], m);
    }
    inv = 1.f / warp_sum(s);
    return true;
}

template <typename T, int NC>
__global__ void __launch_bounds__(BL_THREADS) k3_balance_forward(const BalanceArgs a)
{
    __shared__ float part[BL_WARPS][32 * NC];
    __shared__ unsigned cnt[32 * NC];
    __shared__ unsigned nval, last;
    __shared__ double red[BL_WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < 32 * NC; e += BL_THREADS) cnt[e] = 0u;
    if (threadIdx.x == 0) nval = 0u;
    __syncthreads();
    griddep_launch_dependents();
    griddep_wait();

    float acc[NC];
#pragma unroll
    for (int i = 0; i < NC; i++) acc[i] = 0.f;
    unsigned mine = 0u;
    for (int t = blockIdx.x * BL_WARPS + warp; t < a.T; t += gridDim.x * BL_WARPS) {
        const int id = lane < a.k ? a.ids[(long)t * a.k + lane] : -1;
        float v[NC], m, inv;
        if (!row_probs<T, NC>(a, t, lane, v, m, inv)) continue;
        mine++;
#pragma unroll
        for (int i = 0; i < NC; i++) acc[i] += v[i] * inv;
        if (id >= 0 && id < a.E) atomicAdd(&cnt[id], 1u);
    }
#pragma unroll
    for (int i = 0; i < NC; i++) part[warp][lane + 32 * i] = acc[i];
    if (lane == 0 && mine) atomicAdd(&nval, mine);
    __syncthreads();
    const BalanceWs ws = balance_ws(a.ws, a.E);
    const float unit = __uint_as_float((uint32_t)(127 + a.shift) << 23);
    for (int e = threadIdx.x; e < a.E; e += BL_THREADS) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < BL_WARPS; w++) s += part[w][e];
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

    // the last CTA: the loss from the whole batch's sums, the workspace cleared
    const unsigned n = __ldcg(ws.valid);
    const double unit2 = 1.0 / (double)unit;
    double l = 0.0;
    for (int e = threadIdx.x; e < a.E; e += BL_THREADS) {
        const unsigned c = __ldcg(ws.count + e);
        l += (double)c * ((double)__ldcg(ws.sum + e) * unit2);
        a.counts[e] = (int32_t)c;
        ws.sum[e] = 0ull;
        ws.count[e] = 0u;
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    if (lane == 0) red[warp] = l;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int w = 0; w < BL_WARPS; w++) s += red[w];
        const double nn = (double)n;
        float loss = n ? (float)((double)a.alpha * a.E * s / ((double)a.k * nn * nn)) : 0.f;
        if (__ldcg(ws.bad)) loss = __uint_as_float(0x7fc00000u);
        *a.loss = loss;
        *a.n_valid = (int32_t)n;
        *ws.valid = 0u;
        *ws.bad = 0u;
        *ws.ticket = 0u;
    }
}

template <typename T, int NC>
__global__ void __launch_bounds__(BL_THREADS) k3_balance_backward(const BalanceArgs a)
{
    __shared__ float f1[32 * NC];                    // f_e - 1
    __shared__ float extra[BL_WARPS][32 * NC];       // combine weights' part of a row
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < 32 * NC; e += BL_THREADS)
#pragma unroll
        for (int w = 0; w < BL_WARPS; w++) extra[w][e] = 0.f;
    griddep_launch_dependents();
    griddep_wait();
    const int n = *a.n_valid;
    const long kn = (long)a.k * n;
    for (int e = threadIdx.x; e < 32 * NC; e += BL_THREADS)
        f1[e] = e < a.E && n > 0 ? (float)((long)a.E * a.counts[e] - kn) / (float)kn : 0.f;
    __syncthreads();
    const float scale = n > 0 ? a.alpha * *a.dloss / (float)n : 0.f;

    for (int t = blockIdx.x * BL_WARPS + warp; t < a.T; t += gridDim.x * BL_WARPS) {
        float v[NC], m = 0.f, inv = 0.f;
        int id = -1;
        float w = 0.f, dw = 0.f, lj = 0.f;
        if (a.dw && lane < a.k) {
            id = a.ids[(long)t * a.k + lane];
            w = a.w[(long)t * a.k + lane];
            dw = a.dw[(long)t * a.k + lane];
            if (id < 0 || id >= a.E) id = -1;
            if (id >= 0 && a.rule != K3MOE_ROUTER_SOFTMAX) lj = load1<T>(a.logits, (long)t * a.ld + id);
        }
        const bool on = row_probs<T, NC>(a, t, lane, v, m, inv);
        if (on) {
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < NC; i++) {
                v[i] *= inv;
                dot += v[i] * f1[lane + 32 * i];
            }
            dot = warp_sum(dot);
#pragma unroll
            for (int i = 0; i < NC; i++) v[i] = scale * v[i] * (f1[lane + 32 * i] - dot);
            if (a.rule != K3MOE_ROUTER_SOFTMAX) {
                // 1 - sigma(l) as sigma(-l), which keeps its digits for large l
#pragma unroll
                for (int i = 0; i < NC; i++)
                    if (lane + 32 * i < a.E)
                        v[i] *= 1.f / (1.f + expf(load1<T>(a.logits, (long)t * a.ld + lane + 32 * i)));
            }
        } else {
#pragma unroll
            for (int i = 0; i < NC; i++) v[i] = 0.f;
        }
        if (a.dw && on) {
            const float inner = warp_sum(id >= 0 ? w * dw : 0.f);
            float c;
            if (a.rule == K3MOE_ROUTER_SOFTMAX) {
                c = w * (dw - inner);
            } else {
                const float r = 1.f / (1.f + expf(lj));  // 1 - sigma
                c = a.rule == K3MOE_ROUTER_SIGMOID ? router_sigmoid(lj) * r * dw : w * r * (dw - inner);
            }
            // slots with the same id are added in slot order by the first
            const unsigned same = __match_any_sync(0xffffffffu, id >= 0 ? id : -1 - lane);
            if (__any_sync(0xffffffffu, __popc(same) > 1)) {
                float s = 0.f;
                for (int j = 0; j < a.k; j++) {
                    const float cj = __shfl_sync(0xffffffffu, c, j);
                    if ((same >> j) & 1u) s += cj;
                }
                c = s;
            }
            const bool first = id >= 0 && (same & ((1u << lane) - 1u)) == 0u;
            if (first) extra[warp][id] = c;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < NC; i++) v[i] += extra[warp][lane + 32 * i];
            __syncwarp();
            if (first) extra[warp][id] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < NC; i++) {
            const int e = lane + 32 * i;
            if (e < a.E) {
                if constexpr (sizeof(T) == 2)
                    ((__nv_bfloat16 *)a.dlogits)[(long)t * a.ldd + e] = __float2bfloat16_rn(v[i]);
                else
                    ((float *)a.dlogits)[(long)t * a.ldd + e] = v[i];
            }
        }
    }
}

template <typename T, int NC>
int launch(const BalanceArgs &a, bool backward, cudaStream_t s)
{
    const dim3 grid((unsigned)std::max(1, std::min((a.T + BL_WARPS - 1) / BL_WARPS, 2 * num_sms())));
    const cudaError_t e = backward ? launch_pdl(k3_balance_backward<T, NC>, grid, dim3(BL_THREADS), 0, s, a)
                                   : launch_pdl(k3_balance_forward<T, NC>, grid, dim3(BL_THREADS), 0, s, a);
    return e == cudaSuccess ? K3MOE_OK : (cudaGetLastError(), K3MOE_ECUDA);
}
// Values a lane holds: the next of 4, 8, 16, 24, 32 (a row of E experts).
template <typename T>
int launch_e(const BalanceArgs &a, bool backward, cudaStream_t s)
{
    const int nc = (a.E + 31) / 32;
    if (nc <= 4) return launch<T, 4>(a, backward, s);
    if (nc <= 8) return launch<T, 8>(a, backward, s);
    if (nc <= 16) return launch<T, 16>(a, backward, s);
    if (nc <= 24) return launch<T, 24>(a, backward, s);
    return launch<T, 32>(a, backward, s);
}
int launch_dt(const BalanceArgs &a, int dtype, bool backward, cudaStream_t s)
{
    return dtype == K3MOE_BF16 ? launch_e<uint16_t>(a, backward, s) : launch_e<float>(a, backward, s);
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
    a.dlogits = dlogits, a.dloss = dloss, a.w = w, a.dw = dw;
    return launch_dt(a, dtype, true, s);
}

}  // namespace k3
