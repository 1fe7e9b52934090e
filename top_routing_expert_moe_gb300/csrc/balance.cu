// balance.cu -- per-sequence balance loss and z loss of the router, with gradients.
//
//   p = softmax(l / tau), lse = log sum exp(l / tau)
//   balance = coef mean_s sum_e (E c_se / (k n_s)) P_se,   P_se = (1/n_s) sum_t p_te
//   z       = coef_z (1/n) sum_t lse_t^2
//   dl_t = (1/tau) [ p (w_s - <w_s, p>) + (2 coef_z / n) lse_t p ],
//          w_se = (coef / S') E c_se / (k n_s^2),   S' sequences with tokens
//
// Three kernels: partial sums over chunks of tokens, their sum per sequence, and
// the total; the backward streams the logits once more.  G lanes hold a token's
// experts (E / G each), so a warp's loads of 32 / G tokens are contiguous.
// Floating sums run in a fixed order (no float atomics); counts use integer
// atomics in shared memory, whose order does not matter.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int THREADS = 256;
constexpr int CHUNK = 256;       // tokens per CTA of the forward's first kernel

// A record holds one (chunk, sequence) pair's sums: E probability sums, n, the sum
// of lse^2, then E counts (int32).  Chunks and sequences both ascend, so pair
// (b, s) has the record b + s of its own: every step to the next pair raises one.
__host__ __device__ inline size_t rec_floats(int E) { return 2 * (size_t)E + 2; }

struct BalArgs {
    const float* logits;
    const int32_t *topk, *seq;
    const float *grad_w, *dloss;
    float *rec, *seqsum, *loss, *pbar, *gw, *dlogits;
    int32_t* counts;
    int* status;
    int T, E, k, S, nchunk;
    float bcoef, zcoef, inv_tau;
};

// sequence s's first token, with offsets that are out of order or range clamped
// (the forward records that); without offsets one sequence
__device__ __forceinline__ int seq_at(const BalArgs& a, int s) {
    if (s <= 0) return 0;
    if (s >= a.S) return a.T;
    return min(max(__ldg(a.seq + s), 0), a.T);
}
// the sequence of token t: the last s with seq_at(s) <= t (offsets ascend)
__device__ __forceinline__ int seq_of(const BalArgs& a, int t) {
    int lo = 0, hi = a.S - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (seq_at(a, mid) <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Softmax of one token over its G lanes; lane holds experts lane, lane + G, ...
// (R of them).  lse = -inf and p = 0 where every logit is -inf.
template <int G, int R>
__device__ __forceinline__ float softmax_row(const float* row, int E, int gl, bool on, float inv_tau,
                                             float (&p)[R], bool& bad) {
    float m = -INFINITY;
    bad = false;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int e = gl + i * G;
        p[i] = on && e < E ? __ldg(row + e) * inv_tau : -INFINITY;
        bad |= isnan(p[i]) || p[i] == INFINITY;
        m = fmaxf(m, p[i]);
    }
    m = group_max<G>(m);
    float z = 0.f;
    const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        p[i] = expf(p[i] - mm);
        z += p[i];
    }
    z = group_sum<G>(z);
    const float iz = z == 0.f ? 0.f : 1.f / z;       // (NaN stays NaN)
#pragma unroll
    for (int i = 0; i < R; ++i) p[i] *= iz;
    return z == 0.f ? -INFINITY : m + logf(z);
}

template <int G, int R>
__global__ void __launch_bounds__(THREADS) balance_partial_kernel(const BalArgs a) {
    pdl_wait();
    pdl_trigger();
    constexpr int TOK = THREADS / G;                 // tokens at a time
    extern __shared__ float sm[];                    // [8 warps][E + 2] sums, [E] counts
    float* wsum = sm;
    int* cnt = reinterpret_cast<int*>(sm + 8 * (a.E + 2));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gl = tid % G, grp = tid / G;
    const int b = blockIdx.x;
    const int t0 = b * CHUNK, t1 = min(a.T, t0 + CHUNK);
    if (b == 0)                                      // offsets: ascending from 0 to T
        for (int s = tid; s <= a.S; s += THREADS)
            if (a.seq) {
                const int v = a.seq[s], nx = s < a.S ? a.seq[s + 1] : a.T;
                if (v > nx || v < 0 || (s == 0 && v != 0) || (s == a.S && v != a.T))
                    set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
            }
    int t = t0;
    for (int s = a.seq ? seq_of(a, t0) : 0; t < t1; ++s) {
        const int end = min(t1, a.seq ? seq_at(a, s + 1) : a.T);
        if (end <= t && s + 1 < a.S) continue;       // (its record is not read)
        const int stop = s + 1 >= a.S ? t1 : end;
        for (int i = tid; i < a.E; i += THREADS) cnt[i] = 0;
        __syncthreads();
        float sum[R], n = 0.f, zz = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) sum[i] = 0.f;
        for (int base = t; base < stop; base += TOK) {
            const int tt = base + grp;
            const bool in = tt < stop;
            const bool on = in && a.topk[(size_t)tt * a.k] >= 0;
            float p[R];
            bool bad;
            const float lse = softmax_row<G, R>(a.logits + (size_t)tt * a.E, a.E, gl, on, a.inv_tau, p, bad);
            if (on) {
                if (bad) set_status(a.status, MOE_ERR_NONFINITE);
#pragma unroll
                for (int i = 0; i < R; ++i) sum[i] += p[i];
                if (gl == 0) {
                    n += 1.f;
                    zz += lse == -INFINITY ? 0.f : lse * lse;
                }
            }
            if (in)
                for (int j = gl; j < a.k; j += G) {
                    const int e = a.topk[(size_t)tt * a.k + j];
                    if (e >= a.E || e < -1) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
                    else if (e >= 0 && on) atomicAdd(cnt + e, 1);
                }
        }
        // over the warp's tokens, then the warps in order
#pragma unroll
        for (int o = 16; o >= G; o >>= 1) {
#pragma unroll
            for (int i = 0; i < R; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
            n += __shfl_xor_sync(0xffffffffu, n, o);
            zz += __shfl_xor_sync(0xffffffffu, zz, o);
        }
        if (lane < G) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (gl + i * G < a.E) wsum[warp * (a.E + 2) + gl + i * G] = sum[i];
            if (lane == 0) {
                wsum[warp * (a.E + 2) + a.E] = n;
                wsum[warp * (a.E + 2) + a.E + 1] = zz;
            }
        }
        __syncthreads();
        float* rec = a.rec + (size_t)(b + s) * rec_floats(a.E);
        for (int i = tid; i < a.E + 2; i += THREADS) {
            float v = 0.f;
            for (int w = 0; w < 8; ++w) v += wsum[w * (a.E + 2) + i];
            rec[i] = v;
        }
        for (int i = tid; i < a.E; i += THREADS) rec[a.E + 2 + i] = __int_as_float(cnt[i]);
        __syncthreads();
        t = stop;
    }
}

// One CTA per sequence: its records in order, in double (up to T / CHUNK of them).
__global__ void __launch_bounds__(THREADS) balance_sequence_kernel(const BalArgs a) {
    pdl_wait();
    pdl_trigger();
    const int s = blockIdx.x, E = a.E;
    const int beg = a.seq ? seq_at(a, s) : 0;
    const int end = s + 1 >= a.S ? a.T : seq_at(a, s + 1);
    const int b0 = beg / CHUNK, b1 = end > beg ? (end - 1) / CHUNK : b0 - 1;
    __shared__ double tot[2];                        // n, sum lse^2
    __shared__ double part[THREADS / 32];
    for (int i = threadIdx.x; i < 2; i += THREADS) {
        double v = 0.0;
        for (int b = b0; b <= b1; ++b) v += a.rec[(size_t)(b + s) * rec_floats(E) + E + i];
        tot[i] = v;
    }
    __syncthreads();
    const double n = tot[0], in = n > 0.0 ? 1.0 / n : 0.0;
    double fp = 0.0;
    for (int e = threadIdx.x; e < E; e += THREADS) {
        double v = 0.0;
        int c = 0;
        for (int b = b0; b <= b1; ++b) {
            const float* r = a.rec + (size_t)(b + s) * rec_floats(E);
            v += r[e];
            c += __float_as_int(r[E + 2 + e]);
        }
        const double P = v * in, f = (double)E * c * in / a.k;
        a.counts[(size_t)s * E + e] = c;
        a.pbar[(size_t)s * E + e] = (float)P;
        a.gw[(size_t)s * (E + 2) + e] = (float)(f * in);   // times coef / S' in the backward
        fp += f * P;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) fp += __shfl_xor_sync(0xffffffffu, fp, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = fp;
    __syncthreads();
    if (threadIdx.x == 0) {
        double v = 0.0;
        for (int w = 0; w < THREADS / 32; ++w) v += part[w];
        a.seqsum[s * 3] = (float)v;
        a.seqsum[s * 3 + 1] = (float)n;
        a.seqsum[s * 3 + 2] = (float)tot[1];
    }
}

// The losses, and the two factors of the backward: coef / S' and 2 coef_z / n,
// written beside every sequence's weights.
__global__ void __launch_bounds__(THREADS) balance_total_kernel(const BalArgs a) {
    pdl_wait();
    pdl_trigger();
    __shared__ double sm[4][THREADS];
    double v[4] = {0, 0, 0, 0};                      // sum f P, sequences, tokens, sum lse^2
    for (int s = threadIdx.x; s < a.S; s += THREADS) {
        v[0] += a.seqsum[s * 3];
        v[1] += a.seqsum[s * 3 + 1] > 0.f;
        v[2] += a.seqsum[s * 3 + 1];
        v[3] += a.seqsum[s * 3 + 2];
    }
    for (int i = 0; i < 4; ++i) sm[i][threadIdx.x] = v[i];
    __syncthreads();
    for (int h = THREADS / 2; h > 0; h >>= 1) {
        if (threadIdx.x < h)
            for (int i = 0; i < 4; ++i) sm[i][threadIdx.x] += sm[i][threadIdx.x + h];
        __syncthreads();
    }
    const double ns = fmax(sm[1][0], 1.0), n = fmax(sm[2][0], 1.0);
    if (threadIdx.x == 0) {
        const double b = a.bcoef * sm[0][0] / ns, z = a.zcoef * sm[3][0] / n;
        a.loss[0] = (float)(b + z);
        a.loss[1] = (float)b;
        a.loss[2] = (float)z;
    }
    for (int s = threadIdx.x; s < a.S; s += THREADS) {
        a.gw[(size_t)s * (a.E + 2) + a.E] = (float)(a.bcoef / ns);
        a.gw[(size_t)s * (a.E + 2) + a.E + 1] = (float)(2.0 * a.zcoef / n);
    }
}

template <int G, int R>
__global__ void __launch_bounds__(THREADS) balance_bwd_kernel(const BalArgs a) {
    pdl_wait();
    pdl_trigger();
    constexpr int TOK = THREADS / G;
    const int gl = threadIdx.x % G, grp = threadIdx.x / G;
    const float up = (a.dloss ? __ldg(a.dloss) : 1.f) * a.inv_tau;
    for (int base = blockIdx.x * TOK; base < a.T; base += gridDim.x * TOK) {
        const int t = base + grp;
        const bool in = t < a.T;
        const bool on = in && a.topk[(size_t)t * a.k] >= 0;
        float p[R], w[R];
        bool bad;
        const float lse = softmax_row<G, R>(a.logits + (size_t)t * a.E, a.E, gl, on, a.inv_tau, p, bad);
        const float* gw = a.grad_w + (size_t)(on && a.seq ? seq_of(a, t) : 0) * (a.E + 2);
        const float cb = __ldg(gw + a.E), cz = __ldg(gw + a.E + 1);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int e = gl + i * G;
            w[i] = e < a.E ? cb * __ldg(gw + e) : 0.f;
            dot = fmaf(w[i], p[i], dot);
        }
        dot = group_sum<G>(dot);
        const float zl = lse == -INFINITY ? 0.f : cz * lse;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int e = gl + i * G;
            if (in && e < a.E) a.dlogits[(size_t)t * a.E + e] = on ? up * (p[i] * (w[i] - dot + zl)) : 0.f;
        }
    }
}

// lanes per token and experts per lane: the fewest lanes that leave a lane at most
// eight experts, at least 4 so that a row's loads stay together
template <template <int, int> class F, class... A>
int by_experts(int E, A&&... args) {
    if (E <= 4) return F<4, 1>::go(args...);
    if (E <= 8) return F<8, 1>::go(args...);
    if (E <= 16) return F<16, 1>::go(args...);
    if (E <= 32) return F<32, 1>::go(args...);
    if (E <= 64) return F<32, 2>::go(args...);
    if (E <= 128) return F<32, 4>::go(args...);
    return F<32, 8>::go(args...);
}

template <int G, int R> struct Partial {
    static int go(const BalArgs& a, cudaStream_t st) {
        const size_t smem = (size_t)(8 * (a.E + 2) + a.E) * 4;
        MOE_LAUNCH((balance_partial_kernel<G, R>), a.nchunk, THREADS, smem, st, a);
        return MOE_OK;
    }
};
template <int G, int R> struct Backward {
    static int go(const BalArgs& a, cudaStream_t st) {
        const int tok = THREADS / G;
        const int grid = std::max(1, std::min((a.T + tok - 1) / tok, 8 * num_sms()));
        MOE_LAUNCH((balance_bwd_kernel<G, R>), grid, THREADS, 0, st, a);
        return MOE_OK;
    }
};

int n_chunks(const moe_balance_config& c) { return (c.T + CHUNK - 1) / CHUNK; }

BalArgs bal_args(const moe_balance_config& c) {
    BalArgs a = {};
    a.T = c.T; a.E = c.E; a.k = c.k; a.S = c.S; a.nchunk = n_chunks(c);
    a.bcoef = c.balance_coef; a.zcoef = c.z_coef;
    a.inv_tau = c.temperature > 0.f ? 1.f / c.temperature : 1.f;
    a.status = device_status_ptr();
    return a;
}

}  // namespace

size_t balance_ws_bytes(const moe_balance_config& c) {
    return align_up((size_t)(n_chunks(c) + c.S) * rec_floats(c.E) * 4) + align_up((size_t)c.S * 12);
}

int launch_balance_loss(const moe_balance_config& c, const float* logits, const int32_t* topk,
                        const int32_t* seq, float* loss, int32_t* counts, float* pbar,
                        float* grad_w, void* ws, cudaStream_t st) {
    BalArgs a = bal_args(c);
    a.logits = logits; a.topk = topk; a.seq = seq; a.loss = loss; a.counts = counts; a.pbar = pbar;
    a.gw = grad_w;
    a.rec = static_cast<float*>(ws);
    a.seqsum = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                        align_up((size_t)(n_chunks(c) + c.S) * rec_floats(c.E) * 4));
    if (const int r = by_experts<Partial>(c.E, a, st)) return r;
    MOE_LAUNCH(balance_sequence_kernel, c.S, THREADS, 0, st, a);
    MOE_LAUNCH(balance_total_kernel, 1, THREADS, 0, st, a);
    return MOE_OK;
}

int launch_balance_loss_backward(const moe_balance_config& c, const float* logits, const int32_t* topk,
                                 const int32_t* seq, const float* grad_w, const float* dloss,
                                 float* dlogits, cudaStream_t st) {
    BalArgs a = bal_args(c);
    a.logits = logits; a.topk = topk; a.seq = seq; a.grad_w = grad_w; a.dloss = dloss; a.dlogits = dlogits;
    return by_experts<Backward>(c.E, a, st);
}

}  // namespace moe
