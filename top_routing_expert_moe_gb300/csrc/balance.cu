// balance.cu -- per-sequence balance loss and z loss of the router, with gradients.
//
//   p = softmax(l / tau), lse = log sum exp(l / tau)
//   balance = coef mean_s sum_e (E c_se / (k n_s)) P_se,   P_se = (1/n_s) sum_t p_te
//   z       = coef_z (1/n) sum_t lse_t^2
//   dl_t = (1/tau) [ p (w_s - <w_s, p>) + (2 coef_z / n) lse_t p ],
//          w_se = (coef / S') E c_se / (k n_s^2),   S' sequences with tokens
//
// Forward: partial sums over chunks of tokens, then one CTA a sequence adds them
// and the last of those forms the losses.  The backward streams the logits once
// more.  G lanes hold a token's experts, 4 or 8 each, so that the softmax needs
// log2(G) shuffles and a warp's loads of 32 / G tokens stay contiguous.  Floating
// sums run in a fixed order (no float atomics); counts use integer atomics in
// shared memory, whose order does not matter.
//
// T = 65536, E = 64, k = 8, 37 sequences: 21 us a pass as a graph, of them about 8 the
// partial sums, 4 the sequences, 7 the backward; the logits' two passes and dlogits
// are 5 us of HBM.  Latency bounds it (each kernel's dependent loads, then half of
// the issue slots for the softmax).  32 lanes a token and 256-token chunks took 80 us.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int THREADS = 256;
constexpr int SEQ_THREADS = 512;
constexpr float LOG2E = 1.44269504f;

// A record holds one (chunk of tokens, sequence) pair's sums: E probability sums, n, the sum
// of lse^2, then E counts (int32).  Chunks and sequences both ascend, so pair
// (b, s) has the record b + s of its own: every step to the next pair raises one.
__host__ __device__ inline size_t rec_floats(int E) { return 2 * (size_t)E + 2; }

struct BalArgs {
    const float* logits;
    const int32_t *topk, *seq;
    const float *grad_w, *dloss;
    float *rec, *seqsum, *loss, *pbar, *gw, *dlogits;
    int32_t* counts;
    unsigned* ticket;                                // [0] CTAs done, [1] the offsets descend
    int* status;
    int T, E, k, S, chunk;                           // tokens of a CTA
    float bcoef, zcoef, inv_tau;
};

// sequence s's first token, with offsets out of range clamped (the forward records
// that, and where they still descend leaves every output zero); without offsets one
// sequence
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

// The same for the whole CTA at once: the offsets at or before t are counted in
// parallel (one memory latency instead of log2(S)) where they are few.
__device__ __forceinline__ int cta_seq_of(const BalArgs& a, int t) {
    if (!a.seq) return 0;
    if (a.S > 8 * THREADS) return seq_of(a, t);
    int n = 0;
    for (int s0 = 0; s0 < a.S; s0 += THREADS) {
        const int s = s0 + threadIdx.x;
        n += __syncthreads_count(s < a.S && seq_at(a, s) <= t);
    }
    return max(n, 1) - 1;
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

// A lane's experts: R in groups of W (4 where E is a multiple of 4: one 16-byte
// access each, else 1), group i at (lane + i G) W.
template <int G, int R, int W> struct Row {
    static constexpr int N = R / W;
    __device__ __forceinline__ static int expert(int gl, int i) { return (gl + (i / W) * G) * W + i % W; }
    __device__ __forceinline__ static void load(const float* row, int E, int gl, bool in, float (&v)[R]) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = (gl + i * G) * W;
            if constexpr (W == 4) {
                const float4 f = in && e < E ? __ldg(reinterpret_cast<const float4*>(row + e))
                                             : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
            } else {
                v[i] = in && e < E ? __ldg(row + e) : -INFINITY;
            }
        }
    }
    __device__ __forceinline__ static void store(float* row, int E, int gl, const float (&v)[R]) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = (gl + i * G) * W;
            if (e >= E) continue;
            if constexpr (W == 4) *reinterpret_cast<float4*>(row + e) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            else row[e] = v[i];
        }
    }
};

// Softmax of one token's logits over its G lanes, in place, in powers of two.  The
// maximum is subtracted before anything is rounded: the difference of near logits is
// exact, so the error of p goes by the distance from the maximum and not by the
// logits' size, and no finite logit leaves the range.  Returns lse (0, with p = 0,
// where every logit is -inf or the token is masked; NaN where one is NaN or +inf).
template <int G, int R>
__device__ __forceinline__ float softmax_row(float (&p)[R], bool on, float inv_tau) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        p[i] = on ? p[i] : -INFINITY;
        m = fmaxf(m, p[i]);
    }
    m = group_max<G>(m);
    float z = 0.f;
    const float mm = m == -INFINITY ? 0.f : m, k2 = inv_tau * LOG2E;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p[i]) : "f"((p[i] - mm) * k2));   // 2 ulp
        z += p[i];
    }
    z = group_sum<G>(z);
    const float iz = z == 0.f ? 0.f : __fdividef(1.f, z);   // (1 <= z <= E, or NaN)
#pragma unroll
    for (int i = 0; i < R; ++i) p[i] *= iz;
    return z == 0.f ? 0.f : m * inv_tau + __logf(z);
}

template <int G, int R, int W>
__global__ void __launch_bounds__(THREADS) balance_partial_kernel(const BalArgs a) {
    pdl_wait();
    pdl_trigger();
    using L = Row<G, R, W>;
    constexpr int TOK = THREADS / G;                 // tokens at a time
    extern __shared__ float sm[];                    // [8 warps][E + 2] sums, [E] counts
    float* wsum = sm;
    int* cnt = reinterpret_cast<int*>(sm + 8 * (a.E + 2));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gl = tid % G, grp = tid / G;
    const int b = blockIdx.x;
    const int t0 = b * a.chunk, t1 = min(a.T, t0 + a.chunk);
    if (b == 0) {
        int down = 0;
        if (a.seq)                                   // offsets: ascending from 0 to T
            for (int s = tid; s <= a.S; s += THREADS) {
                const int v = a.seq[s], nx = s < a.S ? a.seq[s + 1] : a.T;
                if (v > nx || v < 0 || (s == 0 && v != 0) || (s == a.S && v != a.T))
                    set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
                // (pairs of chunks and sequences are then no staircase, and records that
                // the next kernel would read are not written)
                if (s < a.S && seq_at(a, s) > seq_at(a, s + 1)) down = 1;
            }
        down = __syncthreads_or(down);
        if (tid == 0) {
            a.ticket[0] = 0;
            a.ticket[1] = down;
        }
    }
    int t = t0;
    // a token's logits are loaded while the one before is worked on
    float nxt[R];
    int32_t nxt_pick = -1;
    auto fetch = [&](int tt) {
        L::load(a.logits + (size_t)tt * a.E, a.E, gl, tt < t1, nxt);
        nxt_pick = tt < t1 ? __ldg(a.topk + (size_t)tt * a.k) : -1;
    };
    fetch(t0 + grp);
    for (int s = cta_seq_of(a, t0); t < t1; ++s) {
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
            float p[R];
#pragma unroll
            for (int i = 0; i < R; ++i) p[i] = nxt[i];
            const int32_t* pick = a.topk + (size_t)tt * a.k;
            const bool on = in && nxt_pick >= 0;
            // the pass's tokens past a sequence's end are its successor's first pass
            fetch((base + TOK < stop ? base + TOK : stop) + grp);
            const float lse = softmax_row<G, R>(p, on, a.inv_tau);
            if (on) {
                if (isnan(lse)) set_status(a.status, MOE_ERR_NONFINITE);
#pragma unroll
                for (int i = 0; i < R; ++i) sum[i] += p[i];
                if (gl == 0) {
                    n += 1.f;
                    zz += lse * lse;
                }
            }
            if (in)
                for (int j = gl; j < a.k; j += G) {
                    const int e = __ldg(pick + j);
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
                if (L::expert(gl, i) < a.E) wsum[warp * (a.E + 2) + L::expert(gl, i)] = sum[i];
            if (lane == 0) {
                wsum[warp * (a.E + 2) + a.E] = n;
                wsum[warp * (a.E + 2) + a.E + 1] = zz;
            }
        }
        __syncthreads();
        float* rec = a.rec + (size_t)(b + s) * rec_floats(a.E);
        for (int i = tid; i < a.E + 2; i += THREADS) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) v += wsum[w * (a.E + 2) + i];
            rec[i] = v;
        }
        for (int i = tid; i < a.E; i += THREADS) rec[a.E + 2 + i] = __int_as_float(cnt[i]);
        __syncthreads();
        t = stop;
    }
}

// One CTA per sequence adds its records: P groups of threads take every P-th one
// (P a power of two), then the groups' sums are added pairwise.  The last CTA to
// finish adds the sequences and writes the losses and the backward's two factors,
// coef / S' and 2 coef_z / n.
__host__ __device__ inline int seq_groups(int E) {
    int P = 1;
    while (2 * P * (E + 2) <= SEQ_THREADS) P *= 2;
    return P;
}
__global__ void __launch_bounds__(SEQ_THREADS) balance_sequence_kernel(const BalArgs a) {
    pdl_wait();
    pdl_trigger();
    const int s = blockIdx.x, E = a.E, W = E + 2, tid = threadIdx.x;
    const unsigned down = __ldcg(a.ticket + 1);
    const int beg = a.seq ? seq_at(a, s) : 0;
    const int end = s + 1 >= a.S ? a.T : seq_at(a, s + 1);
    const int b0 = beg / a.chunk, b1 = end > beg && !down ? (end - 1) / a.chunk : b0 - 1;
    extern __shared__ float sd[];                    // [P][W] sums, then [P][E] counts
    const int P = seq_groups(E);
    int* sc = reinterpret_cast<int*>(sd + P * W);
    __shared__ float part[SEQ_THREADS / 32];
    const int col = tid % W, g = tid / W;
    if (g < P) {
        float v = 0.f;
        int c = 0;
#pragma unroll 4
        for (int b = b0 + g; b <= b1; b += P) {
            const float* r = a.rec + (size_t)(b + s) * rec_floats(E);
            v += r[col];
            if (col < E) c += __float_as_int(r[W + col]);
        }
        sd[g * W + col] = v;
        if (col < E) sc[g * E + col] = c;
    }
    __syncthreads();
    for (int h = P / 2; h > 0; h >>= 1) {
        if (g < h) {
            sd[g * W + col] += sd[(g + h) * W + col];
            if (col < E) sc[g * E + col] += sc[(g + h) * E + col];
        }
        __syncthreads();
    }
    const float n = sd[E], zz = sd[E + 1], in = n > 0.f ? 1.f / n : 0.f;
    float fp = 0.f;
    if (tid < E) {
        const float p = sd[tid] * in, f = (float)E * (float)sc[tid] * in / (float)a.k;
        a.counts[(size_t)s * E + tid] = sc[tid];
        a.pbar[(size_t)s * E + tid] = p;
        a.gw[(size_t)s * W + tid] = f * in;          // times coef / S' in the backward
        fp = f * p;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) fp += __shfl_xor_sync(0xffffffffu, fp, o);
    if ((tid & 31) == 0) part[tid >> 5] = fp;
    __syncthreads();
    __shared__ unsigned order;
    if (tid == 0) {
        float v = 0.f;
        for (int w = 0; w < SEQ_THREADS / 32; ++w) v += part[w];
        a.seqsum[s * 3] = v;
        a.seqsum[s * 3 + 1] = n;
        a.seqsum[s * 3 + 2] = zz;
        __threadfence();
        order = atomicAdd(a.ticket, 1u);
    }
    __syncthreads();
    if (order != (unsigned)a.S - 1) return;
    __threadfence();
    float v[4] = {0.f, 0.f, 0.f, 0.f};               // sum f P, sequences, tokens, sum lse^2
    for (int i = tid; i < a.S; i += SEQ_THREADS) {
        v[0] += __ldcg(a.seqsum + i * 3);
        const float ni = __ldcg(a.seqsum + i * 3 + 1);
        v[1] += ni > 0.f;
        v[2] += ni;
        v[3] += __ldcg(a.seqsum + i * 3 + 2);
    }
    __shared__ float tot[4][SEQ_THREADS / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if ((tid & 31) == 0) tot[i][tid >> 5] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = 0.f;
        for (int w = 0; w < SEQ_THREADS / 32; ++w) v[i] += tot[i][w];
    }
    const float ns = fmaxf(v[1], 1.f), nt = fmaxf(v[2], 1.f);
    if (tid == 0) {
        // (lse^2 of the largest logits is infinite; without a z loss that is no matter)
        const float b = a.bcoef * v[0] / ns, z = a.zcoef == 0.f ? 0.f : a.zcoef * v[3] / nt;
        a.loss[0] = b + z;
        a.loss[1] = b;
        a.loss[2] = z;
    }
    for (int i = tid; i < a.S; i += SEQ_THREADS) {
        a.gw[(size_t)i * W + E] = a.bcoef / ns;
        a.gw[(size_t)i * W + E + 1] = down ? 0.f : 2.f * a.zcoef / nt;
    }
}

template <int G, int R, int W>
__global__ void __launch_bounds__(THREADS) balance_bwd_kernel(const BalArgs a) {
    pdl_wait();
    pdl_trigger();
    using L = Row<G, R, W>;
    constexpr int TOK = THREADS / G;
    const int gl = threadIdx.x % G, grp = threadIdx.x / G;
    const float up = (a.dloss ? __ldg(a.dloss) : 1.f) * a.inv_tau;
    const int t0 = blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
    // the sequence of this group's token, its end and its weights; they ascend with t
    int end = -1;
    float w[R], cz = 0.f, nxt[R];
    int32_t nxt_pick = -1;
    auto fetch = [&](int tt) {
        L::load(a.logits + (size_t)tt * a.E, a.E, gl, tt < t1, nxt);
        nxt_pick = tt < t1 ? __ldg(a.topk + (size_t)tt * a.k) : -1;
    };
    fetch(t0 + grp);
    int s = cta_seq_of(a, t0);
    for (int base = t0; base < t1; base += TOK) {
        const int t = base + grp;
        const bool in = t < t1;
        float p[R];
#pragma unroll
        for (int i = 0; i < R; ++i) p[i] = nxt[i];
        const bool on = nxt_pick >= 0;
        fetch(t + TOK);
        if (in && t >= end) {
            while (s + 1 < a.S && seq_at(a, s + 1) <= t) ++s;
            end = s + 1 < a.S ? seq_at(a, s + 1) : a.T;
            const float* gw = a.grad_w + (size_t)s * (a.E + 2);
            const float cb = __ldg(gw + a.E);
            cz = __ldg(gw + a.E + 1);
#pragma unroll
            for (int i = 0; i < R; ++i) w[i] = L::expert(gl, i) < a.E ? cb * __ldg(gw + L::expert(gl, i)) : 0.f;
        }
        const float lse = softmax_row<G, R>(p, on, a.inv_tau);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) dot = fmaf(on ? w[i] : 0.f, p[i], dot);
        dot = group_sum<G>(dot);
        const float zl = cz == 0.f ? 0.f : cz * lse;
#pragma unroll
        for (int i = 0; i < R; ++i) p[i] = on ? up * (p[i] * (w[i] - dot + zl)) : 0.f;
        if (in) L::store(a.dlogits + (size_t)t * a.E, a.E, gl, p);
    }
}

// Lanes per token: the fewest that leave each at most eight experts.
template <template <int, int, int> class F, class... A>
int by_experts(int E, A&&... args) {
    if (E % 4 == 0) {
        if (E <= 4) return F<1, 4, 4>::go(args...);
        if (E <= 8) return F<2, 4, 4>::go(args...);
        if (E <= 16) return F<4, 4, 4>::go(args...);
        if (E <= 32) return F<4, 8, 4>::go(args...);
        if (E <= 64) return F<8, 8, 4>::go(args...);
        if (E <= 128) return F<16, 8, 4>::go(args...);
        return F<32, 8, 4>::go(args...);
    }
    if (E <= 8) return F<2, 4, 1>::go(args...);
    if (E <= 16) return F<4, 4, 1>::go(args...);
    if (E <= 32) return F<4, 8, 1>::go(args...);
    if (E <= 64) return F<8, 8, 1>::go(args...);
    if (E <= 128) return F<16, 8, 1>::go(args...);
    return F<32, 8, 1>::go(args...);
}

// Tokens of a CTA: about four CTAs an SM, but whole passes (THREADS / G tokens), at
// most 512 tokens, and no fewer than 32 (a chunk's record is 2 E + 2 words).
int chunk_of(const moe_balance_config& c) {
    const int g = c.E <= 4 && c.E % 4 == 0 ? 1 : c.E <= 8 ? 2 : c.E <= 32 ? 4 : c.E <= 64 ? 8 : c.E <= 128 ? 16 : 32;
    const int pass = std::max(32, THREADS / g);
    const int want = (c.T + 4 * num_sms() - 1) / (4 * num_sms());
    return std::min(512, std::max(1, (want + pass - 1) / pass) * pass);
}
int n_chunks(const moe_balance_config& c) { return (c.T + chunk_of(c) - 1) / chunk_of(c); }

template <int G, int R, int W> struct Partial {
    static int go(const BalArgs& a, cudaStream_t st) {
        const size_t smem = (size_t)(8 * (a.E + 2) + a.E) * 4;
        MOE_LAUNCH((balance_partial_kernel<G, R, W>), (a.T + a.chunk - 1) / a.chunk, THREADS, smem, st, a);
        return MOE_OK;
    }
};
template <int G, int R, int W> struct Backward {
    static int go(const BalArgs& a, cudaStream_t st) {
        MOE_LAUNCH((balance_bwd_kernel<G, R, W>), (a.T + a.chunk - 1) / a.chunk, THREADS, 0, st, a);
        return MOE_OK;
    }
};

size_t rec_bytes(const moe_balance_config& c) { return align_up((size_t)(n_chunks(c) + c.S) * rec_floats(c.E) * 4); }

BalArgs bal_args(const moe_balance_config& c) {
    BalArgs a = {};
    a.T = c.T; a.E = c.E; a.k = c.k; a.S = c.S; a.chunk = chunk_of(c);
    a.bcoef = c.balance_coef; a.zcoef = c.z_coef;
    a.inv_tau = c.temperature > 0.f ? 1.f / c.temperature : 1.f;
    a.status = device_status_ptr();
    return a;
}

}  // namespace

size_t balance_ws_bytes(const moe_balance_config& c) {
    return rec_bytes(c) + align_up((size_t)c.S * 12) + 256;
}

int launch_balance_loss(const moe_balance_config& c, const float* logits, const int32_t* topk,
                        const int32_t* seq, float* loss, int32_t* counts, float* pbar,
                        float* grad_w, void* ws, cudaStream_t st) {
    BalArgs a = bal_args(c);
    a.logits = logits; a.topk = topk; a.seq = seq; a.loss = loss; a.counts = counts; a.pbar = pbar;
    a.gw = grad_w;
    a.rec = static_cast<float*>(ws);
    a.seqsum = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + rec_bytes(c));
    a.ticket = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(ws) + rec_bytes(c) + align_up((size_t)c.S * 12));
    if (const int r = by_experts<Partial>(c.E, a, st)) return r;
    MOE_LAUNCH(balance_sequence_kernel, c.S, SEQ_THREADS, (size_t)seq_groups(c.E) * (2 * c.E + 2) * 4, st, a);
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
