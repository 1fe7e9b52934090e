// norm.cu -- the residual stream's norms around a block, forward and backward.
//
//   leave:  n = w_post u r_u (or u),  x' = a x + b g n     r_v = 1/sqrt(mean v^2 + eps)
//   enter:  z = w_pre x' r
// A row belongs to one group of threads, so each tensor passes through HBM once.
// All sums are fp32.
//
// Backward, for one row, with G the gradient of x':
//   a_i = w_pre dz,  G = dx' + r a - x' (r^3/d) A,            A   = sum a x'
//   q   = b g w_post (1 for an absent factor),  dn w_post = q G
//   du  = r_u q G - u (r_u^3/d) S,                            S   = sum q u G
// S is linear in G, so it comes from the first pass's sums,
//   S = sum q u dx' + r sum q u a - (r^3/d) A sum q u x',
// and one reduction of six sums serves the whole row.  r^3 is never formed by itself:
// it leaves fp32's range where r passes 1e12 or 1e-13, and the row's sum brings it back.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "ring_cursor.h"
#include "tma.cuh"

namespace moe {

namespace {

constexpr int SMALL_ROWS = 4;    // rows per CTA when a warp holds a row

// Sums over the threads of a row: a warp, or the whole CTA through shared memory
// (buf: 32 x 8 floats; the caller alternates two buffers, so one barrier a call
// is enough).  Fixed order.
__device__ __forceinline__ float row_sum(float v, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (blockDim.x <= 32) return v;
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < nw ? buf[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Six sums at once, in two steps around a CTA barrier.  Within a warp the first
// three steps of the butterfly halve the values a lane carries as they double the
// lanes it stands for, so that four lanes end with one value's sum: 9 shuffles
// instead of 30.  Then every warp adds the warps' sums from shared memory.
__device__ __forceinline__ float warp_sums6(const float (&s)[6]) {
    const int lane = threadIdx.x & 31;
    const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
    float a[4], b[2], v;
    const float s8[8] = {s[0], s[1], s[2], s[3], s[4], s[5], 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a[i] = (b4 ? s8[i + 4] : s8[i]) + __shfl_xor_sync(0xffffffffu, b4 ? s8[i] : s8[i + 4], 16);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        b[i] = (b3 ? a[i + 2] : a[i]) + __shfl_xor_sync(0xffffffffu, b3 ? a[i] : a[i + 2], 8);
    v = (b2 ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, b2 ? b[0] : b[1], 4);
    v += __shfl_xor_sync(0xffffffffu, v, 2);
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v;                                                // the sum of value lane / 4
}
__device__ __forceinline__ void put_sums6(float v, float* buf) {
    const int lane = threadIdx.x & 31;
    if ((lane & 3) == 0) buf[(threadIdx.x >> 5) * 8 + (lane >> 2)] = v;
}
__device__ __forceinline__ void get_sums6(float (&s)[6], const float* buf) {
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    float v = 0.f;
    for (int w = lane >> 3; w < nw; w += 4) v += buf[w * 8 + (lane & 7)];
    v += __shfl_xor_sync(0xffffffffu, v, 8);
    v += __shfl_xor_sync(0xffffffffu, v, 16);                // value lane % 8
#pragma unroll
    for (int i = 0; i < 6; ++i) s[i] = __shfl_sync(0xffffffffu, v, i);
}
// in one call; rows of a warp need no barrier
__device__ __forceinline__ void row_sums6(float (&s)[6], float* buf) {
    const float v = warp_sums6(s);
    if (blockDim.x > 32) {
        put_sums6(v, buf);
        __syncthreads();
        get_sums6(s, buf);
        return;
    }
#pragma unroll
    for (int i = 0; i < 6; ++i) s[i] = __shfl_sync(0xffffffffu, v, i * 4);
}

// ---------------------------------------------------------------- rows read directly
// For short batches and very wide rows.  A thread's share: vectors tid, tid +
// threads, ... of VEC elements (1 for rows of no whole 16 bytes), EPT in all.
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, int c, int nvec, float (&v)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = 0.f;
    if (c >= nvec) return;
    if constexpr (VEC == 1) v[0] = to_f<T>(p[c]);
    else if constexpr (VEC * sizeof(T) == 32) {                  // 8 fp32 of a channel vector
        load16_f<T>(p + c * VEC, v);
        load16_f<T>(p + c * VEC + 4, v + 4);
    } else load16_f<T>(p + c * VEC, v);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, int c, int nvec, const float (&v)[VEC]) {
    if (c >= nvec) return;
    if constexpr (VEC == 1) p[c] = from_f<T>(v[0]);
    else store16_f<T>(p + c * VEC, v);
}

struct NormArgs {
    const void *x, *u, *gate, *dx_out, *dz;   // x: the stream (x_out in the backward)
    const float *w_post, *w_pre;
    void *x_out, *z, *dx, *du, *dgate;
    float *part;                              // [3][grid][d]: dw_pre, dw_post, dgate partials
    int T, d, leave, post, enter, gmode;
    float eps, ra, ob;
};

template <typename T, int VEC, int EPT, int MAXT>
__global__ void __launch_bounds__(MAXT) block_norm_kernel(const NormArgs a) {
    pdl_wait();
    pdl_trigger();
    constexpr int NC = EPT / VEC;
    __shared__ float buf[2][32];
    const int nvec = a.d / VEC;
    const float invd = 1.f / (float)a.d;
    for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < a.T;
         t += (int64_t)gridDim.x * blockDim.y) {
        const size_t o = (size_t)t * a.d;
        float y[NC][VEC], u[NC][VEC], w[VEC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            load_vec<T, VEC>(static_cast<const T*>(a.x) + o, c, nvec, y[i]);
            if (a.leave) load_vec<T, VEC>(static_cast<const T*>(a.u) + o, c, nvec, u[i]);
        }
        if (a.leave) {
            float f = a.ob;
            if (a.gmode == MOE_GATE_TOKEN) f *= static_cast<const float*>(a.gate)[t];
            if (a.post) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < NC; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) s = fmaf(u[i][j], u[i][j], s);
                f *= rsqrtf(row_sum(s, buf[0]) * invd + a.eps);
            }
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                if (a.post) {
                    load_vec<float, VEC>(a.w_post, c, nvec, w);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) u[i][j] *= w[j];
                }
                if (a.gmode == MOE_GATE_CHANNEL || a.gmode == MOE_GATE_FULL) {
                    if (a.gmode == MOE_GATE_CHANNEL)
                        load_vec<float, VEC>(static_cast<const float*>(a.gate), c, nvec, w);
                    else load_vec<T, VEC>(static_cast<const T*>(a.gate) + o, c, nvec, w);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) u[i][j] *= w[j];
                }
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[i][j] = fmaf(a.ra, y[i][j], f * u[i][j]);
                store_vec<T, VEC>(static_cast<T*>(a.x_out) + o, c, nvec, y[i]);
            }
        }
        if (a.enter) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) s = fmaf(y[i][j], y[i][j], s);
            const float r = rsqrtf(row_sum(s, buf[1]) * invd + a.eps);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                load_vec<float, VEC>(a.w_pre, c, nvec, w);
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[i][j] *= r * w[j];
                store_vec<T, VEC>(static_cast<T*>(a.z) + o, c, nvec, y[i]);
            }
        }
        // buf[0] and buf[1] alternate unless only one of the norms is on
        if (a.post != a.enter && blockDim.x > 32) __syncthreads();
    }
}

// The row is read twice, for the sums and for the outputs (the second time from the
// caches): the channel sums leave no registers to hold it.
template <typename T, int VEC, int EPT, int MAXT>
__global__ void __launch_bounds__(MAXT) block_norm_bwd_kernel(const NormArgs a) {
    pdl_wait();
    pdl_trigger();
    constexpr int NC = EPT / VEC;
    __shared__ float buf[2][32 * 8];
    extern __shared__ float comb[];            // [SMALL_ROWS][d] when a CTA holds several rows
    const int nvec = a.d / VEC;
    const float invd = 1.f / (float)a.d;
    float acc_pre[NC][VEC], acc_post[NC][VEC], acc_g[NC][VEC];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc_pre[i][j] = acc_post[i][j] = acc_g[i][j] = 0.f;
    const bool need_u = a.leave && (a.post || a.gmode != MOE_GATE_NONE);
    int par = 0;
    for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < a.T;
         t += (int64_t)gridDim.x * blockDim.y, par ^= 1) {
        const size_t o = (size_t)t * a.d;
        float tok = a.ob;
        if (a.gmode == MOE_GATE_TOKEN) tok *= static_cast<const float*>(a.gate)[t];
        // one chunk: x', dz, dx', u, w_pre, w_post, gate (a token's gate is in tok)
        auto load = [&](int i, float (&y)[VEC], float (&dz)[VEC], float (&G)[VEC], float (&u)[VEC],
                        float (&wz)[VEC], float (&wq)[VEC], float (&g)[VEC]) {
            const int c = threadIdx.x + i * blockDim.x;
#pragma unroll
            for (int j = 0; j < VEC; ++j) { y[j] = dz[j] = G[j] = u[j] = wz[j] = 0.f; wq[j] = g[j] = 1.f; }
            if (a.enter) {
                load_vec<T, VEC>(static_cast<const T*>(a.x) + o, c, nvec, y);
                load_vec<T, VEC>(static_cast<const T*>(a.dz) + o, c, nvec, dz);
                load_vec<float, VEC>(a.w_pre, c, nvec, wz);
            }
            if (a.dx_out) load_vec<T, VEC>(static_cast<const T*>(a.dx_out) + o, c, nvec, G);
            if (need_u) load_vec<T, VEC>(static_cast<const T*>(a.u) + o, c, nvec, u);
            if (a.post) load_vec<float, VEC>(a.w_post, c, nvec, wq);
            if (a.gmode == MOE_GATE_CHANNEL) load_vec<float, VEC>(static_cast<const float*>(a.gate), c, nvec, g);
            else if (a.gmode == MOE_GATE_FULL) load_vec<T, VEC>(static_cast<const T*>(a.gate) + o, c, nvec, g);
        };
        // s: y^2, a y, u^2, q u dx', q u a, q u y  with a = w_pre dz, q = g w_post
        float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float y[VEC], dz[VEC], G[VEC], u[VEC], wz[VEC], wq[VEC], g[VEC];
            load(i, y, dz, G, u, wz, wq, g);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float az = wz[j] * dz[j], qu = wq[j] * g[j] * u[j];
                s[0] = fmaf(y[j], y[j], s[0]);
                s[1] = fmaf(az, y[j], s[1]);
                s[2] = fmaf(u[j], u[j], s[2]);
                s[3] = fmaf(qu, G[j], s[3]);
                s[4] = fmaf(qu, az, s[4]);
                s[5] = fmaf(qu, y[j], s[5]);
            }
        }
        row_sums6(s, buf[par]);
        const float r = a.enter ? rsqrtf(s[0] * invd + a.eps) : 0.f;
        const float ca = r * (r * (r * (invd * s[1])));
        const float S = s[3] + r * s[4] - ca * s[5];         // sum q u G, without tok
        const float ru = a.post ? rsqrtf(s[2] * invd + a.eps) : 1.f;
        const float cu = a.post ? tok * ru * (ru * (ru * (invd * S))) : 0.f;
        if (a.gmode == MOE_GATE_TOKEN && threadIdx.x == 0)
            static_cast<float*>(a.dgate)[t] = a.ob * ru * S;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            float y[VEC], dz[VEC], G[VEC], u[VEC], wz[VEC], wq[VEC], g[VEC], out[VEC];
            load(i, y, dz, G, u, wz, wq, g);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                G[j] += r * (wz[j] * dz[j]) - ca * y[j];
                acc_pre[i][j] = fmaf(dz[j], r * y[j], acc_pre[i][j]);
                out[j] = a.leave ? a.ra * G[j] : G[j];
            }
            store_vec<T, VEC>(static_cast<T*>(a.dx) + o, c, nvec, out);
            if (!a.leave) continue;
            if (a.gmode == MOE_GATE_FULL) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) out[j] = a.ob * G[j] * (wq[j] * u[j] * ru);
                store_vec<T, VEC>(static_cast<T*>(a.dgate) + o, c, nvec, out);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float h = tok * ru * G[j];
                acc_post[i][j] = fmaf(g[j] * h, u[j], acc_post[i][j]);
                acc_g[i][j] = fmaf(wq[j] * h, u[j], acc_g[i][j]);
                out[j] = wq[j] * g[j] * h - cu * u[j];
            }
            store_vec<T, VEC>(static_cast<T*>(a.du) + o, c, nvec, out);
        }
    }
    // this CTA's partial sums of the channel gradients
    auto flush = [&](int which, const float (&acc)[NC][VEC]) {
        float* dst = a.part + ((size_t)which * gridDim.x + blockIdx.x) * a.d;
        float* to = blockDim.y == 1 ? dst : comb + threadIdx.y * a.d;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < nvec)
#pragma unroll
                for (int j = 0; j < VEC; ++j) to[c * VEC + j] = acc[i][j];
        }
        if (blockDim.y == 1) return;
        __syncthreads();
        for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < a.d; c += blockDim.x * blockDim.y) {
            float v = comb[c];
            for (int y = 1; y < (int)blockDim.y; ++y) v += comb[y * a.d + c];
            dst[c] = v;
        }
        __syncthreads();
    };
    if (a.enter) flush(0, acc_pre);
    if (a.post) flush(1, acc_post);
    if (a.gmode == MOE_GATE_CHANNEL) flush(2, acc_g);
}

// ---------------------------------------------------------------- rows through a ring
// Long batches.  A CTA is one row wide (8 elements a thread) and persistent; its
// rows' tensors arrive by bulk copies in a ring of shared-memory stages, so loads
// run ahead of the two dependent phases of a row (sums, then outputs) that kept
// registers and memory waiting on each other; the vectors over the channels stay in
// registers.  A row's last barrier also tells that its stage has been read and may
// be filled again.  A copy that never arrives is given up after the bounded wait
// (recorded; the outputs are then undefined).
//
// 65536 x 4096 bf16, both norms, channel gate: forward 324 us (6.6 TB/s, 0.99 of the
// copy rate; the direct kernel 526), backward 531 us (6.1 TB/s, 0.91; 1750).
// 65536 x 2048 fp32: 343 us (6.3 TB/s) and 472 us (6.8 TB/s).
constexpr int RE = 8;                      // elements of a row per thread
constexpr int MAX_STAGES = 8;

// bytes of a staged row: whole 16s, around any shift
__host__ __device__ inline uint32_t row_pitch(uint32_t row_bytes) {
    return row_bytes % 16 == 0 ? row_bytes : (row_bytes + 30) / 16 * 16;
}

struct RingArgs {
    NormArgs n;
    const void* in[5];                     // the rows' tensors, in the stage's order
    int nin, stages;
    int* status;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Elements in pairs: one packed instruction does two fp32 operations, and these
// kernels are bound by the instructions they issue before they are by HBM.
struct f2 { uint64_t v; };
__device__ __forceinline__ f2 pk(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpk(f2 a, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v)); }
__device__ __forceinline__ f2 operator*(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ f2 both(float x) { return pk(x, x); }
__device__ __forceinline__ float sum2(f2 a) {
    float lo, hi;
    unpk(a, lo, hi);
    return lo + hi;
}
constexpr int RP = RE / 2;                 // pairs a thread

// A thread's 8 elements of a row.  WIDE (rows of whole 16 bytes): one 16-byte
// piece of bf16, or one of each half of an fp32 row, so that neighbouring threads'
// accesses stay neighbours.  Otherwise elements tid, tid + threads, ...
template <typename T>
__device__ __forceinline__ int part_of(int half) { return (threadIdx.x + half * blockDim.x) * (16 / (int)sizeof(T)); }
template <typename T, bool WIDE>
__device__ __forceinline__ void take(const T* p, int d, f2 (&v)[RP]) {
    if constexpr (!WIDE) {
        float f[RE];
#pragma unroll
        for (int j = 0; j < RE; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            f[j] = c < d ? to_f<T>(p[c]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < RP; ++i) v[i] = pk(f[2 * i], f[2 * i + 1]);
    } else if constexpr (sizeof(T) == 2) {
        // threads past the row's end read its last elements; sums and stores leave them out
        const uint4 u = *reinterpret_cast<const uint4*>(p + min((int)threadIdx.x * RE, d - RE));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < RP; ++i) v[i] = pk(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = part_of<T>(h);
            const float4 f = c < d ? *reinterpret_cast<const float4*>(p + c) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[2 * h] = pk(f.x, f.y);
            v[2 * h + 1] = pk(f.z, f.w);
        }
    }
}
// This thread's share of a sum: its own, or none where it has read again what belongs
// to others (other shares past the end are zeros).  Chosen, not multiplied by 0: the
// elements read again may be infinite, or their squares.
template <typename T, bool WIDE>
__device__ __forceinline__ bool live(int d) { return !WIDE || sizeof(T) == 4 || (int)threadIdx.x * RE < d; }
template <typename T, bool WIDE>
__device__ __forceinline__ void give(T* p, int d, const f2 (&v)[RP]) {
    if constexpr (!WIDE) {
#pragma unroll
        for (int i = 0; i < RP; ++i) {
            float lo, hi;
            unpk(v[i], lo, hi);
            const int c = threadIdx.x + 2 * i * blockDim.x;
            if (c < d) p[c] = from_f<T>(lo);
            if (c + (int)blockDim.x < d) p[c + blockDim.x] = from_f<T>(hi);
        }
    } else {
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int h = 0; h < RE / V; ++h) {
            const int c = part_of<T>(h);
            float f[V];
#pragma unroll
            for (int j = 0; j < V / 2; ++j) unpk(v[h * V / 2 + j], f[2 * j], f[2 * j + 1]);
            if (c < d) store16_f<T>(p + c, f);
        }
    }
}
// the fp32 channel vector's share that goes with it
template <typename T, bool WIDE>
__device__ __forceinline__ void channel(const float* p, int d, f2 (&v)[RP]) {
    constexpr int V = WIDE ? 16 / sizeof(T) : 1;
    float f[RE];
#pragma unroll
    for (int j = 0; j < RE; ++j) {
        const int c = WIDE ? part_of<T>(j / V) + j % V : threadIdx.x + j * blockDim.x;
        f[j] = c < d ? __ldg(p + c) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < RP; ++i) v[i] = pk(f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ void fill(f2 (&v)[RP], float x) {
#pragma unroll
    for (int i = 0; i < RP; ++i) v[i] = both(x);
}
__device__ __forceinline__ float dot2(const f2 (&a)[RP], const f2 (&b)[RP]) {
    f2 s = a[0] * b[0];
#pragma unroll
    for (int i = 1; i < RP; ++i) s = fma2(a[i], b[i], s);
    return sum2(s);
}

// The parts of a pass, known at compile time for the usual forms: registers and
// issue slots that the other parts would take are what these kernels are short of
// (65536 x 4096, both norms, backward: 702 us with run-time flags, 531 so; 16384 x 8192
// 596 and 274).  A full gate stays with the flags: 449 us forward, 773 backward (5.6
// TB/s); above 512 threads its backward spills (16384 x 8192: 885 us, 2.4 TB/s).
enum Form {
    FORM_ANY,        // by the run-time flags
    FORM_BOTH,       // leave with its norm, enter; a gate that is not full; dx_out given
    FORM_ADD,        // leave without norm or gate, enter; dx_out given
    FORM_ENTER,      // enter alone; dx_out given
    FORM_LEAVE,      // leave with its norm, no enter; a gate that is not full
};
struct Parts { bool leave, post, enter, full, along; };
template <int FORM>
__device__ __forceinline__ Parts parts_of(const NormArgs& n) {
    if constexpr (FORM == FORM_BOTH) return {true, true, true, false, true};
    if constexpr (FORM == FORM_ADD) return {true, false, true, false, true};
    if constexpr (FORM == FORM_ENTER) return {false, false, true, false, true};
    if constexpr (FORM == FORM_LEAVE) return {true, true, false, false, true};
    return {n.leave != 0, n.post != 0, n.enter != 0, n.gmode == MOE_GATE_FULL, n.dx_out != nullptr};
}
inline Form form_of(const NormArgs& n, bool backward) {
    if (n.gmode == MOE_GATE_FULL || (backward && !n.dx_out)) return FORM_ANY;
    if (n.leave && n.post) return n.enter ? FORM_BOTH : FORM_LEAVE;
    if (!n.leave) return FORM_ENTER;
    return n.enter && n.gmode == MOE_GATE_NONE ? FORM_ADD : FORM_ANY;
}

// Rows blockIdx.x + i gridDim.x pass through the stages in turn; the cursor follows
// the row being worked on.  One warp watches the barriers: it waits
// for the next row's stage before it joins the current row's last reduction, whose
// CTA barrier then tells the others.
//
// A copy starts and ends on 16 bytes.  A row that does not is copied with the bytes
// around it and read at its shift; the batch's last bytes, where that would pass
// the tensor's end, are stored by the copying thread itself (a barrier follows
// before they are read).
template <bool WIDE> struct RowRing : RingCursor {
    uint32_t base, bar0, row_bytes, pitch, stage_bytes;
    volatile int* abort_flag;
    volatile uint32_t* stop;               // rows from it on are not sent for

    __device__ __forceinline__ uint32_t shift(int64_t row) const { return (uint32_t)((uint64_t)row * row_bytes) & 15u; }
    __device__ __forceinline__ void issue(const RingArgs& a, uint8_t* smem, int64_t row, int s) const {
        if constexpr (WIDE) {
            mbar_expect_tx(bar0 + s * 8, stage_bytes);
            for (int j = 0; j < a.nin; ++j)
                bulk_load(base + s * stage_bytes + j * pitch, static_cast<const uint8_t*>(a.in[j]) + (size_t)row * row_bytes,
                          row_bytes, bar0 + s * 8);
            return;
        }
        const uint64_t at = (uint64_t)row * row_bytes, from = at & ~15ull, all = (uint64_t)a.n.T * row_bytes;
        uint64_t to = (at + row_bytes + 15) & ~15ull;
        if (to > all) to = all & ~15ull;                 // (the batch's end: below)
        const uint32_t bytes = (uint32_t)(to - from), tail = (uint32_t)(at + row_bytes > to ? at + row_bytes - to : 0);
        mbar_expect_tx(bar0 + s * 8, bytes * a.nin);
        for (int j = 0; j < a.nin; ++j) {
            const uint8_t* src = static_cast<const uint8_t*>(a.in[j]);
            const uint32_t off = s * stage_bytes + j * pitch;
            if (bytes) bulk_load(base + off, src + from, bytes, bar0 + s * 8);
            for (uint32_t i = 0; i < tail; ++i) smem[off + bytes + i] = src[to + i];
        }
    }
    __device__ __forceinline__ void start(const RingArgs& a, uint8_t* smem) const {
        int64_t row = blockIdx.x;
        for (int i = 0; i < stages && row < a.n.T; ++i, row += gridDim.x) issue(a, smem, row, i);
    }
    // While row t is worked on.  The thread that sends for rows stops where a wait of its
    // own gave up: the next would have been t's successor in t's stage.
    __device__ __forceinline__ void wait(const RingArgs& a, int64_t t, int s, uint32_t ph) const {
        if (!mbar_wait(bar0 + s * 8, ph, abort_flag, a.status) && threadIdx.x == 0)
            atomicMin(const_cast<uint32_t*>(stop), (uint32_t)t + stages * gridDim.x);
    }
    // before the row's last barrier: the stage of the k-th row after it (k < stages)
    __device__ __forceinline__ void wait_next(const RingArgs& a, int64_t t, int k = 1) const {
        if (threadIdx.x < 32 && t + (int64_t)k * gridDim.x < a.n.T)
            wait(a, t, ahead(k), phase_ahead(k));
    }
    // after it, by one thread: the stage of the current row t takes a later row
    __device__ __forceinline__ void refill(const RingArgs& a, uint8_t* smem, int64_t t) const {
        const int64_t row = t + (int64_t)stages * gridDim.x;
        if (row < *stop) issue(a, smem, row, slot);
    }
    // after an aborted wait: no copy is in flight when the CTA ends.  (The cursor has gone
    // on over the rows that were not sent for.)
    __device__ __forceinline__ void drain() const {
        const uint32_t sent = (*stop - blockIdx.x + gridDim.x - 1) / gridDim.x;
        for (uint32_t s = 0; s < (uint32_t)stages && s < sent; ++s) mbar_drain(bar0 + s * 8, last_parity(sent, stages, s));
    }
};

#define NORM_RING_SETUP()                                                                       \
    extern __shared__ __align__(128) uint8_t ring_smem[];                                       \
    __shared__ __align__(8) uint64_t bars[MAX_STAGES];                                          \
    __shared__ int abort_s;                                                                     \
    __shared__ uint32_t stop_s;                                                                 \
    const NormArgs& n = a.n;                                                                    \
    const int d = n.d;                                                                          \
    const float invd = 1.f / (float)d;                                                          \
    RowRing<WIDE> ring;                                                                          \
    ring.base = smem_u32(ring_smem);                                                            \
    ring.bar0 = smem_u32(bars);                                                                 \
    ring.row_bytes = (uint32_t)(d * sizeof(T));                                                 \
    ring.pitch = row_pitch(ring.row_bytes);                                                     \
    ring.stage_bytes = ring.pitch * a.nin;                                                      \
    ring.stages = a.stages;                                                                     \
    ring.abort_flag = &abort_s;                                                                 \
    ring.stop = &stop_s;                                                                        \
    if (threadIdx.x == 0) {                                                                     \
        for (int i = 0; i < a.stages; ++i) mbar_init(ring.bar0 + i * 8, 1);                     \
        abort_s = 0;                                                                            \
        stop_s = n.T;                                                                           \
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");                      \
    }                                                                                           \
    __syncthreads();                                                                            \
    pdl_wait();                                                                                 \
    pdl_trigger();                                                                              \
    if (threadIdx.x == 0) ring.start(a, ring_smem);                                             \
    __syncthreads();                                                                            \
    ring.wait(a, blockIdx.x, 0, 0)

// CTAs an SM that the registers have to leave room for (0: no bound), where the compiler's
// own choice is not what the plan below counts on.  Entering alone at odd widths took 53
// registers, a wave of CTAs more than the plan's 40 (20000 x 1001 fp32, 30.5 us; so 27.3).
// Backwards of 513-768 threads have an SM to themselves, but were cut to 40 registers with
// spills for a second CTA (16384 x 5120 bf16, addition 170 us, entering 147; 135 and 125).
template <bool WIDE, int FORM, int MAXT> constexpr int FWD_CTAS = !WIDE && FORM == FORM_ENTER && MAXT == 512 ? 3 : 0;
template <int FORM, int MAXT> constexpr int BWD_CTAS = (FORM == FORM_ADD || FORM == FORM_ENTER) && MAXT == 768 ? 1 : 0;

// in: x, u (leave), gate (full)
template <typename T, bool WIDE, int FORM, int MAXT>
__global__ void __launch_bounds__(MAXT, (FWD_CTAS<WIDE, FORM, MAXT>)) block_norm_ring_kernel(const __grid_constant__ RingArgs a) {
    __shared__ float buf[2][32];
    NORM_RING_SETUP();
    const Parts p = parts_of<FORM>(n);
    const int gmode = FORM == FORM_ADD || FORM == FORM_ENTER ? MOE_GATE_NONE : n.gmode;
    const bool on = live<T, WIDE>(d);
    f2 wq[RP], wz[RP];                     // g w_post, w_pre
    fill(wq, 1.f);
    if (p.post) channel<T, WIDE>(n.w_post, d, wq);
    if (gmode == MOE_GATE_CHANNEL) {
        channel<T, WIDE>(static_cast<const float*>(n.gate), d, wz);
#pragma unroll
        for (int i = 0; i < RP; ++i) wq[i] = wq[i] * wz[i];
    }
    if (p.enter) channel<T, WIDE>(n.w_pre, d, wz);
    // Two norms alternate their buffers, entering alone alternates from row to row, so a
    // row's last reduction is the only barrier that is needed after it.  Leaving with one
    // norm or none meets once more (when it was chosen, 65536 x 4096: plain addition and norm
    // 357 us, without that barrier 386; entering alone 197 with it, 186 without).
    int par = 0;
    for (int64_t t = blockIdx.x; t < n.T; t += gridDim.x, ring.next(), par ^= 1) {
        const uint8_t* st = ring_smem + ring.slot * ring.stage_bytes + (WIDE ? 0u : ring.shift(t));
        auto in = [&](int j) { return reinterpret_cast<const T*>(st + j * ring.pitch); };
        const size_t o = (size_t)t * d;
        float tok = n.ob;
        if (gmode == MOE_GATE_TOKEN) tok *= __ldg(static_cast<const float*>(n.gate) + t);
        f2 y[RP], u[RP];
        take<T, WIDE>(in(0), d, y);
        if (p.leave) {
            take<T, WIDE>(in(1), d, u);
            const float s = p.post && on ? dot2(u, u) : 0.f;
            if (p.full) {
                f2 g[RP];
                take<T, WIDE>(in(2), d, g);
#pragma unroll
                for (int i = 0; i < RP; ++i) u[i] = u[i] * g[i];
            }
            if (p.post) {
                tok *= rsqrtf(row_sum(s, buf[0]) * invd + n.eps);
            }
            const f2 c = both(tok), ra = both(n.ra);
#pragma unroll
            for (int i = 0; i < RP; ++i) y[i] = fma2(c * wq[i], u[i], ra * y[i]);
            give<T, WIDE>(static_cast<T*>(n.x_out) + o, d, y);
        }
        if (p.enter) {
            const float s = on ? dot2(y, y) : 0.f;
            ring.wait_next(a, t);
            const f2 r = both(rsqrtf(row_sum(s, buf[p.leave ? 1 : par]) * invd + n.eps));
#pragma unroll
            for (int i = 0; i < RP; ++i) y[i] = y[i] * (r * wz[i]);
            give<T, WIDE>(static_cast<T*>(n.z) + o, d, y);
        }
        if (p.leave && !(p.post && p.enter)) {
            if (!p.enter) ring.wait_next(a, t);
            __syncthreads();
        }
        if (blockDim.x <= 32) __syncwarp();
        if (threadIdx.x == 0) ring.refill(a, ring_smem, t);
    }
    if (threadIdx.x == 0 && *ring.abort_flag) ring.drain();
}

// in: x_out, dz (enter), dx_out (if given), u (post or gate), gate (full)
template <typename T, bool WIDE, int FORM, int MAXT>
__global__ void __launch_bounds__(MAXT, (BWD_CTAS<FORM, MAXT>)) block_norm_bwd_ring_kernel(const __grid_constant__ RingArgs a) {
    __shared__ float buf[2][32 * 8];
    NORM_RING_SETUP();
    const Parts p = parts_of<FORM>(n);
    const bool enter = p.enter, leave = p.leave, post = p.post, full = p.full, along = p.along;
    const int gmode = FORM == FORM_ADD || FORM == FORM_ENTER ? MOE_GATE_NONE : n.gmode;
    const bool need_u = leave && (post || gmode != MOE_GATE_NONE);
    // q: w_post times the channel gate; w_pre.  Both channel gradients of u's side are
    // sums of h = b u r_u G (a full gate's: of g h) times what is constant along the sum:
    // dw_post = g sum h, dgate = w_post sum h.
    f2 wq[RP], wz[RP], acc_pre[RP], acc_h[RP];
    fill(acc_pre, 0.f);
    fill(acc_h, 0.f);
    fill(wq, 1.f);
    if (post) channel<T, WIDE>(n.w_post, d, wq);
    if (gmode == MOE_GATE_CHANNEL) {
        channel<T, WIDE>(static_cast<const float*>(n.gate), d, wz);
#pragma unroll
        for (int i = 0; i < RP; ++i) wq[i] = wq[i] * wz[i];
    }
    fill(wz, 1.f);
    if (enter) channel<T, WIDE>(n.w_pre, d, wz);
    // the tensors' places in a stage
    const int p_dz = 1, p_dx = enter ? 2 : 0, p_u = p_dx + (along ? 1 : 0), p_g = p_u + 1;
    const bool on = live<T, WIDE>(d);
    // A row's tensors, from its stage.  They are taken twice, for the sums and for the
    // outputs: between the two lies a barrier, and the next row's sums come before it.
    auto row = [&](int slot, int64_t t, f2 (&y)[RP], f2 (&dz)[RP], f2 (&G)[RP], f2 (&u)[RP], f2 (&g)[RP]) {
        const uint8_t* st = ring_smem + slot * ring.stage_bytes + (WIDE ? 0u : ring.shift(t));
        auto in = [&](int j) { return reinterpret_cast<const T*>(st + j * ring.pitch); };
        if (along) take<T, WIDE>(in(p_dx), d, G);
        else fill(G, 0.f);
        if (enter) {
            take<T, WIDE>(in(0), d, y);
            take<T, WIDE>(in(p_dz), d, dz);
        } else {
            fill(y, 0.f);
            fill(dz, 0.f);
        }
        if (need_u) take<T, WIDE>(in(p_u), d, u);
        else fill(u, 0.f);
        if (full) take<T, WIDE>(in(p_g), d, g);
    };
    // this warp's part of y^2, a y, u^2, q u dx', q u a, q u y  (a = w_pre dz, q = g w_post)
    auto sums = [&](int slot, int64_t t, float* to) {
        f2 y[RP], dz[RP], G[RP], u[RP], g[RP];
        row(slot, t, y, dz, G, u, g);
        f2 s1 = both(0.f), s3 = s1, s4 = s1, s5 = s1;
#pragma unroll
        for (int i = 0; i < RP; ++i) {
            const f2 az = wz[i] * dz[i];
            s1 = fma2(az, y[i], s1);
            if (need_u) {
                f2 qu = wq[i] * u[i];
                if (full) qu = qu * g[i];
                s3 = fma2(qu, G[i], s3);
                s4 = fma2(qu, az, s4);
                s5 = fma2(qu, y[i], s5);
            }
        }
        float s[6] = {dot2(y, y), sum2(s1), dot2(u, u), sum2(s3), sum2(s4), sum2(s5)};
#pragma unroll
        for (int i = 0; i < 6; ++i) s[i] = on ? s[i] : 0.f;
        put_sums6(warp_sums6(s), to);
    };
    int par = 0;
    if (blockIdx.x < n.T) sums(0, blockIdx.x, buf[0]);
    ring.wait_next(a, blockIdx.x);
    __syncthreads();
    for (int64_t t = blockIdx.x; t < n.T; t += gridDim.x, ring.next(), par ^= 1) {
        if (t + gridDim.x < n.T) sums(ring.ahead(1), t + gridDim.x, buf[par ^ 1]);
        const size_t o = (size_t)t * d;
        float tok = n.ob;
        if (gmode == MOE_GATE_TOKEN) tok *= __ldg(static_cast<const float*>(n.gate) + t);
        float s[6];
        get_sums6(s, buf[par]);
        f2 y[RP], G[RP], u[RP], dz[RP], g[RP], out[RP];   // (b and a token gate are in tok)
        row(ring.slot, t, y, dz, G, u, g);
        float r = 0.f, ca = 0.f;
        if (enter) {
            r = rsqrtf(s[0] * invd + n.eps);
            ca = r * (r * (r * (invd * s[1])));
            const f2 r2 = both(r), c2 = both(-ca);
#pragma unroll
            for (int i = 0; i < RP; ++i) {
                const f2 rz = r2 * dz[i];
                acc_pre[i] = fma2(rz, y[i], acc_pre[i]);
                G[i] = fma2(rz, wz[i], fma2(c2, y[i], G[i]));
            }
        }
        if (leave) {
            const f2 ra = both(n.ra);
#pragma unroll
            for (int i = 0; i < RP; ++i) out[i] = ra * G[i];
            give<T, WIDE>(static_cast<T*>(n.dx) + o, d, out);
            const float S = s[3] + r * s[4] - ca * s[5];
            const float ru = post ? rsqrtf(s[2] * invd + n.eps) : 1.f;
            if (gmode == MOE_GATE_TOKEN && threadIdx.x == 0) static_cast<float*>(n.dgate)[t] = n.ob * ru * S;
            const f2 tr = both(tok * ru), cu = both(post ? -tok * ru * (ru * (ru * (invd * S))) : 0.f);
            if (full) {
#pragma unroll
                for (int i = 0; i < RP; ++i) {
                    const f2 tG = tr * G[i], h = tG * u[i];
                    acc_h[i] = fma2(g[i], h, acc_h[i]);
                    u[i] = fma2(cu, u[i], (g[i] * wq[i]) * tG);
                    out[i] = wq[i] * h;
                }
                give<T, WIDE>(static_cast<T*>(n.dgate) + o, d, out);
#pragma unroll
                for (int i = 0; i < RP; ++i) out[i] = u[i];
            } else {
#pragma unroll
                for (int i = 0; i < RP; ++i) {
                    const f2 tG = tr * G[i];
                    acc_h[i] = fma2(tG, u[i], acc_h[i]);
                    out[i] = fma2(cu, u[i], wq[i] * tG);
                }
            }
            give<T, WIDE>(static_cast<T*>(n.du) + o, d, out);
        } else {
            give<T, WIDE>(static_cast<T*>(n.dx) + o, d, G);
        }
        // the next row's sums are there, its successor's stage has arrived, and this row's
        // stage is free
        ring.wait_next(a, t, 2);
        __syncthreads();
        if (threadIdx.x == 0) ring.refill(a, ring_smem, t);
    }
    auto flush = [&](int which, const f2 (&acc)[RP]) {
        constexpr int V = WIDE ? 16 / sizeof(T) : 1;
        float* dst = n.part + ((size_t)which * gridDim.x + blockIdx.x) * d;
#pragma unroll
        for (int i = 0; i < RP; ++i) {
            float lo, hi;
            unpk(acc[i], lo, hi);
            if constexpr (WIDE) {
                const int c = part_of<T>(2 * i / V) + 2 * i % V;
                if (c < d) *reinterpret_cast<float2*>(dst + c) = make_float2(lo, hi);
            } else {
                const int c = threadIdx.x + 2 * i * blockDim.x;
                if (c < d) dst[c] = lo;
                if (c + (int)blockDim.x < d) dst[c + blockDim.x] = hi;
            }
        }
    };
    if (enter) flush(0, acc_pre);
    if (gmode == MOE_GATE_CHANNEL) {
        if (post) channel<T, WIDE>(n.w_post, d, wq);
        else fill(wq, 1.f);
        channel<T, WIDE>(static_cast<const float*>(n.gate), d, wz);
#pragma unroll
        for (int i = 0; i < RP; ++i) {
            wq[i] = wq[i] * acc_h[i];
            acc_h[i] = wz[i] * acc_h[i];
        }
        flush(2, wq);
    }
    if (post) flush(1, acc_h);
    if (threadIdx.x == 0 && *ring.abort_flag) ring.drain();
}

// Column sums of the CTAs' partials: 32 columns x 32 row lanes a CTA, each lane
// its rows in order, the lanes added in order.  grid.y: which gradient.
struct NormReduceArgs {
    const float* part;
    float* out[3];
    int rows, d;
};
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const NormReduceArgs a) {
    pdl_wait();
    pdl_trigger();
    __shared__ float sm[32][33];
    float* out = a.out[blockIdx.y];
    if (!out) return;
    const int c = blockIdx.x * 32 + threadIdx.x;
    const float* p = a.part + (size_t)blockIdx.y * a.rows * a.d + c;
    float v = 0.f;
    if (c < a.d)
#pragma unroll 4
        for (int r = threadIdx.y; r < a.rows; r += 32) v += p[(size_t)r * a.d];
    sm[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && c < a.d) {
        for (int y = 1; y < 32; ++y) v += sm[y][threadIdx.x];
        out[c] = v;
    }
}

// the direct kernels: elements a thread, threads of a row, rows per CTA
int direct_ept(const moe_norm_config& c) { return c.d <= 8 * 1024 ? 8 : 16; }
dim3 norm_block(const moe_norm_config& c) {
    const int ept = direct_ept(c), tpr = ((c.d + ept - 1) / ept + 31) / 32 * 32;
    return dim3(tpr, tpr == 32 ? SMALL_ROWS : 1);
}
bool wide_rows(const moe_norm_config& c) { return (c.d * (c.dtype == MOE_DTYPE_BF16 ? 2 : 4)) % 16 == 0; }

// The ring's launch: threads, stages and CTAs, or none (0 stages) where the direct
// kernels serve.  Those win while a batch is short, when filling a ring is most of the
// work (us as a graph, direct and ring, bf16 rows, both norms and a channel gate):
//   forward    1216 x 1024   3.6  5.9    16384 x 512  14.9 15.3    16384 x 1024  34.1 27.4
//   backward    304 x 1024   8.0  8.3     4864 x 512  17.8 17.3    16384 x 512   49.2 29.9
//               152 x 4096  14.8 13.0    16384 x 256  24.4 25.1    65536 x 64    55.4 46.0
// Rows of no whole 16 bytes take the ring as soon as every SM has one (608 x 1001: 7.1
// and 6.2 forward, 27.9 and 10.9 backward).  Rows too wide for three stages never do.
// The rule goes by elements alone, and is on the careful side at its edges: wide rows just
// below the forward's bound (2432 x 4096: 22.6 direct, 16.4) and narrow ones in the backward
// (65536 x 64 above) would gain from the ring; entering alone at 16384 x 512 would not
// (10.7, 11.8).
bool ring_pays(const moe_norm_config& c, bool backward) {
    const int64_t n = (int64_t)c.T * c.d;
    if (c.T < num_sms()) return false;
    if (!wide_rows(c)) return true;
    if (!backward) return n >= (10 << 20);
    return c.d >= 1024 || (c.d >= 128 && n >= (4 << 20));
}
struct RingPlan { int threads, stages, grid; size_t smem; };
RingPlan ring_plan(const moe_norm_config& c, int nin, int regs, bool backward) {
    RingPlan p = {0, 0, 0, 0};
    const int es = c.dtype == MOE_DTYPE_BF16 ? 2 : 4;
    p.threads = ((c.d + RE - 1) / RE + 31) / 32 * 32;
    if (p.threads > 1024 || !ring_pays(c, backward)) return p;
    const int stage = nin * (int)row_pitch(c.d * es);
    // CTAs an SM by registers and threads, fewer where they would not have three stages
    // each (228 KB an SM, 3 KB of it a CTA's fixed part)
    int per_sm = std::max(1, std::min(std::min(32, 65536 / (regs * p.threads)), 2048 / p.threads));
    auto room = [&](int n) { return std::min(200 * 1024, 224 * 1024 / n - 3 * 1024); };
    while (per_sm > 1 && room(per_sm) < 3 * stage) --per_sm;
    p.stages = std::min(MAX_STAGES, room(per_sm) / stage);
    if (p.stages < 3) { p.stages = 0; return p; }   // the backward works on two at a time
    p.smem = (size_t)p.stages * stage;
    // four rows a CTA, at least, once every SM has one: a CTA's rows share its set-up and,
    // in the backward, one row of partial sums
    p.grid = (int)std::min<int64_t>(std::min<int64_t>(c.T, (int64_t)per_sm * num_sms()), std::max<int64_t>(num_sms(), c.T / 4));
    return p;
}
int fwd_inputs(const moe_norm_config& c) { return 1 + c.leave + (c.gate == MOE_GATE_FULL); }
bool bwd_needs_u(const moe_norm_config& c) { return c.leave && (c.post_norm || c.gate != MOE_GATE_NONE); }
int bwd_inputs(const moe_norm_config& c) {   // with dx_out
    return 1 + 2 * c.enter + bwd_needs_u(c) + (c.gate == MOE_GATE_FULL);
}
// (the workspace is sized by this plan, so it does not look at which gradients are given:
// a call without dx_out only has more CTAs than its registers let run at once)
RingPlan bwd_ring(const moe_norm_config& c) {
    int regs = 128;
    if (c.gate != MOE_GATE_FULL) {
        if (c.leave && c.post_norm) regs = c.enter ? 100 : 64;
        else if (!c.leave || (c.enter && c.gate == MOE_GATE_NONE)) regs = 64;
    }
    return ring_plan(c, bwd_inputs(c), regs, true);
}

// CTAs of the backward: as many as the GPU holds, none with less than a row
int bwd_grid(const moe_norm_config& c) {
    const RingPlan p = bwd_ring(c);
    if (p.stages) return p.grid;
    // up to four rows a CTA before there are more CTAs than SMs: each adds a row to the
    // partial sums that the last kernel reads
    const dim3 b = norm_block(c);
    const int64_t rows = std::max<int64_t>(1, std::min<int64_t>(4, c.T / num_sms())) * b.y;
    const int per_sm = std::max(1, 1024 / (int)(b.x * b.y));
    return (int)std::min<int64_t>((c.T + rows - 1) / rows, (int64_t)num_sms() * per_sm);
}

template <typename T, bool WIDE, int FORM, int MAXT>
int launch_fwd_ring_t(const RingPlan& p, const RingArgs& r, cudaStream_t st) {
    static bool done[64] = {};
    if (const int e = smem_attr_once(block_norm_ring_kernel<T, WIDE, FORM, MAXT>, 200 * 1024, done)) return e;
    MOE_LAUNCH((block_norm_ring_kernel<T, WIDE, FORM, MAXT>), p.grid, p.threads, p.smem, st, r);
    return MOE_OK;
}
template <typename T, bool WIDE, int FORM>
int launch_fwd_ring_f(const RingPlan& p, const RingArgs& r, cudaStream_t st) {
    return p.threads <= 512 ? launch_fwd_ring_t<T, WIDE, FORM, 512>(p, r, st)
                            : launch_fwd_ring_t<T, WIDE, FORM, 1024>(p, r, st);
}
template <typename T, bool WIDE>
int launch_fwd_ring(const RingPlan& p, const RingArgs& r, cudaStream_t st) {
    switch (form_of(r.n, false)) {
        case FORM_BOTH: return launch_fwd_ring_f<T, WIDE, FORM_BOTH>(p, r, st);
        case FORM_ADD: return launch_fwd_ring_f<T, WIDE, FORM_ADD>(p, r, st);
        case FORM_ENTER: return launch_fwd_ring_f<T, WIDE, FORM_ENTER>(p, r, st);
        default: return launch_fwd_ring_f<T, WIDE, FORM_ANY>(p, r, st);
    }
}
template <typename T, bool WIDE, int FORM, int MAXT>
int launch_bwd_ring_t(const RingPlan& p, const RingArgs& r, cudaStream_t st) {
    static bool done[64] = {};
    if (const int e = smem_attr_once(block_norm_bwd_ring_kernel<T, WIDE, FORM, MAXT>, 200 * 1024, done)) return e;
    MOE_LAUNCH((block_norm_bwd_ring_kernel<T, WIDE, FORM, MAXT>), p.grid, p.threads, p.smem, st, r);
    return MOE_OK;
}
// the fewer the threads, the more registers each may have
template <typename T, bool WIDE, int FORM>
int launch_bwd_ring_f(const RingPlan& p, const RingArgs& r, cudaStream_t st) {
    return p.threads <= 512   ? launch_bwd_ring_t<T, WIDE, FORM, 512>(p, r, st)
           : p.threads <= 768 ? launch_bwd_ring_t<T, WIDE, FORM, 768>(p, r, st)
                              : launch_bwd_ring_t<T, WIDE, FORM, 1024>(p, r, st);
}
template <typename T, bool WIDE>
int launch_bwd_ring(const RingPlan& p, const RingArgs& r, cudaStream_t st) {
    switch (form_of(r.n, true)) {
        case FORM_BOTH: return launch_bwd_ring_f<T, WIDE, FORM_BOTH>(p, r, st);
        case FORM_ADD: return launch_bwd_ring_f<T, WIDE, FORM_ADD>(p, r, st);
        case FORM_ENTER: return launch_bwd_ring_f<T, WIDE, FORM_ENTER>(p, r, st);
        case FORM_LEAVE: return launch_bwd_ring_f<T, WIDE, FORM_LEAVE>(p, r, st);
        default: return launch_bwd_ring_f<T, WIDE, FORM_ANY>(p, r, st);
    }
}

template <typename T, int VEC>
int launch_fwd(const moe_norm_config& c, const NormArgs& a, cudaStream_t st) {
    const RingPlan p = ring_plan(c, fwd_inputs(c), c.post_norm || c.gate != MOE_GATE_NONE ? 64 : 40, false);
    if (p.stages) {
        RingArgs r = {};
        r.n = a;
        r.in[r.nin++] = a.x;
        if (c.leave) r.in[r.nin++] = a.u;
        if (c.gate == MOE_GATE_FULL) r.in[r.nin++] = a.gate;
        r.stages = p.stages;
        r.status = device_status_ptr();
        return launch_fwd_ring<T, (VEC > 1)>(p, r, st);
    }
    const dim3 b = norm_block(c);
    const int grid = (int)std::min<int64_t>(((int64_t)c.T + b.y - 1) / b.y, (int64_t)num_sms() * 64);
    if (direct_ept(c) == 16) MOE_LAUNCH((block_norm_kernel<T, VEC, 16, 1024>), grid, b, 0, st, a);
    else if (b.x <= 256) MOE_LAUNCH((block_norm_kernel<T, VEC, 8, 256>), grid, b, 0, st, a);
    else MOE_LAUNCH((block_norm_kernel<T, VEC, 8, 1024>), grid, b, 0, st, a);
    return MOE_OK;
}
template <typename T, int VEC>
int launch_bwd(const moe_norm_config& c, const NormArgs& a, float* dwpre, float* dwpost, cudaStream_t st) {
    const dim3 b = norm_block(c);
    const int grid = bwd_grid(c);
    const RingPlan p = bwd_ring(c);
    const size_t smem = b.y > 1 ? (size_t)b.y * c.d * 4 : 0;
    if (p.stages) {
        RingArgs q = {};
        q.n = a;
        if (c.enter) q.in[q.nin++] = a.x;
        if (c.enter) q.in[q.nin++] = a.dz;
        if (a.dx_out) q.in[q.nin++] = a.dx_out;
        if (bwd_needs_u(c)) q.in[q.nin++] = a.u;
        if (c.gate == MOE_GATE_FULL) q.in[q.nin++] = a.gate;
        q.stages = p.stages;
        q.status = device_status_ptr();
        if (const int e = (launch_bwd_ring<T, (VEC > 1)>(p, q, st))) return e;
    } else if (direct_ept(c) == 16) {
        MOE_LAUNCH((block_norm_bwd_kernel<T, VEC, 16, 1024>), grid, b, smem, st, a);
    } else if (b.x <= 256) {
        MOE_LAUNCH((block_norm_bwd_kernel<T, VEC, 8, 256>), grid, b, smem, st, a);
    } else if (b.x <= 512) {
        MOE_LAUNCH((block_norm_bwd_kernel<T, VEC, 8, 512>), grid, b, smem, st, a);
    } else {
        MOE_LAUNCH((block_norm_bwd_kernel<T, VEC, 8, 1024>), grid, b, smem, st, a);
    }
    NormReduceArgs r;
    r.part = a.part;
    r.rows = grid;
    r.d = c.d;
    r.out[0] = c.enter ? dwpre : nullptr;
    r.out[1] = c.post_norm ? dwpost : nullptr;
    r.out[2] = c.gate == MOE_GATE_CHANNEL ? static_cast<float*>(a.dgate) : nullptr;
    if (r.out[0] || r.out[1] || r.out[2])
        MOE_LAUNCH(norm_reduce_kernel, dim3((c.d + 31) / 32, 3), dim3(32, 32), 0, st, r);
    return MOE_OK;
}

NormArgs base_args(const moe_norm_config& c) {
    NormArgs a = {};
    a.T = c.T; a.d = c.d; a.leave = c.leave; a.post = c.post_norm; a.enter = c.enter;
    a.gmode = c.gate; a.eps = c.eps; a.ra = c.res_scale; a.ob = c.out_scale;
    return a;
}

}  // namespace

size_t norm_ws_bytes(const moe_norm_config& c) { return align_up((size_t)3 * bwd_grid(c) * c.d * 4); }

int launch_block_norm(const moe_norm_config& c, const void* x, const void* u, const float* w_post,
                      const void* gate, const float* w_pre, void* x_out, void* z, cudaStream_t st) {
    NormArgs a = base_args(c);
    a.x = x; a.u = u; a.w_post = w_post; a.gate = gate; a.w_pre = w_pre; a.x_out = x_out; a.z = z;
    const bool wide = wide_rows(c);
    if (c.dtype == MOE_DTYPE_BF16)
        return wide ? launch_fwd<__nv_bfloat16, 8>(c, a, st) : launch_fwd<__nv_bfloat16, 1>(c, a, st);
    return wide ? launch_fwd<float, 4>(c, a, st) : launch_fwd<float, 1>(c, a, st);
}

int launch_block_norm_backward(const moe_norm_config& c, const void* x_out, const void* u,
                               const float* w_post, const void* gate, const float* w_pre,
                               const void* dx_out, const void* dz, void* dx, void* du,
                               float* dw_post, void* dgate, float* dw_pre, void* ws, cudaStream_t st) {
    NormArgs a = base_args(c);
    a.x = x_out; a.u = u; a.w_post = w_post; a.gate = gate; a.w_pre = w_pre; a.dx_out = dx_out;
    a.dz = dz; a.dx = dx; a.du = du; a.dgate = dgate; a.part = static_cast<float*>(ws);
    const bool wide = wide_rows(c);
    if (c.dtype == MOE_DTYPE_BF16)
        return wide ? launch_bwd<__nv_bfloat16, 8>(c, a, dw_pre, dw_post, st)
                    : launch_bwd<__nv_bfloat16, 1>(c, a, dw_pre, dw_post, st);
    return wide ? launch_bwd<float, 4>(c, a, dw_pre, dw_post, st)
                : launch_bwd<float, 1>(c, a, dw_pre, dw_post, st);
}

}  // namespace moe
