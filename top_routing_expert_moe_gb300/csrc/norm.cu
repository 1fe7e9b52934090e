// norm.cu -- the residual stream's norms around a block, forward and backward.
//
//   leave:  n = w_post u r_u (or u),  x' = a x + b g n     r_v = 1/sqrt(mean v^2 + eps)
//   enter:  z = w_pre x' r
// A row is held in registers by one group of threads (16 elements a thread), so
// each tensor passes through HBM once.  All sums are fp32.
//
// Backward, for one row, with G the gradient of x':
//   a_i = w_pre dz,  G = dx' + r a - x' (r^3/d) A,            A   = sum a x'
//   q   = b g w_post (1 for an absent factor),  dn w_post = q G
//   du  = r_u q G - u (r_u^3/d) S,                            S   = sum q u G
// S is linear in G, so it comes from the first pass's sums,
//   S = sum q u dx' + r sum q u a - (r^3/d) A sum q u x',
// and one reduction of six sums serves the whole row.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int EPT = 16;          // elements of a row per thread
constexpr int SMALL_ROWS = 4;    // rows per CTA when a warp holds a row

template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// Sums over the threads of a row: a warp, or the whole CTA through shared memory
// (buf: 32 x N floats; the caller alternates two buffers, so one barrier a call
// is enough), warps added in order.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* buf) {
    warp_sums(v);
    if (blockDim.x <= 32) return;
    const int w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) buf[w * N + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = buf[i];
    for (int j = 1; j < nw; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += buf[j * N + i];
}

// A thread's share of a row: vectors tid, tid + TPR, ... of VEC elements.
template <typename T, int VEC>
__device__ __forceinline__ void load_row(const T* p, int nvec, float (&v)[EPT]) {
#pragma unroll
    for (int i = 0; i < EPT / VEC; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if constexpr (VEC == 1) {
            v[i] = c < nvec ? to_f<T>(p[c]) : 0.f;
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[i * VEC + j] = 0.f;
            if (c < nvec) load16_f<T>(p + c * VEC, v + i * VEC);
        }
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_row(T* p, int nvec, const float (&v)[EPT]) {
#pragma unroll
    for (int i = 0; i < EPT / VEC; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nvec) continue;
        if constexpr (VEC == 1) p[c] = from_f<T>(v[i]);
        else store16_f<T>(p + c * VEC, v + i * VEC);
    }
}
// fp32 vector over the channels, in the thread's share
template <int VEC>
__device__ __forceinline__ void load_vec(const float* p, int nvec, float (&v)[EPT]) {
#pragma unroll
    for (int i = 0; i < EPT / VEC; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if constexpr (VEC == 1) {
            v[i] = c < nvec ? __ldg(p + c) : 0.f;
        } else {
#pragma unroll
            for (int j = 0; j < VEC; j += 4) {
                const float4 f = c < nvec ? __ldg(reinterpret_cast<const float4*>(p + c * VEC + j))
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
                v[i * VEC + j] = f.x; v[i * VEC + j + 1] = f.y;
                v[i * VEC + j + 2] = f.z; v[i * VEC + j + 3] = f.w;
            }
        }
    }
}

struct NormArgs {
    const void *x, *u, *gate, *dx_out, *dz;   // x: the stream (x_out in the backward)
    const float *w_post, *w_pre;
    void *x_out, *z, *dx, *du, *dgate;
    float *part;                              // [3][grid][d]: dw_pre, dw_post, dgate partials
    int T, d, leave, post, enter, gmode;
    float eps, ra, ob;
};

template <typename T, int VEC, int MAXT>
__global__ void __launch_bounds__(MAXT) block_norm_kernel(const NormArgs a) {
    pdl_wait();
    pdl_trigger();
    __shared__ float buf[2][32];
    const int nvec = a.d / VEC;
    const float invd = 1.f / (float)a.d;
    for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < a.T;
         t += (int64_t)gridDim.x * blockDim.y) {
        const size_t o = (size_t)t * a.d;
        float y[EPT], u[EPT], w[EPT];
        load_row<T, VEC>(static_cast<const T*>(a.x) + o, nvec, y);
        if (a.leave) {
            load_row<T, VEC>(static_cast<const T*>(a.u) + o, nvec, u);
            float c = a.ob;
            if (a.gmode == MOE_GATE_TOKEN) c *= static_cast<const float*>(a.gate)[t];
            if (a.post) {
                float s[1] = {0.f};
#pragma unroll
                for (int i = 0; i < EPT; ++i) s[0] = fmaf(u[i], u[i], s[0]);
                row_sums<1>(s, buf[0]);
                c *= 1.f / sqrtf(s[0] * invd + a.eps);
                load_vec<VEC>(a.w_post, nvec, w);
#pragma unroll
                for (int i = 0; i < EPT; ++i) u[i] *= w[i];
            }
            if (a.gmode == MOE_GATE_CHANNEL || a.gmode == MOE_GATE_FULL) {
                if (a.gmode == MOE_GATE_CHANNEL) load_vec<VEC>(static_cast<const float*>(a.gate), nvec, w);
                else load_row<T, VEC>(static_cast<const T*>(a.gate) + o, nvec, w);
#pragma unroll
                for (int i = 0; i < EPT; ++i) u[i] *= w[i];
            }
#pragma unroll
            for (int i = 0; i < EPT; ++i) y[i] = fmaf(a.ra, y[i], c * u[i]);
            store_row<T, VEC>(static_cast<T*>(a.x_out) + o, nvec, y);
        }
        if (a.enter) {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < EPT; ++i) s[0] = fmaf(y[i], y[i], s[0]);
            row_sums<1>(s, buf[1]);
            const float r = 1.f / sqrtf(s[0] * invd + a.eps);
            load_vec<VEC>(a.w_pre, nvec, w);
#pragma unroll
            for (int i = 0; i < EPT; ++i) y[i] *= r * w[i];
            store_row<T, VEC>(static_cast<T*>(a.z) + o, nvec, y);
        }
        // buf[0] and buf[1] alternate unless only one of the norms is on
        if (a.post != a.enter && blockDim.x > 32) __syncthreads();
    }
}

template <typename T, int VEC, int MAXT>
__global__ void __launch_bounds__(MAXT) block_norm_bwd_kernel(const NormArgs a) {
    pdl_wait();
    pdl_trigger();
    __shared__ float buf[2][32 * 6];
    extern __shared__ float comb[];            // [SMALL_ROWS][d] when a CTA holds several rows
    const int nvec = a.d / VEC;
    const float invd = 1.f / (float)a.d;
    float acc_pre[EPT], acc_post[EPT], acc_g[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i) acc_pre[i] = acc_post[i] = acc_g[i] = 0.f;
    const bool need_u = a.leave && (a.post || a.gmode != MOE_GATE_NONE);
    int par = 0;
    for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < a.T;
         t += (int64_t)gridDim.x * blockDim.y, par ^= 1) {
        const size_t o = (size_t)t * a.d;
        float y[EPT], u[EPT], dz[EPT], G[EPT], w[EPT], q[EPT];
        if (a.enter) {
            load_row<T, VEC>(static_cast<const T*>(a.x) + o, nvec, y);
            load_row<T, VEC>(static_cast<const T*>(a.dz) + o, nvec, dz);
        }
        if (a.dx_out) load_row<T, VEC>(static_cast<const T*>(a.dx_out) + o, nvec, G);
        else
#pragma unroll
            for (int i = 0; i < EPT; ++i) G[i] = 0.f;
        if (need_u) load_row<T, VEC>(static_cast<const T*>(a.u) + o, nvec, u);
        else
#pragma unroll
            for (int i = 0; i < EPT; ++i) u[i] = 0.f;
        // q = b g w_post
        float tok = a.ob;
        if (a.gmode == MOE_GATE_TOKEN) tok *= static_cast<const float*>(a.gate)[t];
        if (a.post) load_vec<VEC>(a.w_post, nvec, q);
        else
#pragma unroll
            for (int i = 0; i < EPT; ++i) q[i] = 1.f;
        if (a.gmode == MOE_GATE_CHANNEL) load_vec<VEC>(static_cast<const float*>(a.gate), nvec, w);
        else if (a.gmode == MOE_GATE_FULL) load_row<T, VEC>(static_cast<const T*>(a.gate) + o, nvec, w);
        else
#pragma unroll
            for (int i = 0; i < EPT; ++i) w[i] = 1.f;       // (the token gate is in tok)
        // s: y^2, a y, u^2, q u dx', q u a, q u y  (q without the factor tok)
        float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        float wp[EPT];
        if (a.enter) {
            load_vec<VEC>(a.w_pre, nvec, wp);
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                s[0] = fmaf(y[i], y[i], s[0]);
                s[1] = fmaf(wp[i] * dz[i], y[i], s[1]);
            }
        }
        if (need_u) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                const float qu = q[i] * w[i] * u[i];
                s[2] = fmaf(u[i], u[i], s[2]);
                s[3] = fmaf(qu, G[i], s[3]);
                if (a.enter) {
                    s[4] = fmaf(qu, wp[i] * dz[i], s[4]);
                    s[5] = fmaf(qu, y[i], s[5]);
                }
            }
        }
        row_sums<6>(s, buf[par]);
        float r = 0.f, ca = 0.f;
        if (a.enter) {
            r = 1.f / sqrtf(s[0] * invd + a.eps);
            ca = r * r * r * invd * s[1];
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                G[i] += r * (wp[i] * dz[i]) - ca * y[i];
                acc_pre[i] = fmaf(dz[i], r * y[i], acc_pre[i]);
            }
        }
        if (!a.leave) {
            store_row<T, VEC>(static_cast<T*>(a.dx) + o, nvec, G);
            continue;
        }
        const float S = s[3] + r * s[4] - ca * s[5];     // sum q u G, without tok
        float out[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) out[i] = a.ra * G[i];
        store_row<T, VEC>(static_cast<T*>(a.dx) + o, nvec, out);
        const float ru = a.post ? 1.f / sqrtf(s[2] * invd + a.eps) : 1.f;
        if (a.gmode == MOE_GATE_TOKEN && threadIdx.x == 0)
            static_cast<float*>(a.dgate)[t] = a.ob * ru * S;
        if (a.gmode == MOE_GATE_CHANNEL) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) acc_g[i] = fmaf(a.ob * G[i], q[i] * u[i] * ru, acc_g[i]);
        } else if (a.gmode == MOE_GATE_FULL) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) out[i] = a.ob * G[i] * (q[i] * u[i] * ru);
            store_row<T, VEC>(static_cast<T*>(a.dgate) + o, nvec, out);
        }
        const float cu = a.post ? tok * ru * ru * ru * invd * S : 0.f;
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const float dn = tok * w[i] * G[i];
            acc_post[i] = fmaf(dn, u[i] * ru, acc_post[i]);
            out[i] = a.post ? ru * q[i] * dn - cu * u[i] : dn;
        }
        store_row<T, VEC>(static_cast<T*>(a.du) + o, nvec, out);
    }
    // this CTA's partial sums of the channel gradients
    auto flush = [&](int which, const float (&acc)[EPT]) {
        float* dst = a.part + ((size_t)which * gridDim.x + blockIdx.x) * a.d;
        if (blockDim.y == 1) {
#pragma unroll
            for (int i = 0; i < EPT / VEC; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                if (c < nvec)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) dst[c * VEC + j] = acc[i * VEC + j];
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < EPT / VEC; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < nvec)
#pragma unroll
                for (int j = 0; j < VEC; ++j) comb[threadIdx.y * a.d + c * VEC + j] = acc[i * VEC + j];
        }
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

// threads of a row, rows per CTA
dim3 norm_block(const moe_norm_config& c) {
    const int tpr = ((c.d + EPT - 1) / EPT + 31) / 32 * 32;
    return dim3(tpr, tpr == 32 ? SMALL_ROWS : 1);
}
bool wide_rows(const moe_norm_config& c) { return (c.d * (c.dtype == MOE_DTYPE_BF16 ? 2 : 4)) % 16 == 0; }

// CTAs of the backward: as many as the GPU holds, none with less than a row
int bwd_grid(const moe_norm_config& c) {
    const dim3 b = norm_block(c);
    const int per_sm = std::max(1, 512 / (int)(b.x * b.y));
    return (int)std::max<int64_t>(1, std::min<int64_t>(((int64_t)c.T + b.y - 1) / b.y, (int64_t)num_sms() * per_sm));
}

template <typename T, int VEC>
int launch_fwd(const moe_norm_config& c, const NormArgs& a, cudaStream_t st) {
    const dim3 b = norm_block(c);
    const int grid = (int)std::min<int64_t>(((int64_t)c.T + b.y - 1) / b.y, (int64_t)num_sms() * 64);
    if (b.x <= 256) MOE_LAUNCH((block_norm_kernel<T, VEC, 256>), grid, b, 0, st, a);
    else MOE_LAUNCH((block_norm_kernel<T, VEC, 1024>), grid, b, 0, st, a);
    return MOE_OK;
}
template <typename T, int VEC>
int launch_bwd(const moe_norm_config& c, const NormArgs& a, float* dwpre, float* dwpost, cudaStream_t st) {
    const dim3 b = norm_block(c);
    const int grid = bwd_grid(c);
    const size_t smem = b.y > 1 ? (size_t)b.y * c.d * 4 : 0;
    if (b.x <= 256) MOE_LAUNCH((block_norm_bwd_kernel<T, VEC, 256>), grid, b, smem, st, a);
    else if (b.x <= 512) MOE_LAUNCH((block_norm_bwd_kernel<T, VEC, 512>), grid, b, smem, st, a);
    else MOE_LAUNCH((block_norm_bwd_kernel<T, VEC, 1024>), grid, b, smem, st, a);
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
