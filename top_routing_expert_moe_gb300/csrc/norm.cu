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
#include "norm_rows.cuh"

namespace moe {

namespace {

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
