// mx8.cu -- microscaled 8-bit numbers (mx8.cuh): quantisation of rows and of expert
// weights, the values that codes and scales stand for, and the permutation of 8-bit
// rows into expert segments.
//
// Memory-bound: 2 (or 4) bytes read, 33/32 written an element, and back: 65536 x 4096 bf16
// rows 116 us (7.0 TB/s), their values 122 (6.7); weights 8 x 4096 x 14336 219 (6.5), their
// values 209 in bf16 (6.8) and 440 in fp32 (5.4: a thread's four stores are 64 bytes apart
// from its neighbour's).
#include <algorithm>

#include "kernels.h"
#include "mx8.cuh"

namespace moe {

namespace {

constexpr int ROW_THREADS = 256, ROW_UNROLL = 4;
constexpr int ROW_VECS = ROW_THREADS * ROW_UNROLL;      // vectors of a CTA's turn

// A CTA's turn: whole rows while they fit, else a part of one row.  Vector i of the
// turn lies in row i / nvec of it (by a product: i and nvec stay below 2^11 then, and a row,
// whole blocks, has at least two vectors, so that 2^32 / nvec fits 32 bits).
struct Turns {
    int64_t rows, turns;                                // rows, and turns of `per` of them
    int nvec, per, parts;                               // vectors a row; rows a turn; turns a row
    uint32_t magic;
};
Turns turns_of(int64_t rows, int nvec) {
    Turns t;
    t.rows = rows;
    t.nvec = nvec;
    t.per = std::max(1, ROW_VECS / nvec);
    t.parts = nvec > ROW_VECS ? (nvec + ROW_VECS - 1) / ROW_VECS : 1;
    t.turns = (rows + t.per - 1) / t.per * t.parts;
    t.magic = (uint32_t)(((1ull << 32) + nvec - 1) / nvec);
    return t;
}
// places of this thread's vectors in turn `u`: row and vector, row -1 past the end
struct Place { int64_t row; int vec; };
__device__ __forceinline__ Place place(const Turns& t, int64_t used, int64_t u, int j) {
    const int i = threadIdx.x + j * ROW_THREADS;
    Place p;
    if (t.parts == 1) {
        const int r = (int)__umulhi((uint32_t)i, t.magic);
        p.row = u * t.per + r;
        p.vec = i - r * t.nvec;
        if (r >= t.per) p.row = -1;
    } else {
        p.row = u / t.parts;
        p.vec = (int)(u - p.row * t.parts) * ROW_VECS + i;
        if (p.vec >= t.nvec) p.row = -1;
    }
    if (p.row >= used) p.row = -1;
    return p;
}
int turn_grid(const Turns& t) { return (int)std::max<int64_t>(1, std::min<int64_t>(t.turns, (int64_t)num_sms() * 32)); }

// 32 bytes of elements as loaded
template <typename T> struct Raw32 {
    static constexpr int N = 32 / sizeof(T);
    uint4 a, b;
    __device__ __forceinline__ void load(const T* p) {
        a = __ldg(reinterpret_cast<const uint4*>(p));
        b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void values(float (&v)[N]) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(T) == 2) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                v[i] = __uint_as_float(w[i]);
            }
        }
    }
};

// Rows: 32 bytes a thread, so two (bf16) or four (fp32) neighbouring lanes hold a block
// (rows are whole blocks, so those lanes are of one row).  65536 x 4096 bf16 116 us (7.0 TB/s),
// with 16 bytes a thread 144; fp32 191 us (7.1 TB/s).
template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) mx8_rows_kernel(const T* __restrict__ x, const Turns t, int K, int pitch,
                                                               const int32_t* __restrict__ rows_used,
                                                               uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    pdl_wait();
    pdl_trigger();
    constexpr int N = Raw32<T>::N;
    int64_t used = t.rows;
    if (rows_used) used = min(used, (int64_t)max(*rows_used, 0));
    for (int64_t u = blockIdx.x; u < t.turns; u += gridDim.x) {
        Place p[ROW_UNROLL];
        Raw32<T> raw[ROW_UNROLL];
#pragma unroll
        for (int j = 0; j < ROW_UNROLL; ++j) {
            p[j] = place(t, used, u, j);
            if (p[j].row >= 0) raw[j].load(x + p[j].row * K + p[j].vec * N);
            else raw[j].zero();
        }
#pragma unroll
        for (int j = 0; j < ROW_UNROLL; ++j) {
            float v[N];
            raw[j].values(v);
            uint32_t m = amax_bits<N>(v);
#pragma unroll
            for (int o = 1; o < 32 / N; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            const uint32_t s = mx8_scale_byte(m);
            uint32_t w[N / 4];
            mx8_codes<N>(v, s, w);
            if (p[j].row < 0) continue;
            uint8_t* dst = codes + p[j].row * K + p[j].vec * N;
            if constexpr (N == 16) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            else *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
            if (threadIdx.x % (32 / N) == 0) scales[p[j].row * pitch + p[j].vec / (32 / N)] = (uint8_t)s;
        }
    }
}

// Values: as many codes a thread as 16 bytes of the output hold, so that a warp's stores
// lie side by side (32 bytes a thread, two stores: 16384 x 4096 to bf16 39 us, so 32)
template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) mx8_values_kernel(const uint8_t* __restrict__ codes,
                                                                 const uint8_t* __restrict__ scales, const Turns t, int K,
                                                                 int pitch, T* __restrict__ out) {
    pdl_wait();
    pdl_trigger();
    constexpr int V = Vec16<T>::N;
    for (int64_t u = blockIdx.x; u < t.turns; u += gridDim.x) {
        Place p[ROW_UNROLL];
        uint32_t c[ROW_UNROLL][V / 4], s[ROW_UNROLL];
#pragma unroll
        for (int j = 0; j < ROW_UNROLL; ++j) {
            p[j] = place(t, t.rows, u, j);
            if (p[j].row < 0) continue;
            const uint8_t* src = codes + p[j].row * K + p[j].vec * V;
            if constexpr (V == 8) {
                const uint2 w = __ldg(reinterpret_cast<const uint2*>(src));
                c[j][0] = w.x;
                c[j][1] = w.y;
            } else {
                c[j][0] = __ldg(reinterpret_cast<const uint32_t*>(src));
            }
            s[j] = __ldg(scales + p[j].row * pitch + p[j].vec / (32 / V));
        }
#pragma unroll
        for (int j = 0; j < ROW_UNROLL; ++j) {
            if (p[j].row < 0) continue;
            const float m = mx8_scale_value(s[j]);
            float v[V];
#pragma unroll
            for (int i = 0; i < V / 4; ++i) mx8_unpack4(c[j][i], v + 4 * i);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] *= m;
            store16_f<T>(out + p[j].row * K + p[j].vec * V, v);
        }
    }
}

// Weights W [E, K, N] -> blocks of 128 n x 128 k (the header's order): a CTA takes 128 k x
// 64 n through shared memory and writes half a block, 8 KB in a row; a thread forms one
// run of 32 k of one column.  Places past N or K hold zeros.
constexpr int WN = 64, W_THREADS = WN * 4;
template <typename T>
__global__ void __launch_bounds__(W_THREADS) mx8_weight_kernel(const T* __restrict__ W, int K, int N,
                                                               uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    pdl_wait();
    pdl_trigger();
    constexpr int V = 16 / sizeof(T);
    __shared__ __align__(16) T sm[128][WN + V];
    __shared__ __align__(16) uint8_t sc[WN][128 + 16];
    __shared__ __align__(4) uint8_t sb[WN][4];
    const int k0 = blockIdx.x * 128, n0 = blockIdx.y * WN, e = blockIdx.z;
    const T* We = W + (size_t)e * K * N;
#pragma unroll
    for (int i = threadIdx.x; i < 128 * (WN / V); i += W_THREADS) {
        const int k = i / (WN / V), c = i % (WN / V) * V;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (k0 + k < K && n0 + c < N) u = __ldg(reinterpret_cast<const uint4*>(We + (size_t)(k0 + k) * N + n0 + c));
        *reinterpret_cast<uint4*>(&sm[k][c]) = u;
    }
    __syncthreads();
    const int n = threadIdx.x % WN, kb = threadIdx.x / WN;
    float v[32];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        v[i] = to_f<T>(sm[kb * 32 + i][n]);
        m = max(m, abs_bits(v[i]));
    }
    const uint32_t s = mx8_scale_byte(m);
    uint32_t w[8];
    mx8_codes<32>(v, s, w);
    *reinterpret_cast<uint4*>(&sc[n][kb * 32]) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(&sc[n][kb * 32 + 16]) = make_uint4(w[4], w[5], w[6], w[7]);
    sb[n][kb] = (uint8_t)s;
    __syncthreads();
    const size_t block = ((size_t)e * (gridDim.y / 2) + blockIdx.y / 2) * gridDim.x + blockIdx.x;
    const int r0 = blockIdx.y % 2 * WN;                     // this half's first row
    uint8_t* dst = codes + block * 16384 + r0 * 128;
#pragma unroll
    for (int i = threadIdx.x; i < WN * 8; i += W_THREADS)
        *reinterpret_cast<uint4*>(dst + i * 16) = *reinterpret_cast<const uint4*>(&sc[i / 8][i % 8 * 16]);
    if (threadIdx.x < WN) {
        const int r = r0 + threadIdx.x;
        *reinterpret_cast<uint32_t*>(scales + block * 512 + r % 32 * 16 + r / 32 * 4) =
            *reinterpret_cast<const uint32_t*>(sb[threadIdx.x]);
    }
}

// The values of weights: 16 codes a thread, out [E, N, K] written along K
template <typename T>
__global__ void __launch_bounds__(256) mx8_weight_values_kernel(const uint8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, int K, int N,
                                                                T* __restrict__ out) {
    pdl_wait();
    pdl_trigger();
    const int kt = (K + 127) / 128, nt = (N + 127) / 128, e = blockIdx.z;
    const int k = (blockIdx.x % kt * 8 + (threadIdx.x & 7)) * 16, n = blockIdx.x / kt * 32 + (threadIdx.x >> 3);
    if (k >= K || n >= N) return;
    const size_t block = ((size_t)e * nt + n / 128) * kt + k / 128;
    const int r = n % 128;
    const uint4 c = __ldg(reinterpret_cast<const uint4*>(codes + block * 16384 + r * 128 + k % 128));
    const float m = mx8_scale_value(__ldg(scales + block * 512 + r % 32 * 16 + r / 32 * 4 + k % 128 / 32));
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    float v[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) mx8_unpack4(w[i], v + 4 * i);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= m;
    T* dst = out + ((size_t)e * N + n) * K + k;
#pragma unroll
    for (int i = 0; i < 16; i += Vec16<T>::N) store16_f<T>(dst + i, v + i);
}

// Rows of 8-bit numbers to their places: a warp takes a token and writes each of its
// slots, so a row is read once however many experts it goes to.  32768 x 2048 to eight
// experts each: 101 us (6.2 TB/s); with the two launches that find the places 118.
__global__ void __launch_bounds__(256) mx8_scatter_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                          const int32_t* __restrict__ slot_of, int T, int k, int d, int pitch,
                                                          uint8_t* __restrict__ codes_perm, uint8_t* __restrict__ scales_perm) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, nc = d / 16, nv = nc + pitch / 16;
    for (int t = blockIdx.x * 8 + (threadIdx.x >> 5); t < T; t += gridDim.x * 8) {
        const int mine = lane < k ? slot_of[(size_t)t * k + lane] : -1;
        const uint4* c = reinterpret_cast<const uint4*>(codes + (size_t)t * d);
        const uint4* s = reinterpret_cast<const uint4*>(scales + (size_t)t * pitch);
        for (int v0 = 0; v0 < nv; v0 += 128) {
            uint4 r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int v = v0 + i * 32 + lane;
                if (v < nv) r[i] = __ldg(v < nc ? c + v : s + v - nc);
            }
            for (int j = 0; j < k; ++j) {
                const int row = __shfl_sync(0xffffffffu, mine, j);
                if (row < 0) continue;
                uint4* dc = reinterpret_cast<uint4*>(codes_perm + (size_t)row * d);
                uint4* ds = reinterpret_cast<uint4*>(scales_perm + (size_t)row * pitch);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int v = v0 + i * 32 + lane;
                    if (v < nv) *(v < nc ? dc + v : ds + v - nc) = r[i];
                }
            }
        }
    }
}

// A batch of up to 256 tokens in one launch: every CTA finds all places by itself (a thread
// a token; ranks by lane masks, as in permute.cu), the first writes them down, and each
// copies its tokens' rows.  Three launches for 17 tokens took 6.0 us.
constexpr int FEW = 256;
__global__ void __launch_bounds__(FEW) mx8_dispatch_few_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, const int32_t* __restrict__ topk, int T, int E,
    int k, int C, int d, int pitch, uint8_t* __restrict__ codes_perm, uint8_t* __restrict__ scales_perm,
    int32_t* __restrict__ perm_token, int32_t* __restrict__ slot_of, int32_t* __restrict__ kept,
    int32_t* __restrict__ offsets, float* __restrict__ stats, int* status) {
    pdl_wait();
    pdl_trigger();
    __shared__ unsigned picks[FEW / 32][64];   // per warp and expert, the lanes whose token picks it
    __shared__ int s_off[65], s_slot[FEW][8];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const bool first = blockIdx.x == 0;
    for (int i = t; i < FEW / 32 * 64; i += FEW) (&picks[0][0])[i] = 0;
    __syncthreads();
    int sel[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        sel[j] = t < T && j < k ? topk[t * k + j] : -1;
        if (first && (sel[j] < -1 || sel[j] >= E)) set_status(status, MOE_ERR_DEVICE_BOUNDS);
        if (sel[j] >= 0 && sel[j] < E) atomicOr(&picks[warp][sel[j]], 1u << lane);
    }
    __syncthreads();
    if (warp == 0) {                       // segments: two experts a lane
        int n[2], total[2], before = 0;
        long dropped = 0;
        int kmax = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = lane + 32 * i;
            total[i] = 0;
            if (e < E)
                for (int w = 0; w < FEW / 32; ++w) total[i] += __popc(picks[w][e]);
            n[i] = min(total[i], C);
            int sum = n[i];
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            if (e < E) s_off[e] = before + sum - n[i];
            before += __shfl_sync(0xffffffffu, sum, 31);
            dropped += total[i] - n[i];
            kmax = max(kmax, n[i]);
        }
        if (lane == 0) s_off[E] = before;
        if (first) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int e = lane + 32 * i;
                if (e < E) {
                    kept[e] = n[i];
                    offsets[e] = s_off[e];
                }
            }
            int drop = (int)dropped;
            for (int o = 16; o > 0; o >>= 1) {
                drop += __shfl_xor_sync(0xffffffffu, drop, o);
                kmax = max(kmax, __shfl_xor_sync(0xffffffffu, kmax, o));
            }
            if (lane == 0) {
                offsets[E] = before;
                if (stats) {
                    stats[MOE_STAT_DROPPED] = (float)drop;
                    stats[MOE_STAT_MAX_OVER_MEAN_KEPT] = before > 0 ? (float)kmax / ((float)before / (float)E) : 0.f;
                }
            }
        }
    }
    __syncthreads();
    if (t < T)
        for (int j = 0; j < k; ++j) {
            int slot = -1;
            if (sel[j] >= 0 && sel[j] < E) {
                int r = __popc(picks[warp][sel[j]] & ((1u << lane) - 1u));
                for (int w = 0; w < warp; ++w) r += __popc(picks[w][sel[j]]);
                if (r < C) slot = s_off[sel[j]] + r;
            }
            s_slot[t][j] = slot;
            if (first) {
                slot_of[t * k + j] = slot;
                if (slot >= 0) perm_token[slot] = t;
            }
        }
    __syncthreads();
    const int nc = d / 16, nv = nc + pitch / 16;
    for (int row = blockIdx.x; row < T; row += gridDim.x)
        for (int v = t; v < nv; v += FEW) {
            const bool code = v < nc;
            const uint4 x = __ldg(code ? reinterpret_cast<const uint4*>(codes + (size_t)row * d) + v
                                       : reinterpret_cast<const uint4*>(scales + (size_t)row * pitch) + v - nc);
            for (int j = 0; j < k; ++j) {
                const int to = s_slot[row][j];
                if (to >= 0)
                    *(code ? reinterpret_cast<uint4*>(codes_perm + (size_t)to * d) + v
                           : reinterpret_cast<uint4*>(scales_perm + (size_t)to * pitch) + v - nc) = x;
            }
        }
}

template <typename T>
int rows_t(int64_t rows, int K, const void* x, const int32_t* used, void* codes, void* scales, cudaStream_t st) {
    const Turns t = turns_of(rows, K / Raw32<T>::N);
    MOE_LAUNCH(mx8_rows_kernel<T>, turn_grid(t), ROW_THREADS, 0, st, static_cast<const T*>(x), t, K, (int)mx8_pitch(K), used,
               static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
    return MOE_OK;
}
template <typename T>
int weight_t(int E, int K, int N, const void* W, void* codes, void* scales, cudaStream_t st) {
    const dim3 grid((K + 127) / 128, (N + 127) / 128 * 2, E);
    MOE_LAUNCH(mx8_weight_kernel<T>, grid, W_THREADS, 0, st, static_cast<const T*>(W), K, N, static_cast<uint8_t*>(codes),
               static_cast<uint8_t*>(scales));
    return MOE_OK;
}
template <typename T>
int weight_values_t(int E, int K, int N, const void* codes, const void* scales, void* out, cudaStream_t st) {
    const dim3 grid((K + 127) / 128 * ((N + 31) / 32), 1, E);
    MOE_LAUNCH(mx8_weight_values_kernel<T>, grid, 256, 0, st, static_cast<const uint8_t*>(codes),
               static_cast<const uint8_t*>(scales), K, N, static_cast<T*>(out));
    return MOE_OK;
}
template <typename T>
int values_t(int64_t rows, int K, const void* codes, const void* scales, void* out, cudaStream_t st) {
    const Turns t = turns_of(rows, K / Vec16<T>::N);
    MOE_LAUNCH(mx8_values_kernel<T>, turn_grid(t), ROW_THREADS, 0, st, static_cast<const uint8_t*>(codes),
               static_cast<const uint8_t*>(scales), t, K, (int)mx8_pitch(K), static_cast<T*>(out));
    return MOE_OK;
}

}  // namespace

int launch_mx8_quantize(int dtype, int64_t rows, int K, const void* x, const int32_t* rows_used, void* codes,
                        void* scales, cudaStream_t st) {
    return dtype == MOE_DTYPE_BF16 ? rows_t<__nv_bfloat16>(rows, K, x, rows_used, codes, scales, st)
                                   : rows_t<float>(rows, K, x, rows_used, codes, scales, st);
}
int launch_mx8_quantize_weight(int dtype, int E, int K, int N, const void* W, void* codes, void* scales,
                               cudaStream_t st) {
    return dtype == MOE_DTYPE_BF16 ? weight_t<__nv_bfloat16>(E, K, N, W, codes, scales, st)
                                   : weight_t<float>(E, K, N, W, codes, scales, st);
}
int launch_mx8_dequantize(int dtype, int64_t rows, int K, const void* codes, const void* scales, void* out,
                          cudaStream_t st) {
    return dtype == MOE_DTYPE_BF16 ? values_t<__nv_bfloat16>(rows, K, codes, scales, out, st)
                                   : values_t<float>(rows, K, codes, scales, out, st);
}
int launch_mx8_dequantize_weight(int dtype, int E, int K, int N, const void* codes, const void* scales, void* out,
                                 cudaStream_t st) {
    return dtype == MOE_DTYPE_BF16 ? weight_values_t<__nv_bfloat16>(E, K, N, codes, scales, out, st)
                                   : weight_values_t<float>(E, K, N, codes, scales, out, st);
}
int launch_permute_mx8(const moe_config& c, const void* codes, const void* scales, const int32_t* topk,
                       void* codes_perm, void* scales_perm, int32_t* perm_token, int32_t* slot_of, int32_t* kept,
                       int32_t* offsets, float* stats, void* ws, cudaStream_t st) {
    if (c.T <= FEW) {
        MOE_LAUNCH(mx8_dispatch_few_kernel, std::min(c.T, num_sms()), FEW, 0, st, static_cast<const uint8_t*>(codes),
                   static_cast<const uint8_t*>(scales), topk, c.T, c.E, c.k, capacity_of(c), c.d, (int)mx8_pitch(c.d),
                   static_cast<uint8_t*>(codes_perm), static_cast<uint8_t*>(scales_perm), perm_token, slot_of, kept,
                   offsets, stats, device_status_ptr());
        return MOE_OK;
    }
    if (const int r = launch_permute_index(c, 1, topk, perm_token, slot_of, kept, offsets, stats, ws, st)) return r;
    const int grid = std::min((c.T + 7) / 8, num_sms() * 8);
    MOE_LAUNCH(mx8_scatter_kernel, grid, 256, 0, st, static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales),
               slot_of, c.T, c.k, c.d, (int)mx8_pitch(c.d), static_cast<uint8_t*>(codes_perm),
               static_cast<uint8_t*>(scales_perm));
    return MOE_OK;
}

}  // namespace moe
