// mx4.cu -- microscaled 4-bit numbers: quantisation of rows and of expert
// weights, and the values that codes and scales stand for.
//
// A block of 32 elements along the reduction axis shares the scale 2^(s-127),
//   s = max(exponent(amax) - 2, 0)     (255 where an element is Inf or NaN),
// so that amax / scale lies in [4, 8) and the largest code, 6, is reached.  All
// steps are exact but the rounding to a code (nearest, ties to even, by the
// conversion instruction): the results do not depend on any order.
//
// Memory-bound: 2 (or 4) bytes read, 17/32 written an element.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

// scale byte of a block with largest magnitude m (>= 0, Inf or NaN: 255)
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    const uint32_t e = amax_bits >> 23;
    return e == 255 ? 255u : (e > 2 ? e - 2 : 0u);
}
// 2^(127 - s): what a block's elements are multiplied by (0 for s = 255: codes 0)
__device__ __forceinline__ float inv_scale(uint32_t s) { return __uint_as_float(s == 255 ? 0u : (254 - s) << 23); }
// 2^(s - 127), NaN for s = 255
__device__ __forceinline__ float scale_value(uint32_t s) {
    return __uint_as_float(s == 255 ? 0x7fc00000u : s == 0 ? 0x00400000u : s << 23);
}

// 8 values -> 8 codes, element 0 in the lowest 4 bits
__device__ __forceinline__ uint32_t pack8(const float* v) {
    uint32_t r;
    asm("{\n.reg .b8 b0, b1, b2, b3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        "mov.b32 %0, {b0, b1, b2, b3};\n}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
// a block of a 255 byte holds Inf or NaN: 0 times those is no number, so its codes are set to 0
__device__ __forceinline__ uint32_t codes8(float* v, uint32_t s) {
    const float m = inv_scale(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= m;
    return s == 255 ? 0u : pack8(v);
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* v) {
    load16_f<T>(p, v);
    if constexpr (sizeof(T) == 4) load16_f<T>(p + 4, v + 4);
}

// as integers magnitudes compare as their bits do, NaN above Inf
__device__ __forceinline__ uint32_t amax8(const float* v) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}

// Rows.  A warp takes 256 columns (8 a lane, so four lanes hold a block) of the
// four rows r, r + 32, r + 64, r + 96 of a 128-row tile: their scale words are
// neighbours in the scale tile and leave as one 16-byte store per 128 columns.
template <typename T>
__global__ void __launch_bounds__(256) mx4_rows_kernel(const T* __restrict__ x, int64_t rows, int K,
                                                       const int32_t* __restrict__ rows_used,
                                                       uint8_t* __restrict__ codes,
                                                       uint8_t* __restrict__ scales) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int nch = (K + 255) / 256, kt = (K + 127) / 128;
    int64_t used = rows;
    if (rows_used) used = min(rows, (int64_t)max(*rows_used, 0));
    const int64_t items = (used + 127) / 128 * 32 * nch;
    for (int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += (int64_t)gridDim.x * 8) {
        const int r = (int)(it & 31);                       // (rows fastest: neighbours share a tile)
        const int64_t rest = it >> 5;
        const int ch = (int)(rest % nch);
        const int64_t tile = rest / nch;
        const int col = ch * 256 + lane * 8;
        const bool in = col < K;
        float v[4][8];
        uint32_t word[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t row = tile * 128 + r + 32 * j;
            if (in && row < used) load8<T>(x + row * K + col, v[j]);
            else
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t row = tile * 128 + r + 32 * j;
            uint32_t m = amax8(v[j]);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const uint32_t s = scale_byte(m);
            const uint32_t c = codes8(v[j], s);
            if (in && row < used) *reinterpret_cast<uint32_t*>(codes + row * (K / 2) + col / 2) = c;
            uint32_t w = s << (8 * ((lane >> 2) & 3));      // the scale tile's word of this row
            w |= __shfl_xor_sync(0xffffffffu, w, 4);
            word[j] = w | __shfl_xor_sync(0xffffffffu, w, 8);
        }
        const int t = ch * 2 + (lane >> 4);
        if ((lane & 15) == 0 && t < kt)
            *reinterpret_cast<uint4*>(scales + (tile * kt + t) * 512 + r * 16) =
                make_uint4(word[0], word[1], word[2], word[3]);
    }
}

// Weights W [E, K, N] -> [E, N, K / 2]: a CTA takes 128 k x 64 n through shared
// memory; thread (n, kb) forms block kb of column n.
constexpr int WN = 64;
template <typename T>
__global__ void __launch_bounds__(256) mx4_weight_kernel(const T* __restrict__ W, int K, int N,
                                                         uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ scales) {
    pdl_wait();
    pdl_trigger();
    constexpr int V = 16 / sizeof(T);
    __shared__ __align__(16) T sm[128][WN + V];
    __shared__ uint8_t sb[WN][4];
    const int kt = (K + 127) / 128, nt = (N + 127) / 128;
    const int k0 = blockIdx.x * 128, n0 = blockIdx.y * WN, e = blockIdx.z;
    const T* We = W + (size_t)e * K * N;
    for (int i = threadIdx.x; i < 128 * (WN / V); i += 256) {
        const int k = i / (WN / V), c = i % (WN / V) * V;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (k0 + k < K && n0 + c < N) u = *reinterpret_cast<const uint4*>(We + (size_t)(k0 + k) * N + n0 + c);
        *reinterpret_cast<uint4*>(&sm[k][c]) = u;
    }
    __syncthreads();
    const int n = threadIdx.x % WN, kb = threadIdx.x / WN;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) m = max(m, __float_as_uint(to_f<T>(sm[kb * 32 + i][n])) & 0x7fffffffu);
    const uint32_t s = scale_byte(m);
    uint32_t c[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f<T>(sm[kb * 32 + q * 8 + i][n]);
        c[q] = codes8(v, s);
    }
    if (n0 + n < N && k0 + kb * 32 < K)
        *reinterpret_cast<uint4*>(codes + ((size_t)e * N + n0 + n) * (K / 2) + k0 / 2 + kb * 16) =
            make_uint4(c[0], c[1], c[2], c[3]);
    sb[n][kb] = (uint8_t)s;                                 // (0 past the tensor's end: m = 0)
    __syncthreads();
    if (threadIdx.x < WN) {
        const int row = n0 + threadIdx.x;
        *reinterpret_cast<uint32_t*>(scales + (((size_t)e * nt + row / 128) * kt + blockIdx.x) * 512 +
                                     (row % 32) * 16 + (row % 128) / 32 * 4) =
            *reinterpret_cast<const uint32_t*>(sb[threadIdx.x]);
    }
}

// Values of codes and scales: 8 a thread
template <typename T>
__global__ void __launch_bounds__(256) mx4_values_kernel(const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales,
                                                         int64_t rows, int64_t all_rows, int K,
                                                         T* __restrict__ out) {
    pdl_wait();
    pdl_trigger();
    const int kt = (K + 127) / 128, per = K / 8;
    const int64_t rt = (rows + 127) / 128, n = all_rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per;
        const int k = (int)(i - row * per) * 8;
        const int64_t set = row / rows, r = row - set * rows;
        const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + row * (K / 2) + k / 2);
        const uint32_t s = scales[((set * rt + r / 128) * kt + k / 128) * 512 + (r % 32) * 16 +
                                  (r % 128) / 32 * 4 + (k % 128) / 32];
        const float sc = scale_value(s);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t q = c >> (4 * j), e = (q >> 1) & 3, mt = q & 1;
            // +-2^(e-1) (1 + m/2), or +-m/2 for e = 0
            const float a = e ? __uint_as_float(((e + 126) << 23) | (mt << 22)) : (mt ? 0.5f : 0.f);
            v[j] = (q & 8 ? -a : a) * sc;
        }
        store16_f<T>(out + row * K + k, v);
        if constexpr (sizeof(T) == 4) store16_f<T>(out + row * K + k + 4, v + 4);
    }
}

template <typename T>
int rows_t(int64_t rows, int K, const void* x, const int32_t* used, void* codes, void* scales, cudaStream_t st) {
    const int64_t items = (rows + 127) / 128 * 32 * ((K + 255) / 256);
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>((items + 7) / 8, (int64_t)num_sms() * 32));
    MOE_LAUNCH(mx4_rows_kernel<T>, grid, 256, 0, st, static_cast<const T*>(x), rows, K, used,
               static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
    return MOE_OK;
}
template <typename T>
int weight_t(int E, int K, int N, const void* W, void* codes, void* scales, cudaStream_t st) {
    // both 64-column halves of every 128-row scale tile, past the end too (their bytes are 0)
    const dim3 grid((K + 127) / 128, (N + 127) / 128 * 2, E);
    MOE_LAUNCH(mx4_weight_kernel<T>, grid, 256, 0, st, static_cast<const T*>(W), K, N,
               static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
    return MOE_OK;
}
template <typename T>
int values_t(int sets, int64_t rows, int K, const void* codes, const void* scales, void* out, cudaStream_t st) {
    const int64_t n = sets * rows * (K / 8);
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>((n + 255) / 256, (int64_t)num_sms() * 64));
    MOE_LAUNCH(mx4_values_kernel<T>, grid, 256, 0, st, static_cast<const uint8_t*>(codes),
               static_cast<const uint8_t*>(scales), rows, sets * rows, K, static_cast<T*>(out));
    return MOE_OK;
}

}  // namespace

int launch_mx4_quantize(int dtype, int64_t rows, int K, const void* x, const int32_t* rows_used,
                        void* codes, void* scales, cudaStream_t st) {
    return dtype == MOE_DTYPE_BF16 ? rows_t<__nv_bfloat16>(rows, K, x, rows_used, codes, scales, st)
                                   : rows_t<float>(rows, K, x, rows_used, codes, scales, st);
}
int launch_mx4_quantize_weight(int dtype, int E, int K, int N, const void* W, void* codes, void* scales,
                               cudaStream_t st) {
    return dtype == MOE_DTYPE_BF16 ? weight_t<__nv_bfloat16>(E, K, N, W, codes, scales, st)
                                   : weight_t<float>(E, K, N, W, codes, scales, st);
}
int launch_mx4_dequantize(int dtype, int sets, int64_t rows, int K, const void* codes, const void* scales,
                          void* out, cudaStream_t st) {
    return dtype == MOE_DTYPE_BF16 ? values_t<__nv_bfloat16>(sets, rows, K, codes, scales, out, st)
                                   : values_t<float>(sets, rows, K, codes, scales, out, st);
}

}  // namespace moe
