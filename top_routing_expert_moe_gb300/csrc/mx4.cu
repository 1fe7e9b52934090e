// mx4.cu -- microscaled 4-bit numbers: quantisation of rows and of expert
// weights, and the values that codes and scales stand for.
//
// A block of 32 elements along the reduction axis shares the scale 2^(s-127),
//   s = max(exponent(amax) - 2, 0)     (255 where an element is Inf or NaN),
// so that amax / scale lies in [4, 8) and the largest code, 6, is reached.  All
// steps are exact but the rounding to a code (nearest, ties to even, by the
// conversion instruction): the results do not depend on any order.
//
// Memory-bound: 2 (or 4) bytes read, 17/32 written an element.  65536 x 4096 bf16 rows
// 106 us (6.4 TB/s), back to values 117 us (5.8 TB/s); fp32 178 us (6.8 TB/s) and 261 us
// (4.7); weights of 8 x 2048 x 4096 31 us (5.5 TB/s).  Decoding each code by its bits and finding each element's place by
// division took 296 us where byte tables and the quantiser's split take 115.
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

// Magnitudes compare as their bits do, NaN above Inf.  A bf16 pair's are compared
// in one instruction, and their maximum stands in the upper half as fp32's would.
template <typename T> struct Raw8;                          // 8 elements as loaded
template <> struct Raw8<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ uint32_t amax() const {
        const uint32_t k = 0x7fff7fffu;
        const uint32_t m = __vmaxu2(__vmaxu2(w.x & k, w.y & k), __vmaxu2(w.z & k, w.w & k));
        return max(m & 0xffff0000u, m << 16);
    }
    __device__ __forceinline__ void values(float* v) const {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(a[i] << 16);
            v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
        }
    }
};
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void values(float* v) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    __device__ __forceinline__ uint32_t amax() const {
        float v[8];
        values(v);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
        return m;
    }
};

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
    const uint32_t nch = (K + 255) / 256, kt = (K + 127) / 128;
    int64_t used = rows;
    if (rows_used) used = min(rows, (int64_t)max(*rows_used, 0));
    const uint32_t tiles = (uint32_t)((used + 127) / 128);
    const int shift = 8 * ((lane >> 2) & 3);
    // blockIdx.y: chunk of columns; warps: (row in tile, tile), neighbours in a tile
    for (uint32_t it = blockIdx.x * 8 + (threadIdx.x >> 5); it < tiles * 32; it += gridDim.x * 8) {
        const uint32_t r = it & 31, tile = it >> 5;
        const int64_t row0 = (int64_t)tile * 128 + r;
        for (uint32_t ch = blockIdx.y; ch < nch; ch += gridDim.y) {
            const int col = ch * 256 + lane * 8;
            const bool in = col < K;
            Raw8<T> raw[4];
            uint32_t word[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (in && row0 + 32 * j < used) raw[j].load(x + (row0 + 32 * j) * K + col);
                else raw[j].zero();
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t m = raw[j].amax();
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const uint32_t s = scale_byte(m);
                float v[8];
                raw[j].values(v);
                const uint32_t c = codes8(v, s);
                if (in && row0 + 32 * j < used)
                    *reinterpret_cast<uint32_t*>(codes + (row0 + 32 * j) * (K / 2) + col / 2) = c;
                uint32_t w = s << shift;                    // the scale tile's word of this row
                w |= __shfl_xor_sync(0xffffffffu, w, 4);
                word[j] = w | __shfl_xor_sync(0xffffffffu, w, 8);
            }
            const uint32_t t = ch * 2 + (lane >> 4);
            if ((lane & 15) == 0 && t < kt)
                *reinterpret_cast<uint4*>(scales + ((size_t)tile * kt + t) * 512 + r * 16) =
                    make_uint4(word[0], word[1], word[2], word[3]);
        }
    }
}

// Two neighbouring columns' elements, as loaded.
template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    uint32_t w;
    __device__ __forceinline__ float lo() const { return __uint_as_float(w << 16); }
    __device__ __forceinline__ float hi() const { return __uint_as_float(w & 0xffff0000u); }
};
template <> struct __align__(8) Pair<float> {
    float a, b;
    __device__ __forceinline__ float lo() const { return a; }
    __device__ __forceinline__ float hi() const { return b; }
};
// the largest magnitudes' bits of both columns over a block
__device__ __forceinline__ uint2 amax32(const Pair<__nv_bfloat16> (&v)[32]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) m = __vmaxu2(m, v[i].w & 0x7fff7fffu);
    return make_uint2(m << 16, m & 0xffff0000u);
}
__device__ __forceinline__ uint2 amax32(const Pair<float> (&v)[32]) {
    uint2 m = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        m.x = max(m.x, __float_as_uint(v[i].a) & 0x7fffffffu);
        m.y = max(m.y, __float_as_uint(v[i].b) & 0x7fffffffu);
    }
    return m;
}

// Weights W [E, K, N] -> [E, N, K / 2]: a CTA takes 128 k x 64 n through shared
// memory; a thread forms one block (32 k) of two neighbouring columns, which it
// reads as pairs and holds in registers.
constexpr int WN = 64, W_THREADS = WN / 2 * 4;
template <typename T>
__global__ void __launch_bounds__(W_THREADS) mx4_weight_kernel(const T* __restrict__ W, int K, int N,
                                                               uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales) {
    pdl_wait();
    pdl_trigger();
    constexpr int V = 16 / sizeof(T);
    __shared__ __align__(16) T sm[128][WN + V];
    __shared__ __align__(4) uint8_t sb[WN][4];
    const int kt = (K + 127) / 128, nt = (N + 127) / 128;
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
    const int n = threadIdx.x % (WN / 2) * 2, kb = threadIdx.x / (WN / 2);
    Pair<T> v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = *reinterpret_cast<const Pair<T>*>(&sm[kb * 32 + i][n]);
    const uint2 m = amax32(v);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t s = scale_byte(h ? m.y : m.x);
        uint32_t c[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = h ? v[q * 8 + i].hi() : v[q * 8 + i].lo();
            c[q] = codes8(f, s);
        }
        if (n0 + n + h < N && k0 + kb * 32 < K)
            *reinterpret_cast<uint4*>(codes + ((size_t)e * N + n0 + n + h) * (K / 2) + k0 / 2 + kb * 16) =
                make_uint4(c[0], c[1], c[2], c[3]);
        sb[n + h][kb] = (uint8_t)s;                         // (0 past the tensor's end: m = 0)
    }
    __syncthreads();
    if (threadIdx.x < WN) {
        const int row = n0 + threadIdx.x;
        *reinterpret_cast<uint32_t*>(scales + (((size_t)e * nt + row / 128) * kt + blockIdx.x) * 512 +
                                     (row % 32) * 16 + (row % 128) / 32 * 4) =
            *reinterpret_cast<const uint32_t*>(sb[threadIdx.x]);
    }
}

// Four codes (the low 16 bits of c) as bf16 pairs, by byte tables: a byte permute
// picks each code's high and low byte by its magnitude bits, the signs are spread
// over the high bytes.
__device__ __forceinline__ uint2 values4(uint32_t c) {
    const uint32_t sel = c & 0x7777u;
    uint32_t hi = __byte_perm(0x3f3f3f00u, 0x40404040u, sel);       // 0 .5 1 1.5 | 2 3 4 6
    const uint32_t lo = __byte_perm(0xc0800000u, 0xc0804000u, sel);
    uint32_t s = (c & 0x88u) | ((c & 0x8800u) << 8);
    s = ((s << 4) & 0x00800080u) | ((s << 8) & 0x80008000u);        // code j's sign at bit 8 j + 7
    hi |= s;
    return make_uint2(__byte_perm(lo, hi, 0x5140), __byte_perm(lo, hi, 0x7362));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Values of codes and scales, by the quantiser's split: a warp takes 256 columns of
// four rows of a scale tile, 8 columns a lane.  Codes and scales are powers of two
// times 0..1.5, exact in bf16, and so are their products.
template <typename T>
__global__ void __launch_bounds__(256) mx4_values_kernel(const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales,
                                                         int64_t rows, int sets, int K,
                                                         T* __restrict__ out) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const uint32_t nch = (K + 255) / 256, kt = (K + 127) / 128, rt = (uint32_t)((rows + 127) / 128);
    const uint32_t tiles = rt * sets;                      // row tiles over all sets
    // blockIdx.y: chunk of columns; warps: (row in tile, tile)
    for (uint32_t it = blockIdx.x * 8 + (threadIdx.x >> 5); it < tiles * 32; it += gridDim.x * 8) {
        const uint32_t r = it & 31, tile = it >> 5;
        const uint32_t set = sets == 1 ? 0 : tile / rt;
        const int64_t row0 = (int64_t)(tile - set * rt) * 128 + r;
        for (uint32_t ch = blockIdx.y; ch < nch; ch += gridDim.y) {
            const int col = ch * 256 + lane * 8;
            if (col >= K) continue;
            const uint4 sw = __ldg(reinterpret_cast<const uint4*>(
                scales + ((size_t)tile * kt + ch * 2 + (lane >> 4)) * 512 + r * 16));
            const uint32_t words[4] = {sw.x, sw.y, sw.z, sw.w};
            uint32_t c[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (row0 + 32 * j < rows)
                    c[j] = __ldg(reinterpret_cast<const uint32_t*>(codes + ((size_t)set * rows + row0 + 32 * j) * (K / 2) + col / 2));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (row0 + 32 * j >= rows) break;
                const uint32_t sb = (words[j] >> (8 * ((lane >> 2) & 3))) & 255u;
                uint32_t sc = __float_as_uint(scale_value(sb)) >> 16;
                sc |= sc << 16;
                const uint2 a = values4(c[j]), b = values4(c[j] >> 16);
                const uint32_t v[4] = {mul_bf16x2(a.x, sc), mul_bf16x2(a.y, sc), mul_bf16x2(b.x, sc),
                                       mul_bf16x2(b.y, sc)};
                T* dst = out + ((size_t)set * rows + row0 + 32 * j) * K + col;
                if constexpr (sizeof(T) == 2) {
                    *reinterpret_cast<uint4*>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        *reinterpret_cast<uint4*>(dst + 4 * h) =
                            make_uint4(v[2 * h] << 16, v[2 * h] & 0xffff0000u, v[2 * h + 1] << 16, v[2 * h + 1] & 0xffff0000u);
                }
            }
        }
    }
}

// CTAs of the two kernels above: 8 warps each over the row tiles' 32 row groups, and
// over the 256-column chunks
dim3 tile_grid(int64_t row_tiles, int K) {
    const int nch = (K + 255) / 256;
    const int gx = (int)std::min<int64_t>(row_tiles * 4, (int64_t)num_sms() * 32);
    const int gy = (int)std::min<int64_t>(nch, std::max<int64_t>(1, (int64_t)num_sms() * 32 / gx));
    return dim3(std::max(1, gx), gy);
}

template <typename T>
int rows_t(int64_t rows, int K, const void* x, const int32_t* used, void* codes, void* scales, cudaStream_t st) {
    MOE_LAUNCH(mx4_rows_kernel<T>, tile_grid((rows + 127) / 128, K), 256, 0, st, static_cast<const T*>(x), rows, K, used,
               static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
    return MOE_OK;
}
template <typename T>
int weight_t(int E, int K, int N, const void* W, void* codes, void* scales, cudaStream_t st) {
    // both 64-column halves of every 128-row scale tile, past the end too (their bytes are 0)
    const dim3 grid((K + 127) / 128, (N + 127) / 128 * 2, E);
    MOE_LAUNCH(mx4_weight_kernel<T>, grid, W_THREADS, 0, st, static_cast<const T*>(W), K, N,
               static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
    return MOE_OK;
}
template <typename T>
int values_t(int sets, int64_t rows, int K, const void* codes, const void* scales, void* out, cudaStream_t st) {
    MOE_LAUNCH(mx4_values_kernel<T>, tile_grid((rows + 127) / 128 * sets, K), 256, 0, st, static_cast<const uint8_t*>(codes),
               static_cast<const uint8_t*>(scales), rows, sets, K, static_cast<T*>(out));
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
