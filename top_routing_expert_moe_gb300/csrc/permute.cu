// permute.cu -- capacity dropping and the expert-contiguous permutation.
//
// [LLaMA4-MoE] §2.4: sort the [B,K] index by expert id, take each expert's
// token-count interval, split, run each expert.  [ZeRO3-MoE] §3.1/§3.4:
// a per-expert capacity (capacity_factor) caps the tokens an expert takes.
//
// A stable counting sort, deterministic (no order-dependent atomics):
//   1. tile histogram: per 256-token tile, selections per expert;
//   2. per tile (one CTA each): the expert's tokens in earlier tiles and in all
//      tiles (every CTA sums the small histogram itself, so no separate scan
//      launch), the capacity and the padded segments (offsets); then bit masks of
//      the warps' lanes give each assignment its rank among the expert's assignments
//      in token order; rank < C keeps it at row offsets[e] + rank; padding rows
//      are marked, each CTA a strided share of them;
//   3. gather: one warp per destination row copies the token's x row with
//      16-byte vectors (zeros on padding rows), rows read from device offsets.
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int PT_TOK = 256;  // tokens per tile (one per thread)

__global__ void __launch_bounds__(PT_TOK) tile_hist_kernel(const int32_t* __restrict__ topk,
                                                           int T, int E, int k,
                                                           int32_t* __restrict__ tile_counts,
                                                           int* status)
{
    pdl_wait();      // the preceding kernel's writes are visible from here on
    pdl_trigger();
    __shared__ int h[64];
    if (threadIdx.x < E) h[threadIdx.x] = 0;
    __syncthreads();
    const int t = blockIdx.x * PT_TOK + threadIdx.x;
    if (t < T) {
        unsigned long long seen = 0;               // an expert named twice takes the token once
        for (int j = 0; j < k; ++j) {
            const int e = topk[(size_t)t * k + j];
            if (e >= 0 && e < E) {
                if (!(seen >> e & 1)) atomicAdd(&h[e], 1);  // integer count: order-free
                seen |= 1ull << e;
            } else if (e != -1) {
                set_status(status, MOE_ERR_DEVICE_BOUNDS);  // -1: masked token
            }
        }
    }
    __syncthreads();
    if (threadIdx.x < E) tile_counts[(size_t)blockIdx.x * E + threadIdx.x] = h[threadIdx.x];
}

// One CTA per 256-token tile.  Its threads sum the experts' counts over the earlier
// tiles (this tile's first rank) and over all tiles, neighbouring threads neighbouring
// experts (a warp per expert read the histogram across: 32768 tokens, 64 experts, top-8:
// 26 us for this kernel); a warp then applies the capacity and lays out the padded
// segments (every CTA finds the same layout; CTA 0 writes offsets, kept and the
// statistics).
__global__ void __launch_bounds__(PT_TOK) scan_assign_kernel(
    const int32_t* __restrict__ topk, int T, int E, int k, int C, int pad_m,
    const int32_t* __restrict__ tile_counts, int ntiles, int32_t* __restrict__ kept,
    int32_t* __restrict__ offsets, int32_t* __restrict__ slot_of, int32_t* __restrict__ perm_token,
    float* __restrict__ stats)
{
    pdl_wait();      // the preceding kernel's writes are visible from here on
    pdl_trigger();
    __shared__ int s_base[64], s_total[64], s_off[65];
    __shared__ unsigned picks[PT_TOK / 32][64];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int blk = blockIdx.x;
    const int t = blk * PT_TOK + tid;
    int sel[8];                                           // (asked for ahead of the histogram)
#pragma unroll
    for (int j = 0; j < 8; ++j) sel[j] = (j < k && t < T) ? topk[(size_t)t * k + j] : -1;
    if (tid < 64) s_base[tid] = s_total[tid] = 0;
    for (int i = tid; i < PT_TOK / 32 * 64; i += PT_TOK) (&picks[0][0])[i] = 0;
    __syncthreads();
    const int shift = E > 1 ? 32 - __clz(E - 1) : 0;      // threads in groups of 2^shift >= E
    const int e0 = tid & ((1 << shift) - 1), step = PT_TOK >> shift;
    if (e0 < E) {
        int before = 0, total = 0;
#pragma unroll 8
        for (int b = tid >> shift; b < ntiles; b += step) {
            const int v = tile_counts[(size_t)b * E + e0];
            total += v;
            if (b < blk) before += v;
        }
        atomicAdd(&s_base[e0], before);                   // integers: order-free
        atomicAdd(&s_total[e0], total);
    }
    // for the ranks within the tile: per warp and expert, the lanes whose token picks it
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (sel[j] >= 0 && sel[j] < E) atomicOr(&picks[warp][sel[j]], 1u << lane);
    __syncthreads();
    if (warp == 0) {                                      // two experts a lane
        int off = 0, kmax = 0;
        long long ksum = 0, dropped = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = lane + 32 * i;
            const int total = e < E ? s_total[e] : 0, ke = min(total, C);
            const int padded = (ke + pad_m - 1) / pad_m * pad_m;
            int sum = padded;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            if (e < E) {
                s_off[e] = off + sum - padded;
                if (blk == 0) {
                    offsets[e] = off + sum - padded;
                    kept[e] = ke;
                }
            }
            off += __shfl_sync(0xffffffffu, sum, 31);
            kmax = max(kmax, ke);
            ksum += ke;
            dropped += total - ke;
        }
        if (lane == 0) s_off[E] = off;
        if (blk == 0) {
            for (int o = 16; o > 0; o >>= 1) {
                kmax = max(kmax, __shfl_xor_sync(0xffffffffu, kmax, o));
                ksum += __shfl_xor_sync(0xffffffffu, ksum, o);
                dropped += __shfl_xor_sync(0xffffffffu, dropped, o);
            }
            if (lane == 0) {
                offsets[E] = off;
                if (stats) {
                    stats[MOE_STAT_DROPPED] = (float)dropped;
                    stats[MOE_STAT_MAX_OVER_MEAN_KEPT] =
                        ksum > 0 ? (float)kmax / ((float)ksum / (float)E) : 0.f;
                }
            }
        }
    }
    __syncthreads();
    // padding rows carry token -1 (this CTA: every ntiles-th group of 256 rows)
    for (int e = 0; e < E; ++e) {
        const int end = s_off[e + 1];
        for (int r = s_off[e] + min(s_total[e], C) + blk * PT_TOK + tid; r < end; r += ntiles * PT_TOK)
            perm_token[r] = -1;
    }
    if (t >= T) return;
    const unsigned lt = (1u << lane) - 1u;
    for (int j = 0; j < k; ++j) {
        const int e = sel[j];
        if (e < 0 || e >= E) { slot_of[(size_t)t * k + j] = -1; continue; }
        int r = s_base[e] + __popc(picks[warp][e] & lt);
        for (int w = 0; w < warp; ++w) r += __popc(picks[w][e]);
        if (r < C) {
            const int row = s_off[e] + r;
            slot_of[(size_t)t * k + j] = row;
            perm_token[row] = t;
        } else {
            slot_of[(size_t)t * k + j] = -1;
        }
    }
}

// one warp per destination row; 16-byte vectors; the row count is read on the device
template <typename T>
__global__ void __launch_bounds__(256) gather_rows_kernel(const T* __restrict__ x,
                                                          const int32_t* __restrict__ perm_token,
                                                          const int32_t* __restrict__ offsets,
                                                          int E, int d, T* __restrict__ x_perm)
{
    pdl_wait();      // the preceding kernel's writes are visible from here on
    pdl_trigger();
    constexpr int V = 16 / sizeof(T);
    const int rows = offsets[E];
    const int nv = d / V;
    const int warps = gridDim.x * (blockDim.x >> 5);
    for (int r = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); r < rows; r += warps) {
        const int t = perm_token[r];
        uint4* dst = reinterpret_cast<uint4*>(x_perm + (size_t)r * d);
        if (t < 0) {
            for (int v = threadIdx.x & 31; v < nv; v += 32) dst[v] = make_uint4(0, 0, 0, 0);
        } else {
            const uint4* src = reinterpret_cast<const uint4*>(x + (size_t)t * d);
            int v = threadIdx.x & 31;
            for (; v + 96 < nv; v += 128) {
                uint4 a = __ldg(src + v), b = __ldg(src + v + 32), c = __ldg(src + v + 64),
                      e = __ldg(src + v + 96);
                dst[v] = a; dst[v + 32] = b; dst[v + 64] = c; dst[v + 96] = e;
            }
            for (; v < nv; v += 32) dst[v] = __ldg(src + v);
        }
    }
}

}  // namespace

size_t permute_ws_bytes(const moe_config& c) {
    const size_t ntiles = (size_t)(c.T + PT_TOK - 1) / PT_TOK;
    return align_up(ntiles * c.E * 4);
}

int launch_permute_index(const moe_config& c, int pad_m, const int32_t* topk, int32_t* perm_token,
                         int32_t* slot_of, int32_t* kept, int32_t* offsets, float* stats, void* ws,
                         cudaStream_t st)
{
    const int ntiles = (c.T + PT_TOK - 1) / PT_TOK;
    int32_t* tile_counts = static_cast<int32_t*>(ws);
    const int C = capacity_of(c);
    MOE_LAUNCH(tile_hist_kernel, ntiles, PT_TOK, 0, st, topk, c.T, c.E, c.k, tile_counts,
                                                device_status_ptr());
    MOE_LAUNCH(scan_assign_kernel, ntiles, PT_TOK, 0, st, topk, c.T, c.E, c.k, C, pad_m, tile_counts,
               ntiles, kept, offsets, slot_of, perm_token, stats);
    return MOE_OK;
}

int launch_permute(const moe_config& c, const void* x, const int32_t* topk, void* x_perm,
                   int32_t* perm_token, int32_t* slot_of, int32_t* kept, int32_t* offsets,
                   float* stats, void* ws, cudaStream_t st)
{
    if (const int r = launch_permute_index(c, c.pad_m, topk, perm_token, slot_of, kept, offsets, stats,
                                           ws, st))
        return r;
    const int64_t rows = rows_cap_of(c);
    const int grid = (int)std::min<int64_t>((rows + 7) / 8, (int64_t)num_sms() * 8);
    if (c.dtype == MOE_DTYPE_BF16)
        MOE_LAUNCH(gather_rows_kernel<__nv_bfloat16>, grid, 256, 0, st, static_cast<const __nv_bfloat16*>(x), perm_token, offsets, c.E, c.d,
            static_cast<__nv_bfloat16*>(x_perm));
    else
        MOE_LAUNCH(gather_rows_kernel<float>, grid, 256, 0, st, static_cast<const float*>(x), perm_token,
                                                        offsets, c.E, c.d,
                                                        static_cast<float*>(x_perm));
    return MOE_OK;
}

}  // namespace moe
