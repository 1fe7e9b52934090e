// mx4_gemm.cu -- grouped product of the experts with both operands in
// microscaled 4-bit numbers, on the block-scaled tensor cores (sm_103a).
//
//   u[r, n] = sum_i x[r, i] W_e[n, i],  x and W e2m1 codes times 2^(s - 127) per
//   32 elements along i;  out = u, silu(u), or silu(g) u with g from a second W.
//
// A persistent kernel like the bf16 grouped GEMM (gemm_tc.cu): a CTA pair takes
// 256 rows x 256 accumulator columns, warp-specialised:
//   warp 0      TMA producer: per stage of 256 elements, 128 bytes a row, this
//               CTA's 128 rows of x, its 128 rows of W (for SwiGLU the even CTA's
//               are the gate's, the odd CTA's the up matrix's) and the scale tiles:
//               its rows' and all 256 columns'.
//   warp 1      the even CTA's thread copies the stage's scale tiles to tensor
//               memory (tcgen05.cp, 32 lanes x 16 bytes, to all four lane
//               quarters) and issues the block-scaled MMAs, 64 elements each.
//   warps 2-9   epilogue: activation, rounding, TMA stores of 32 x 64-byte boxes.
//
// Tensor memory: 512 columns = two accumulators of 256 that overlap in 32, and
// 24 columns of scales.  A tile's epilogue drains the overlapping columns first;
// the next tile's MMAs start as soon as it has.
//
// Codes are K-major with 128-byte swizzle, so a step of 64 elements (32 bytes)
// advances the descriptor as a bf16 step of 16 does.  A scale tile (128 rows x 4
// blocks, 512 bytes) is stored as tcgen05.cp takes it: row r's four bytes are
// word r / 32 of the 16 bytes of lane r % 32.
#include <cuda.h>

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "kernels.h"
#include "tma.cuh"

namespace moe {

namespace {

constexpr int BM = 128;                    // rows per CTA
constexpr int BN = 256;                    // accumulator columns per tile (SwiGLU: 128 gate + 128 up)
constexpr int BKB = 128;                   // bytes of a row per stage: 256 elements
constexpr int A_BYTES = BM * BKB;
constexpr int SF_TILE = 512;               // scale bytes of 128 rows x 128 elements
constexpr int NUM_EPI_WARPS = 8;
constexpr int NTHREADS = 64 + 32 * NUM_EPI_WARPS;
constexpr int STAGING_BYTES = NUM_EPI_WARPS * 4096;
constexpr int CTRL_BYTES = 1024;
constexpr int TMEM_COLS = 512;
constexpr int ACC1 = 224;                  // second accumulator's first column (columns 224-255 overlap)
constexpr int SFA_COL = 480, SFB_COL = 488;
constexpr int RASTER_ROWS = 4096;          // rows of x that pass over an expert's weights together

template <int CG> struct Ring {            // CG CTAs a tile: stages and their bytes per CTA
    static constexpr int B_ROWS = BN / CG;
    static constexpr int SFA_OFF = A_BYTES + B_ROWS * BKB;
    static constexpr int SFB_OFF = SFA_OFF + 2 * SF_TILE;
    static constexpr int BYTES = SFB_OFF + 4 * SF_TILE;            // a multiple of 1024
    static constexpr int STAGES = CG == 1 ? 3 : 5;
    static constexpr int SMEM = 1024 + STAGES * BYTES + STAGING_BYTES + CTRL_BYTES;
};
static_assert(Ring<1>::BYTES % 1024 == 0 && Ring<2>::BYTES % 1024 == 0, "128B swizzle atoms");
static_assert(Ring<1>::SMEM <= 232448 && Ring<2>::SMEM <= 232448, "227 KB of dynamic shared memory");

struct Mx4Params {
    CUtensorMap tmA, tmB0, tmB1, tmSA, tmSB0, tmSB1, tmO;
    const int32_t* offsets;
    int* status;
    int64_t rows;
    int E, K, N, n_blocks, act, f32;
};

__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
    uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)1 << 16;                // leading offset: not used with one swizzle atom along K
    d |= (uint64_t)(1024 >> 4) << 32;      // 8-row groups
    d |= (uint64_t)1 << 46;                // descriptor version
    d |= (uint64_t)2 << 61;                // 128-byte swizzle
    return d;
}
__device__ __forceinline__ uint64_t desc_scales(uint32_t saddr) {   // 32 x 16 bytes, no swizzle
    uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(128 >> 4) << 32;       // 8 rows of 16 bytes
    d |= (uint64_t)1 << 46;
    return d;
}
// kind::mxf4: e2m1 x e2m1, scales of 8 exponent bits for 32 elements; `half` picks the
// lower or upper two bytes of a scale word
__device__ __forceinline__ uint32_t idesc_mx4(int M, int N, int half) {
    return ((uint32_t)(2 * half) << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
           ((uint32_t)(M >> 7) << 27) | ((uint32_t)(2 * half) << 29);
}
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

template <int CG>
__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate));
    else
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate));
}
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t sdesc) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
template <int CG>
__device__ __forceinline__ void commit_all(uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)0x3)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void commit_local(uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
}
template <int CG>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
    return CG == 1 ? mbar_wait(bar, parity, abort_flag, status) : mbar_wait_cl(bar, parity, abort_flag, status);
}
template <int CG>
__device__ __forceinline__ void drain_bar(uint32_t bar, uint32_t parity) {
    if constexpr (CG == 1) mbar_drain(bar, parity);
    else mbar_drain_cl(bar, parity);
}

__device__ __forceinline__ float silu_quick(float z) { return __fdividef(z, 1.0f + __expf(-z)); }

// A tile is CG * 128 rows x BN accumulator columns; tiles run over experts, then
// groups of RASTER_ROWS rows, columns, rows.
struct Mx4Tile { int e, m0, nb, valid; };   // valid: 128-row blocks of the segment from m0 on
template <int CG>
__device__ __forceinline__ Mx4Tile decode(const int* offs, const int* prefix, int E, int n_blocks, int tix) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= tix) lo = mid; else hi = mid - 1;
    }
    const int local = tix - prefix[lo];
    const int mb = (offs[lo + 1] - offs[lo]) / BM, mt = (mb + CG - 1) / CG;
    constexpr int RG = RASTER_ROWS / (CG * BM);
    const int grp = local / (RG * n_blocks), first = grp * RG, gm = min(RG, mt - first);
    const int r = local - grp * RG * n_blocks;
    const int m = first + r % gm;
    return {lo, offs[lo] + m * CG * BM, r / gm, mb - m * CG};
}

template <int CG>
__global__ void __launch_bounds__(NTHREADS, 1) mx4_grouped_kernel(const __grid_constant__ Mx4Params P) {
    using R = Ring<CG>;
    constexpr int S = R::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* ctrl = base + S * R::BYTES + STAGING_BYTES;
    uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);
    uint64_t* empty = full + 8;
    uint64_t* tfull = empty + 8;
    uint64_t* tempty = tfull + 1;
    uint64_t* drain = tempty + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* offs = reinterpret_cast<int*>(tmem_slot + 2);   // [E + 1]
    int* prefix = offs + 66;                             // [E + 1]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = CG == 1 ? 0u : cluster_rank();
    const bool leader = rank == 0;
    const int unit = (int)blockIdx.x / CG, nunits = (int)gridDim.x / CG;
    const bool dual = P.act == MOE_MX4_ACT_SWIGLU;

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(tfull), 1);
        mbar_init(smem_u32(tempty), CG * NUM_EPI_WARPS);
        mbar_init(smem_u32(drain), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if constexpr (CG == 2) cluster_sync_all();
    pdl_wait();
    pdl_trigger();
    if (tid < P.E + 1) offs[tid] = P.offsets[tid];
    if (warp == 1) {
        if constexpr (CG == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                         "r"(TMEM_COLS));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                         "r"(TMEM_COLS));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0) {
        // segments start at multiples of 128 rows and lie in 0..rows: no tile's box
        // has a negative coordinate; others are recorded and nothing is computed
        bool ok = offs[0] >= 0 && offs[P.E] <= P.rows;
        for (int e = 0; e <= P.E; ++e) ok = ok && offs[e] % BM == 0 && (e == 0 || offs[e] >= offs[e - 1]);
        if (!ok) set_status(P.status, MOE_ERR_DEVICE_BOUNDS);
        int acc = 0;
        for (int e = 0; e < P.E; ++e) {
            prefix[e] = acc;
            if (ok) acc += ((offs[e + 1] - offs[e]) / BM + CG - 1) / CG * P.n_blocks;
        }
        prefix[P.E] = acc;
        if (timeout_pending(P.status)) *abort_flag = 1;
    }
    __syncthreads();
    const uint32_t tmem = *tmem_slot;
    const int total = prefix[P.E];
    const uint32_t smem0 = smem_u32(base);
    const bool live = *abort_flag == 0;
    const int nk = (P.K / 2 + BKB - 1) / BKB;            // stages of a tile

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------ TMA producer (each CTA)
        const CUtensorMap* maps[7] = {&P.tmA, &P.tmB0, &P.tmSA, &P.tmSB0, &P.tmO, &P.tmB1, &P.tmSB1};
        for (int i = 0; i < (dual ? 7 : 5); ++i)
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(maps[i])) : "memory");
        int it = 0;
        bool ok = live;
        for (int tix = unit; ok && tix < total; tix += nunits) {
            const Mx4Tile t = decode<CG>(offs, prefix, P.E, P.n_blocks, tix);
            const int am = t.m0 + (int)rank * BM;
            for (int kb = 0; kb < nk; ++kb, ++it) {
                const int s = it % S;
                if (!wait_bar<1>(smem_u32(&empty[s]), ((uint32_t)(it / S) & 1u) ^ 1u, abort_flag, P.status)) {
                    ok = false;
                    break;
                }
                const uint32_t st = smem0 + s * R::BYTES;
                const uint32_t bar = CG == 1 ? smem_u32(&full[s]) : mapa_shared(smem_u32(&full[s]), 0);
                if (leader) mbar_expect_tx(smem_u32(&full[s]), CG * R::BYTES);   // every byte of a stage
                auto ld = [&](const CUtensorMap* m, uint32_t dst, int c0, int c1, int c2) {
                    if constexpr (CG == 1) tma_load3(m, dst, bar, c0, c1, c2);
                    else tma_load3_pair(m, dst, bar, c0, c1, c2);
                };
                ld(&P.tmA, st, kb * BKB, am, 0);
                ld(&P.tmSA, st + R::SFA_OFF, 0, kb * 2, am / BM);
                // 128 rows of W at a time: box rows of the weight maps
                if (dual) {
                    if (CG == 1 || rank == 0) ld(&P.tmB0, st + A_BYTES, kb * BKB, t.nb * 128, t.e);
                    if (CG == 1 || rank == 1)
                        ld(&P.tmB1, st + A_BYTES + (CG == 1 ? 128 * BKB : 0), kb * BKB, t.nb * 128, t.e);
                    const int nt = (P.N + 127) / 128;
                    ld(&P.tmSB0, st + R::SFB_OFF, 0, kb * 2, t.e * nt + t.nb);
                    ld(&P.tmSB1, st + R::SFB_OFF + 2 * SF_TILE, 0, kb * 2, t.e * nt + t.nb);
                } else {
                    for (int h = 0; h < 2 / CG; ++h)
                        ld(&P.tmB0, st + A_BYTES + h * 128 * BKB, kb * BKB,
                           t.nb * BN + (CG == 1 ? h : (int)rank) * 128, t.e);
                    const int nt = (P.N + 127) / 128;
                    for (int h = 0; h < 2; ++h)
                        ld(&P.tmSB0, st + R::SFB_OFF + h * 2 * SF_TILE, 0, kb * 2, t.e * nt + t.nb * 2 + h);
                }
            }
        }
        if (leader)
            for (int i = max(0, it - S); i < it; ++i) drain_bar<CG>(smem_u32(&full[i % S]), (uint32_t)(i / S) & 1u);
    } else if (warp == 1 && lane == 0 && leader) {
        // ------------------------------------------------ MMA issuer
        int it = 0, tcount = 0;
        bool ok = live;
        const uint32_t id[2] = {idesc_mx4(BM * CG, BN, 0), idesc_mx4(BM * CG, BN, 1)};
        for (int tix = unit; ok && tix < total; tix += nunits, ++tcount) {
            // the previous tile's epilogue is past the columns that both accumulators hold
            if (!wait_bar<CG>(smem_u32(tempty), ((uint32_t)tcount & 1u) ^ 1u, abort_flag, P.status)) break;
            tc_fence_after();
            const uint32_t dt = tmem + (tcount & 1 ? ACC1 : 0);
            uint32_t accum = 0;
            for (int kb = 0; kb < nk; ++kb, ++it) {
                const int s = it % S;
                if (!wait_bar<CG>(smem_u32(&full[s]), (uint32_t)(it / S) & 1u, abort_flag, P.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t st = smem0 + s * R::BYTES;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    copy_scales<CG>(tmem + SFA_COL + k * 4, desc_scales(st + R::SFA_OFF + k * SF_TILE));
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        copy_scales<CG>(tmem + SFB_COL + k * 8 + h * 4,
                                        desc_scales(st + R::SFB_OFF + (h * 2 + k) * SF_TILE));
                }
                const int steps = min(4, (P.K - kb * 256 + 63) / 64);   // past K the codes are 0
                for (int ks = 0; ks < steps; ++ks) {
                    mma_mx4<CG>(dt, desc_sw128(st + ks * 32), desc_sw128(st + A_BYTES + ks * 32), id[ks & 1],
                                tmem + SFA_COL + (ks >> 1) * 4, tmem + SFB_COL + (ks >> 1) * 8, accum);
                    accum = 1;
                }
                commit_all<CG>(smem_u32(&empty[s]));
            }
            if (!ok) break;
            commit_all<CG>(smem_u32(tfull));
        }
        commit_local<CG>(smem_u32(drain));
        drain_bar<CG>(smem_u32(drain), 0);
    } else if (warp >= 2) {
        // ------------------------------------------------ epilogue (each CTA, its 128 rows)
        const int qd = warp & 3, half = (warp - 2) / 4;
        const uint32_t bar_te = CG == 1 ? smem_u32(tempty) : mapa_shared(smem_u32(tempty), 0);
        uint8_t* stg = base + S * R::BYTES + (warp - 2) * 4096;
        int nst = 0;
        // a 32-row x 64-byte box (64-byte swizzle): 32 bf16 or 16 fp32 columns
        auto put = [&](const uint4 (&w)[4], int col, int row) {
            uint8_t* buf = stg + (nst & 1) * 2048;
            if (nst >= 2) {
                if (lane == 0) bulk_wait_read<1>();
                __syncwarp();
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4*>(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = w[j];
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store3(&P.tmO, smem_u32(buf), col, row, 0);
                bulk_commit();
            }
            ++nst;
        };
        const int cpw = dual ? 2 : 4;                   // 32-column chunks of this warp
        int tcount = 0;
        for (int tix = unit; tix < total; tix += nunits, ++tcount) {
            const Mx4Tile t = decode<CG>(offs, prefix, P.E, P.n_blocks, tix);
            const int buf = tcount & 1;
            const bool valid = (int)rank < t.valid;
            const int row = t.m0 + (int)rank * BM + qd * 32;
            const int col0 = t.nb * (dual ? 128 : BN);
            const bool got = __all_sync(0xffffffffu, wait_bar<CG>(smem_u32(tfull), (uint32_t)tcount & 1u, abort_flag, P.status));
            if (!got) break;
            tc_fence_after();
            const uint32_t ta = tmem + (buf ? ACC1 : 0) + ((uint32_t)(qd * 32) << 16);
            // columns 224-255 of tensor memory are the first accumulator's last and the
            // second's first: their warps drain them first
            const bool owner = buf ? half == 0 : half == 1;
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 1) mbar_arrive(bar_te);
                    else mbar_arrive_remote(bar_te);
                }
            };
            if (!owner) release();
            for (int i = 0; i < cpw; ++i) {
                const int c = half * cpw + (owner && !buf ? (i + cpw - 1) % cpw : i);
                float v[32];
                tmem_ld32(ta + c * 32, v);
                if (dual) {
                    float u[32];
                    tmem_ld32(ta + 128 + c * 32, u);
                    tmem_wait_ld();
                    if (owner && i == 0) release();
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = (P.f32 ? silu_f(v[j]) : silu_quick(v[j])) * u[j];
                } else {
                    tmem_wait_ld();
                    if (owner && i == 0) release();
                    if (P.act == MOE_MX4_ACT_SILU)
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = P.f32 ? silu_f(v[j]) : silu_quick(v[j]);
                }
                const int col = col0 + c * 32;
                if (!valid || col >= P.N) continue;
                if (P.f32) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (col + h * 16 >= P.N) continue;
                        uint4 w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = make_uint4(__float_as_uint(v[h * 16 + 4 * j]), __float_as_uint(v[h * 16 + 4 * j + 1]),
                                              __float_as_uint(v[h * 16 + 4 * j + 2]), __float_as_uint(v[h * 16 + 4 * j + 3]));
                        put(w, col + h * 16, row);
                    }
                } else {
                    uint4 w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t p[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            __nv_bfloat162 b2 = __floats2bfloat162_rn(v[8 * j + 2 * k], v[8 * j + 2 * k + 1]);
                            p[k] = *reinterpret_cast<uint32_t*>(&b2);
                        }
                        w[j] = make_uint4(p[0], p[1], p[2], p[3]);
                    }
                    put(w, col, row);
                }
            }
        }
        if (lane == 0) bulk_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (CG == 1)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS));
        else
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS));
    }
}

// ---------------------------------------------------------------- host
#define MX4_TRY(x)                   \
    do {                             \
        int _r = (x);                \
        if (_r != MOE_OK) return _r; \
    } while (0)

// codes [sets, rows, K / 2]: boxes of 128 bytes x 128 rows
int codes_map(CUtensorMap* m, const void* p, int64_t rows, int sets, int K) {
    const uint64_t dims[3] = {(uint64_t)K / 2, (uint64_t)rows, (uint64_t)sets};
    const uint64_t st[2] = {(uint64_t)K / 2, (uint64_t)K / 2 * rows};
    const uint32_t box[3] = {BKB, BM, 1};
    return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, 3, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
// scale tiles [row tiles, K tiles, 128 words]: boxes of two K tiles
int scales_map(CUtensorMap* m, const void* p, int64_t row_tiles, int K) {
    const uint64_t kt = ((uint64_t)K + 127) / 128;
    const uint64_t dims[3] = {SF_TILE / 4, kt, (uint64_t)row_tiles};
    const uint64_t st[2] = {SF_TILE, SF_TILE * kt};
    const uint32_t box[3] = {SF_TILE / 4, 2, 1};
    return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, p, 3, dims, st, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <int CG>
int launch_mx4(const moe_mx4_product_config& c, const Mx4Params& P, cudaStream_t st) {
    static bool attr_done[64] = {};
    if (const int r = smem_attr_once(mx4_grouped_kernel<CG>, Ring<CG>::SMEM, attr_done)) return r;
    const int64_t mt = (c.rows / BM + CG - 1) / CG + (CG - 1) * c.E;   // a segment may round up
    const int64_t units = std::max<int64_t>(1, std::min<int64_t>(mt * P.n_blocks, num_sms() / CG));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(CG * units));
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = Ring<CG>::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 2 : 1;
    void* args[] = {const_cast<Mx4Params*>(&P)};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(mx4_grouped_kernel<CG>), args);
    note_launch();
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

}  // namespace

int launch_mx4_product(const moe_mx4_product_config& c, const void* xq, const void* xs, const int32_t* offsets,
                       const void* wq, const void* ws, const void* gq, const void* gs, void* out,
                       cudaStream_t st) {
    Mx4Params P;
    memset(&P, 0, sizeof(P));
    const bool dual = c.act == MOE_MX4_ACT_SWIGLU;
    const int64_t nt = (c.N + 127) / 128;
    MX4_TRY(codes_map(&P.tmA, xq, c.rows, 1, c.K));
    MX4_TRY(scales_map(&P.tmSA, xs, (c.rows + 127) / 128, c.K));
    // the accumulator's first half is the gate's for SwiGLU
    MX4_TRY(codes_map(&P.tmB0, dual ? gq : wq, c.N, c.E, c.K));
    MX4_TRY(scales_map(&P.tmSB0, dual ? gs : ws, nt * c.E, c.K));
    if (dual) {
        MX4_TRY(codes_map(&P.tmB1, wq, c.N, c.E, c.K));
        MX4_TRY(scales_map(&P.tmSB1, ws, nt * c.E, c.K));
    }
    const bool f32 = c.out_dtype == MOE_DTYPE_F32;
    const uint64_t es = f32 ? 4 : 2;
    const uint64_t dims[3] = {(uint64_t)c.N, (uint64_t)c.rows, 1};
    const uint64_t strides[2] = {c.N * es, c.N * es * c.rows};
    const uint32_t box[3] = {(uint32_t)(64 / es), 32, 1};
    MX4_TRY(encode_map(&P.tmO, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, out, 3,
                       dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B));
    P.offsets = offsets;
    P.status = device_status_ptr();
    P.rows = c.rows;
    P.E = c.E; P.K = c.K; P.N = c.N; P.act = c.act; P.f32 = f32;
    P.n_blocks = dual ? (c.N + 127) / 128 : (c.N + BN - 1) / BN;
    return launch_mx4<1>(c, P, st);
}

}  // namespace moe
