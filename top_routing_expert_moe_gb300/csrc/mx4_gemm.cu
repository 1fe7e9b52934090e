// mx4_gemm.cu -- grouped product of the experts with both operands in
// microscaled 4-bit numbers, on the block-scaled tensor cores (sm_103a).
//
//   u[r, n] = sum_i x[r, i] W_e[n, i],  x and W e2m1 codes times 2^(s - 127) per
//   32 elements along i;  out = u, silu(u), or silu(g) u with g from a second W.
//
// A persistent kernel like the bf16 grouped GEMM (gemm_tc.cu).  A CTA pair takes
// 256 rows x 256 accumulator columns (a single CTA 128 x 128 where segments are
// short), warp-specialised:
//   warp 0       TMA producer: per stage of 256 elements, 128 bytes a row, this CTA's
//                128 rows of x and its 128 rows of W (for SwiGLU the even CTA's are
//                the gate's, the odd CTA's the up matrix's).
//   warp 1       the even CTA's issues the block-scaled MMAs, 64 elements each.
//   warps 2-9    epilogue: activation, rounding, TMA stores of 32-row x 128-byte boxes.
//   warps 10-13  scale tiles: to shared memory by cp.async, then to tensor memory.
//
// What it costs (8192 x 4096 x 8192, us): MMAs alone 74; with the epilogue's stores,
// the loads and the scales 95.  Before the issuing warp stayed together (one thread
// of a divergent branch moved every operand to a uniform register first) the same
// stages took 131: at 4 bits a stage's MMAs last 512 cycles, so the issuing thread's
// instructions and every wait on its way count.  Scales by tcgen05.cp from the stage
// (six of 512 bytes) cost 1 % more, but the three TMA loads that bring them cost 12 %:
// two loads a stage is what the producer can issue in the time of its MMAs.
//
// Tensor memory: two accumulators of 256 columns that overlap in 128, and buffers of
// 24 columns of scales.  A tile's epilogue takes the overlapping columns to registers
// first; the next tile's MMAs start as soon as it has.
//
// Codes are K-major with 128-byte swizzle, so a step of 64 elements (32 bytes)
// advances the descriptor as a bf16 step of 16 does.  A scale tile (128 rows x 4
// blocks, 512 bytes) holds row r's four bytes as word r / 32 of the 16 bytes of lane
// r % 32, which is how tensor memory holds them, once in each lane quarter.
#include <cuda.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "tma.cuh"

namespace moe {

namespace {

constexpr int BM = 128;                    // rows per CTA
constexpr int BKB = 128;                   // bytes of a row per stage: 256 elements
constexpr int A_BYTES = BM * BKB;
constexpr int SF_TILE = 512;               // scale bytes of 128 rows x 128 elements
constexpr int SF_SLOT = 6 * SF_TILE;       // a stage's: two tiles of x, four of W
constexpr int SF_AHEAD = 4, SF_SLOTS = SF_AHEAD + 1;
constexpr int NUM_EPI_WARPS = 8;
constexpr int NUM_SF_WARPS = 4;           // one per lane quarter of tensor memory
constexpr int NTHREADS = 64 + 32 * (NUM_EPI_WARPS + NUM_SF_WARPS);
constexpr int STAGING_BYTES = NUM_EPI_WARPS * 4096;
constexpr int CTRL_BYTES = 1024;
constexpr int TMEM_COLS = 512;
constexpr int ACC1 = 128;                  // second accumulator's first column (a pair's overlap in 128-255)
constexpr int SF_COL = 384, SF_COLS = 24;  // buffers of 24 columns: 8 of x's scales, 16 of W's
constexpr int RASTER_ROWS = 4096;          // rows of x that pass over an expert's weights together

template <int CG> struct Ring {            // CG CTAs a tile: stages and their bytes per CTA
    static constexpr int BN = 128 * CG;    // accumulator columns (SwiGLU: half gate, half up)
    static constexpr int BYTES = A_BYTES + 128 * BKB;
    static constexpr int STAGES = 5;
    static constexpr int SF_BUFS = STAGES;               // see the scale warps
    static constexpr int SMEM = 1024 + STAGES * BYTES + STAGING_BYTES + SF_SLOTS * SF_SLOT + CTRL_BYTES;
};
static_assert(Ring<1>::BYTES % 1024 == 0 && Ring<2>::BYTES % 1024 == 0, "128B swizzle atoms");
static_assert(Ring<1>::SMEM <= 232448 && Ring<2>::SMEM <= 232448, "227 KB of dynamic shared memory");

struct Mx4Params {
    CUtensorMap tmA, tmB0, tmB1, tmO;
    const uint4 *sa, *sb0, *sb1;           // scale tiles of x, and of the accumulator's two halves' W
    const int32_t* offsets;
    int* status;
    int64_t rows;
    int E, K, N, n_blocks, act;
    int ways;                              // CTAs of a cluster that may share a tile's K (single CTAs only)
    int max_tiles;                         // their grid: tiles of the rows that are not padding
};

__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
    uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)1 << 16;                // leading offset: not used with one swizzle atom along K
    d |= (uint64_t)(1024 >> 4) << 32;      // 8-row groups
    d |= (uint64_t)1 << 46;                // descriptor version
    d |= (uint64_t)2 << 61;                // 128-byte swizzle
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

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
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
__device__ __forceinline__ void mma_mx4(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n.reg .pred p;\n.reg .b64 da, db;\nsetp.ne.b32 p, %7, 0;\nmov.b64 da, {%1, %3};\nmov.b64 db, {%2, %3};\n"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %4, [%5], [%6], p;\n}" ::"r"(d),
            "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate));
    else
        asm volatile(
            "{\n.reg .pred p;\n.reg .b64 da, db;\nsetp.ne.b32 p, %7, 0;\nmov.b64 da, {%1, %3};\nmov.b64 db, {%2, %3};\n"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %4, [%5], [%6], p;\n}" ::"r"(d),
            "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate));
}
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p;
}
// words of this warp's 32 lanes, from column taddr on
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint4 (&v)[2]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0].x),
                 "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z), "r"(v[1].w)
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint4 (&v)[4]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0].x), "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z), "r"(v[1].w),
        "r"(v[2].x), "r"(v[2].y), "r"(v[2].z), "r"(v[2].w), "r"(v[3].x), "r"(v[3].y), "r"(v[3].z), "r"(v[3].w)
        : "memory");
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
// Bounded wait of one thread (CG = 2: acquire at cluster scope), as mbar_wait, but the clock and the
// flags are looked at every 1024 tries only: a stage of these kernels lasts no longer
// than one look at them.
template <int CG>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
    unsigned long long t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (CG == 1 ? mbar_try(bar, parity) : mbar_try_cl(bar, parity)) return true;
        if ((it & 1023) == 0) {
            if (*abort_flag) return false;
            const unsigned long long now = gtimer();
            if (t0 == 0) t0 = now;
            const bool late = now - t0 > WAIT_NS;
            if (late) set_status(status, MOE_ERR_TIMEOUT);
            if (late || timeout_pending(status)) {
                *abort_flag = 1;
                return false;
            }
        }
    }
}
// The lanes of a warp that all look may differ when a wait gives up (one sees the phase,
// another the abort flag), and a warp that parted there would not meet again: they go on
// together or not at all.
__device__ __forceinline__ bool agreed(bool got) { return __all_sync(0xffffffffu, got); }
// a whole warp waits: one lane looks
template <int CG>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
    int got = 0;
    if ((threadIdx.x & 31) == 0) got = wait_bar<CG>(bar, parity, abort_flag, status);
    return __shfl_sync(0xffffffffu, got, 0) != 0;
}
// Arrival on the pair's even CTA.  What it announces (tensor memory written or read)
// is ordered by the tcgen05 waits and fences around it, so it carries no release of
// ordinary memory to the cluster, which costs more than a stage's MMAs.
__device__ __forceinline__ void arrive_pair(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
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

template <int CG, bool F32, bool DUAL>
__global__ void __launch_bounds__(NTHREADS, 1) mx4_grouped_kernel(const __grid_constant__ Mx4Params P) {
    using R = Ring<CG>;
    constexpr int S = R::STAGES, SB = R::SF_BUFS, BN = R::BN;
    constexpr int OUT = DUAL ? BN / 2 : BN;              // output columns of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sf_smem = base + S * R::BYTES + STAGING_BYTES;
    uint8_t* ctrl = sf_smem + SF_SLOTS * SF_SLOT;
    uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);
    uint64_t* empty = full + 8;
    uint64_t* tfull = empty + 8;
    uint64_t* tempty = tfull + 1;
    uint64_t* sfull = tempty + 1;          // [SF_BUFS]
    uint64_t* drain = sfull + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* offs = reinterpret_cast<int*>(tmem_slot + 2);   // [E + 1]
    int* prefix = offs + 66;                             // [E + 1]

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t rank = CG == 1 ? 0u : cluster_rank();   // within the pair
    const bool leader = rank == 0;
    constexpr bool dual = DUAL;            // SwiGLU: gate and up

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(tfull), 1);
        mbar_init(smem_u32(tempty), CG * NUM_EPI_WARPS);
        for (int b = 0; b < R::SF_BUFS; ++b) mbar_init(smem_u32(&sfull[b]), CG * NUM_SF_WARPS);
        mbar_init(smem_u32(drain), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        const CUtensorMap* maps[4] = {&P.tmA, &P.tmB0, &P.tmO, &P.tmB1};
        for (int i = 0; i < (dual ? 4 : 3); ++i)
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(maps[i])) : "memory");
    }
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
    if constexpr (CG == 2) cluster_sync_all();   // both CTAs' barriers exist before any cross-CTA use
    pdl_wait();
    pdl_trigger();
    if (warp == 0) {
        // Each lane two segments: their tiles, and the tiles before them.  Segments start
        // at multiples of 128 rows and lie in 0..rows, so that no tile's box has a
        // negative coordinate; others are recorded and nothing is computed.
        int lo[2], hi[2], n[2], before = 0;
        bool ok = true;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = lane + 32 * i;
            lo[i] = e < P.E ? P.offsets[e] : 0;
            hi[i] = e < P.E ? P.offsets[e + 1] : 0;
        }
        const bool pending = lane == 0 && timeout_pending(P.status);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            ok = ok && lo[i] >= 0 && hi[i] >= lo[i] && hi[i] <= P.rows && lo[i] % BM == 0 && hi[i] % BM == 0;
            n[i] = (((hi[i] - lo[i]) / BM + CG - 1) / CG) * P.n_blocks;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0) set_status(P.status, MOE_ERR_DEVICE_BOUNDS);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = lane + 32 * i;
            int sum = ok ? n[i] : 0;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            if (e < P.E) {
                offs[e] = lo[i];
                prefix[e] = before + sum - (ok ? n[i] : 0);
            }
            if (e == P.E - 1) {
                offs[P.E] = hi[i];
                prefix[P.E] = before + sum;
            }
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
        // a timeout recorded earlier on this device (not yet read by the host): skip the work
        if (pending) *abort_flag = 1;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int total = prefix[P.E];
    const uint32_t smem0 = smem_u32(base);
    const bool live = *abort_flag == 0;
    const int nk = (P.K / 2 + BKB - 1) / BKB;            // stages of a tile
    // Few tiles: the CTAs of a cluster each take a share of one tile's stages, and the
    // first adds the others' sums.  Every CTA then has one tile at most, so the ring
    // is free to hold its sums once they are formed.
    const bool split = CG == 1 && P.ways > 1 && total * P.ways <= (int)gridDim.x;
    const int share = split ? (int)cluster_rank() : 0, ways = split ? P.ways : 1;
    const int unit = (int)blockIdx.x / (CG * ways), nunits = (int)gridDim.x / (CG * ways);
    const int kb0 = nk * share / ways, kb1 = nk * (share + 1) / ways;

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------ TMA producer (each CTA)
        int it = 0;
        bool ok = live;
        for (int tix = unit; ok && tix < total; tix += nunits) {
            const Mx4Tile t = decode<CG>(offs, prefix, P.E, P.n_blocks, tix);
            const int am = t.m0 + (int)rank * BM;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
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
                // this CTA's 128 rows of W: a pair's halves are gate and up, or columns;
                // one CTA has 64 of each
                if (dual && CG == 1) {
                    ld(&P.tmB0, st + A_BYTES, kb * BKB, t.nb * OUT, t.e);
                    ld(&P.tmB1, st + A_BYTES + 64 * BKB, kb * BKB, t.nb * OUT, t.e);
                } else if (dual) {
                    ld(rank ? &P.tmB1 : &P.tmB0, st + A_BYTES, kb * BKB, t.nb * OUT, t.e);
                } else {
                    ld(&P.tmB0, st + A_BYTES, kb * BKB, t.nb * OUT + (int)rank * 128, t.e);
                }
            }
        }
        if (leader)
            for (int i = max(0, it - S); i < it; ++i) drain_bar<CG>(smem_u32(&full[i % S]), (uint32_t)(i / S) & 1u);
    } else if (warp == 1 && leader) {
        // ------------------------------------------------ MMA issuer
        // The warp stays together and elects a thread for the tcgen05 instructions: their
        // operands then live in uniform registers, and a stage's four MMAs issue in less
        // time than they take.  Descriptors differ in their low words only.
        const uint32_t elected = elect_one();
        const uint32_t a_lo = (uint32_t)desc_sw128(smem0), b_lo = (uint32_t)desc_sw128(smem0 + A_BYTES);
        const uint32_t hi = (uint32_t)(desc_sw128(0) >> 32);
        const uint32_t id0 = idesc_mx4(BM * CG, BN, 0), id1 = idesc_mx4(BM * CG, BN, 1);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const int tail = (P.K - (nk - 1) * 256 + 63) / 64;   // MMAs of a tile's last stage
        int s = 0, tcount = 0;
        uint32_t ph = 0;
        bool ok = live;
        for (int tix = unit; ok && tix < total; tix += nunits, ++tcount) {
            // the previous tile's epilogue is past the columns that both accumulators hold
            if (!agreed(wait_bar<1>(smem_u32(tempty), ((uint32_t)tcount & 1u) ^ 1u, abort_flag, P.status))) break;
            tc_fence_after();
            const uint32_t dt = tm + (tcount & 1 ? ACC1 : 0);
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = agreed(wait_bar<1>(smem_u32(&full[s]), ph, abort_flag, P.status) &&
                            wait_bar<1>(smem_u32(&sfull[s]), ph, abort_flag, P.status));
                if (!ok) break;
                tc_fence_after();
                if (elected) {
                    const uint32_t al = a_lo + s * (R::BYTES >> 4), bl = b_lo + s * (R::BYTES >> 4);
                    const uint32_t sf = tm + SF_COL + s * SF_COLS;
                    const int steps = kb + 1 == nk ? tail : 4;
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        if (ks < steps)
                            mma_mx4<CG>(dt, al + ks * 2, bl + ks * 2, hi, ks & 1 ? id1 : id0, sf + (ks >> 1) * 4,
                                        sf + 8 + (ks >> 1) * 8, kb > kb0 || ks > 0);
                    commit_all<CG>(smem_u32(&empty[s]));
                }
                __syncwarp();
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (!ok) break;
            if (elected) commit_all<CG>(smem_u32(tfull));
            __syncwarp();
        }
        if (elected) {
            commit_local<CG>(smem_u32(drain));
            drain_bar<CG>(smem_u32(drain), 0);
        }
        __syncwarp();
    } else if (warp >= 2 + NUM_EPI_WARPS) {
        // ------------------------------------------------ scales (each CTA: its rows' and all columns')
        // The four warps copy a stage's six tiles to shared memory, four stages ahead
        // (cp.async; a tile is one warp's 32 x 16 bytes), and write them to tensor
        // memory, each its lane quarter, as the MMA reads every quarter's copy.  A
        // buffer there is free once the MMAs SF_BUFS = STAGES stages back have read
        // it, which is when that stage's "empty" barrier completes.  (With more buffers
        // than stages the barrier could pass that phase and the next unseen.)
        const int w = warp - 2 - NUM_EPI_WARPS;
        const uint32_t ta = tmem + ((uint32_t)((warp & 3) * 32) << 16) + SF_COL;
        const uint32_t bar0 = CG == 1 ? smem_u32(&sfull[0]) : mapa_shared(smem_u32(&sfull[0]), 0);
        const uint32_t sf0 = smem_u32(sf_smem) + lane * 16;
        const int kt = (P.K + 127) / 128, nt = (P.N + 127) / 128, at = (int)((P.rows + BM - 1) / BM);
        const int stages = unit < total ? ((total - 1 - unit) / nunits + 1) * (kb1 - kb0) : 0;
        // this warp's tiles: w (0, 1: x's; 2, 3: the first k tile's W halves), and for the
        // first two warps the second k tile's W halves
        int f_tix = unit, f_kb = kb0, f_slot = 0;         // the next stage to copy
        const uint4 *pa = nullptr, *pb = nullptr;       // its tile's first words (k tile 0), null past the end
        uint32_t upper = 0, uppers = 0;                 // one CTA, SwiGLU: a tile is the upper or the lower 64
                                                        // rows of W's tile; a bit per slot
        auto locate = [&]() {
            if (f_tix >= total) return;
            const Mx4Tile t = decode<CG>(offs, prefix, P.E, P.n_blocks, f_tix);
            const int ra = t.m0 / BM + (int)rank;
            auto wt = [&](int h) -> const uint4* {      // half h of the accumulator's columns
                const int r = dual ? t.nb * OUT / 128 : t.nb * CG + h;
                return (dual || h < CG) && r < nt ? (dual && h ? P.sb1 : P.sb0) + ((int64_t)t.e * nt + r) * kt * 32 + lane : nullptr;
            };
            // (w == 1 and the second piece take the stage's second k tile)
            pa = w >= 2 ? wt(w - 2) : ra < at ? P.sa + (int64_t)ra * kt * 32 + lane : nullptr;
            pb = w < 2 ? wt(w) : nullptr;
            if (pa) pa += (kb0 * 2 + (w == 1)) * 32;
            if (pb) pb += (kb0 * 2 + 1) * 32;
            upper = t.nb & 1;
        };
        locate();
        const uint32_t dst_a = sf0 + w * SF_TILE, dst_b = sf0 + (4 + w) * SF_TILE;
        const bool odd = kt & 1;
        auto copy = [&]() {                             // one group a stage, empty ones past the last
            if (f_tix < total) {
                const bool second = !odd || f_kb + 1 < nk;    // the stage has a second k tile
                const bool on_a = pa && (second || w != 1), on_b = pb && second;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst_a + f_slot * SF_SLOT),
                             "l"(on_a ? pa : P.sa), "r"(on_a ? 16 : 0)
                             : "memory");
                if (w < 2)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst_b + f_slot * SF_SLOT),
                                 "l"(on_b ? pb : P.sa), "r"(on_b ? 16 : 0)
                                 : "memory");
                if (pa) pa += 64;
                if (pb) pb += 64;
                if (dual && CG == 1) uppers = (uppers & ~(1u << f_slot)) | upper << f_slot;
                f_slot = f_slot + 1 == SF_SLOTS ? 0 : f_slot + 1;
                if (++f_kb == kb1) {
                    f_kb = kb0;
                    f_tix += nunits;
                    locate();
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        for (int i = 0; i < SF_AHEAD; ++i) copy();
        int slot = 0, buf = 0;
        uint32_t ph = 1;                                // of the "empty" barrier looked at
        bool ok = live;
        for (int it = 0; it < stages; ++it) {
            asm volatile("cp.async.wait_group %0;" ::"n"(SF_AHEAD - 1) : "memory");
            asm volatile("bar.sync 1, 128;" ::: "memory");   // every warp's tiles are there
            uint4 a[2], b[4];
            const uint8_t* t = sf_smem + slot * SF_SLOT + lane * 16;
#pragma unroll
            for (int k = 0; k < 2; ++k) a[k] = *reinterpret_cast<const uint4*>(t + k * SF_TILE);
#pragma unroll
            for (int k = 0; k < 4; ++k) b[k] = *reinterpret_cast<const uint4*>(t + (2 + k) * SF_TILE);
            if (dual && CG == 1) {                      // rows 0-63: the gate's, 64-127: up's
                const bool up = uppers >> slot & 1;
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const uint4 g = b[k], u = b[k + 1];
                    b[k] = up ? make_uint4(g.z, g.w, u.z, u.w) : make_uint4(g.x, g.y, u.x, u.y);
                }
            }
            copy();      // into the slot that the previous stage's reads, before the barrier, left
            ok = ok && warp_wait<1>(smem_u32(&empty[buf]), ph, abort_flag, P.status);
            if (ok) {    // (a warp that gave up still joins the barriers above)
                tc_fence_after();
                tmem_st8(ta + buf * SF_COLS, a);
                tmem_st16(ta + buf * SF_COLS + 8, b);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 1) mbar_arrive(bar0 + buf * 8);
                    else arrive_pair(bar0 + buf * 8);
                }
            }
            slot = slot + 1 == SF_SLOTS ? 0 : slot + 1;
            if (++buf == SB) {
                buf = 0;
                ph ^= 1u;
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else if (warp >= 2) {
        // ------------------------------------------------ epilogue (each CTA, its 128 rows)
        const int qd = warp & 3, half = (warp - 2) / 4;
        const uint32_t bar_te = CG == 1 ? smem_u32(tempty) : mapa_shared(smem_u32(tempty), 0);
        uint8_t* stg = base + S * R::BYTES + (warp - 2) * 4096 + lane * 128;
        // 32 columns of this lane's row into piece `at` (16 bytes each, 128-byte swizzle)
        // of the warp's 32-row x 128-byte staging box: bf16 half of it, fp32 all
        auto stage_bf16 = [&](const float (&o)[32], int at) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t p[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    __nv_bfloat162 b2 = __floats2bfloat162_rn(o[8 * j + 2 * k], o[8 * j + 2 * k + 1]);
                    p[k] = *reinterpret_cast<uint32_t*>(&b2);
                }
                *reinterpret_cast<uint4*>(stg + (((at + j) ^ (lane & 7)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
            }
        };
        auto stage_f32 = [&](const float (&o)[32]) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<float4*>(stg + ((j ^ (lane & 7)) << 4)) =
                    make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        };
        auto box_free = [&]() {                          // the last box has been read
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
        };
        auto send = [&](int col, int row) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store3(&P.tmO, smem_u32(stg), col, row, 0);
                bulk_commit();
            }
        };
        const bool silu = P.act == MOE_MX4_ACT_SILU;
        // fp32 outputs take the exact form
        auto act = [](float z) { return F32 ? silu_f(z) : silu_quick(z); };
        // 64 neighbouring columns, in two halves of 32
        auto store = [&](const float (&o)[2][32], int col, int row, bool valid) {
            if (!valid || col >= P.N) return;
            if constexpr (F32) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (col + 32 * i >= P.N) break;
                    box_free();
                    stage_f32(o[i]);
                    send(col + 32 * i, row);
                }
            } else {
                box_free();
                stage_bf16(o[0], 0);
                stage_bf16(o[1], 4);
                send(col, row);
            }
        };
        // a cluster's sums: 64 columns of a lane quarter's rows, by lane, in pieces of 16 bytes
        const uint32_t sums = smem0 + (uint32_t)(qd * 2) * 8192 + lane * 16;
        if (split && share > 0) {
            if (unit < total && warp_wait<1>(smem_u32(tfull), 0, abort_flag, P.status)) {
                tc_fence_after();
                const uint32_t ta = tmem + ((uint32_t)(qd * 32) << 16) + half * 64;
                float v[2][32];
                tmem_ld32(ta, v[0]);
                tmem_ld32(ta + 32, v[1]);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float* x = v[i >> 3] + (i & 7) * 4;
                    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(sums + half * 8192 + i * 512), "f"(x[0]),
                                 "f"(x[1]), "f"(x[2]), "f"(x[3])
                                 : "memory");
                }
            }
            cluster_sync_all();                          // the sums are there
        }
        // adds 16 columns from 4 p on of half h's 64 of the other CTAs' sums, in order; their
        // loads are issued together, as each takes a trip to the other SM
        auto add_shares = [&](float* x, int h, int p) {
            for (int q = 1; q < ways; ++q) {
                const uint32_t from = mapa_shared(sums + h * 8192 + p * 512, (uint32_t)q);
                float f[16];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(f[4 * i]), "=f"(f[4 * i + 1]), "=f"(f[4 * i + 2]), "=f"(f[4 * i + 3])
                                 : "r"(from + i * 512));
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] += f[i];
            }
        };
        int tcount = 0;
        bool joined = false;
        for (int tix = unit; share == 0 && tix < total; tix += nunits, ++tcount) {
            const Mx4Tile t = decode<CG>(offs, prefix, P.E, P.n_blocks, tix);
            const int buf = tcount & 1;
            const bool valid = (int)rank < t.valid;
            const int row = t.m0 + (int)rank * BM + qd * 32;
            const int col0 = t.nb * OUT;
            const bool got = warp_wait<1>(smem_u32(tfull), (uint32_t)tcount & 1u, abort_flag, P.status);
            if (!got) break;
            tc_fence_after();
            if (split) {
                cluster_sync_all();                      // the others' sums are there
                joined = true;
            }
            const uint32_t ta = tmem + (buf ? ACC1 : 0) + ((uint32_t)(qd * 32) << 16);
            float v[2][32];
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 1) mbar_arrive(bar_te);
                    else arrive_pair(bar_te);
                }
            };
            if constexpr (CG == 1) {
                // 128 columns: 64 a warp, or for SwiGLU the gate's 64 and up's by one warp
                const bool work = !DUAL || half == 0;
                if (work) {
                    const uint32_t cols = ta + (DUAL ? 0 : half * 64);
                    tmem_ld32(cols, v[0]);
                    tmem_ld32(cols + 32, v[1]);
                    tmem_wait_ld();
                    if (split)
#pragma unroll
                        for (int i = 0; i < 4; ++i) add_shares(v[i >> 1] + (i & 1) * 16, DUAL ? 0 : half, 4 * i);
                    if constexpr (DUAL) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float o[16], (&w)[32] = v[i >> 1];
                            const int k = (i & 1) * 16;
                            tmem_ld16(cols + 64 + 16 * i, o);
                            tmem_wait_ld();
                            if (split) add_shares(o, 1, 4 * i);
#pragma unroll
                            for (int j = 0; j < 16; ++j) w[k + j] = act(w[k + j]) * o[j];
                        }
                    } else if (silu) {
#pragma unroll
                        for (int i = 0; i < 64; ++i) v[i >> 5][i & 31] = act(v[i >> 5][i & 31]);
                    }
                }
                release();
                if (work) store(v, col0 + (DUAL ? 0 : half * 64), row, valid);
                continue;
            }
            // A pair.  Columns 128-255 of tensor memory belong to both accumulators (the
            // first's upper half, the second's lower): each warp takes its 64 of them to
            // registers first, and releases them to the next tile's MMAs.
            const int c = half * 64;
            const uint32_t shared_cols = ta + (buf ? 0 : 128) + c, own_cols = ta + (buf ? 128 : 0) + c;
            tmem_ld32(shared_cols, v[0]);
            tmem_ld32(shared_cols + 32, v[1]);
            tmem_wait_ld();
            release();
            if constexpr (DUAL) {                       // gate: columns 0-127, up: 128-255
#pragma unroll
                for (int i = 0; i < 4; ++i) {           // 16 columns: registers are short
                    float o[16], (&w)[32] = v[i >> 1];
                    const int k = (i & 1) * 16;
                    tmem_ld16(own_cols + 16 * i, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) w[k + j] = buf ? act(w[k + j]) * o[j] : act(o[j]) * w[k + j];
                }
                store(v, col0 + c, row, valid);
            } else {
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    if (h) {
                        tmem_ld32(own_cols, v[0]);
                        tmem_ld32(own_cols + 32, v[1]);
                        tmem_wait_ld();
                    }
                    if (silu)
#pragma unroll
                        for (int i = 0; i < 64; ++i) v[i >> 5][i & 31] = act(v[i >> 5][i & 31]);
                    store(v, col0 + ((buf == 0) == (h == 0) ? 128 : 0) + c, row, valid);
                }
            }
        }
        if (split && share == 0 && !joined) cluster_sync_all();   // (no tile, or given up)
        if (lane == 0) bulk_wait_all();
    }
    // a cluster that shares a tile meets twice, every warp of it: when the sums are
    // there (the epilogue's warps did so above), and when they have been read
    if (split) {
        __syncwarp();
        if (warp < 2 || warp >= 2 + NUM_EPI_WARPS) cluster_sync_all();
        cluster_sync_all();
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

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}
// 3-D map with 128-byte swizzle: dims[0] contiguous, strides[i] the byte stride of dims[i + 1]
int encode_map(CUtensorMap* m, CUtensorMapDataType type, const void* ptr, const uint64_t (&dims)[3],
               const uint64_t (&strides)[2], const uint32_t (&box)[3]) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return MOE_ERR_CUDA;
    const cuuint64_t d[3] = {dims[0], dims[1], dims[2]}, st[2] = {strides[0], strides[1]};
    const cuuint32_t b[3] = {box[0], box[1], box[2]}, es[3] = {1, 1, 1};
    return fn(m, type, 3, const_cast<void*>(ptr), d, st, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? MOE_OK
               : MOE_ERR_CUDA;
}

// codes [sets, rows, K / 2]: boxes of 128 bytes x `box_rows` rows
int codes_map(CUtensorMap* m, const void* p, int64_t rows, int sets, int K, int box_rows) {
    const uint64_t dims[3] = {(uint64_t)K / 2, (uint64_t)rows, (uint64_t)sets};
    const uint64_t st[2] = {(uint64_t)K / 2, (uint64_t)K / 2 * rows};
    const uint32_t box[3] = {BKB, (uint32_t)box_rows, 1};
    return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, dims, st, box);
}
template <int CG, bool F32, bool DUAL>
int launch_mx4_t(const moe_mx4_product_config& c, const Mx4Params& P, cudaStream_t st) {
    static bool attr_done[64] = {};
    if (const int r = smem_attr_once(mx4_grouped_kernel<CG, F32, DUAL>, Ring<CG>::SMEM, attr_done)) return r;
    const int64_t mt = (c.rows / BM + CG - 1) / CG + (CG - 1) * c.E;   // a segment may round up
    const int64_t units = std::max<int64_t>(1, std::min<int64_t>(mt * P.n_blocks, num_sms() / CG));
    const int cluster = CG == 2 ? 2 : P.ways;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(P.ways > 1 ? P.ways * P.max_tiles : CG * units));
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = Ring<CG>::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    void* args[] = {const_cast<Mx4Params*>(&P)};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(mx4_grouped_kernel<CG, F32, DUAL>), args);
    note_launch();
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

template <int CG>
int launch_mx4(const moe_mx4_product_config& c, const Mx4Params& P, cudaStream_t st) {
    const bool f32 = c.out_dtype == MOE_DTYPE_F32, dual = c.act == MOE_MX4_ACT_SWIGLU;
    if (dual) return f32 ? launch_mx4_t<CG, true, true>(c, P, st) : launch_mx4_t<CG, false, true>(c, P, st);
    return f32 ? launch_mx4_t<CG, true, false>(c, P, st) : launch_mx4_t<CG, false, false>(c, P, st);
}

}  // namespace

int launch_mx4_product(const moe_mx4_product_config& c, const void* xq, const void* xs, const int32_t* offsets,
                       const void* wq, const void* ws, const void* gq, const void* gs, void* out,
                       cudaStream_t st) {
    Mx4Params P;
    memset(&P, 0, sizeof(P));
    const bool dual = c.act == MOE_MX4_ACT_SWIGLU;
    // A pair's tile is 256 rows x 256 columns: it pays where an expert has two 128-row
    // blocks or more (2048 rows of 8 experts, K = 4096, N = 14336, SwiGLU: 96 us against
    // 116); with fewer half the pair idles.  A single CTA takes 128 x 128: it serves
    // short segments, where W's bytes bound it and more, smaller tiles spread them
    // evenly.  The host knows the rows' bound only, and takes 127 of it for each expert's
    // padding, which is what moe_permute's bound holds.
    const bool pair = c.rows >= (int64_t)(256 + 127) * c.E;
    const int w_rows = dual && !pair ? 64 : 128;
    MX4_TRY(codes_map(&P.tmA, xq, c.rows, 1, c.K, BM));
    // the accumulator's first half is the gate's for SwiGLU
    MX4_TRY(codes_map(&P.tmB0, dual ? gq : wq, c.N, c.E, c.K, w_rows));
    if (dual) MX4_TRY(codes_map(&P.tmB1, wq, c.N, c.E, c.K, w_rows));
    P.sa = static_cast<const uint4*>(xs);
    P.sb0 = static_cast<const uint4*>(dual ? gs : ws);
    P.sb1 = static_cast<const uint4*>(ws);
    const bool f32 = c.out_dtype == MOE_DTYPE_F32;
    const uint64_t es = f32 ? 4 : 2;
    const uint64_t dims[3] = {(uint64_t)c.N, (uint64_t)c.rows, 1};
    const uint64_t strides[2] = {c.N * es, c.N * es * c.rows};
    const uint32_t box[3] = {(uint32_t)(128 / es), 32, 1};
    MX4_TRY(encode_map(&P.tmO, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, out, dims,
                       strides, box));
    P.offsets = offsets;
    P.status = device_status_ptr();
    P.rows = c.rows;
    P.E = c.E; P.K = c.K; P.N = c.N; P.act = c.act;
    const int cols = (pair ? 256 : 128) / (dual ? 2 : 1);       // output columns of a tile
    P.n_blocks = (c.N + cols - 1) / cols;
    // Few tiles (a token or two in decoding): two or four CTAs share a tile's K, if each
    // then has four stages or more.  256 rows of 2 experts, K = 14336, N = 4096 (64
    // tiles): 18 us against 24.  Tiles are counted from the rows that are not padding: a
    // bound without padding makes more of them than that, and the few CTAs take them in turn
    // (8064 rows of 64 experts, all real, K = 4096, N = 1024: 101 us; 16128 rows 47).
    const int64_t real = std::max<int64_t>(1, c.rows - 127 * (int64_t)c.E);
    const int64_t tiles = (real / BM + std::min<int64_t>(c.E, real)) * P.n_blocks;
    const int nk = (c.K / 2 + BKB - 1) / BKB;
    P.ways = pair ? 1 : nk >= 16 && tiles * 4 <= num_sms() ? 4 : nk >= 8 && tiles * 2 <= num_sms() ? 2 : 1;
    P.max_tiles = (int)std::min<int64_t>(tiles, num_sms());
    return pair ? launch_mx4<2>(c, P, st) : launch_mx4<1>(c, P, st);
}

}  // namespace moe
