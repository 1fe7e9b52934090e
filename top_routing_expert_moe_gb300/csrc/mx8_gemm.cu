// mx8_gemm.cu -- grouped product of the experts with both operands in microscaled 8-bit
// numbers, on the block-scaled tensor cores (sm_103a), over segments of any length.
//
//   u[r, n] = sum_i x[r, i] W_e[n, i],  x and W e4m3 codes times 2^(s - 127) per
//   32 elements along i;  out = u, silu(u), or silu(g) u with g from a second W, in
//   bf16, fp32, or 8-bit numbers again (a lane holds 32 columns of a row: a block).
//
// A persistent kernel like the 4-bit one (mx4_gemm.cu), whose roles it keeps.  A CTA pair
// takes 256 rows x 256 accumulator columns (a single CTA 128 x 128 where segments are
// short), warp-specialised:
//   warp 0       TMA producer: per stage of 128 elements, 128 bytes a row, this CTA's
//                128 rows of x and its 128 rows of W (for SwiGLU the even CTA's are
//                the gate's, the odd CTA's the up matrix's).
//   warp 1       the even CTA's issues the block-scaled MMAs, 32 elements each.
//   warps 2-9    epilogue: activation, rounding, a lane's row in pieces of 32 bytes
//                (fp32: 32-row boxes by TMA).
//   warps 10-13  scales: rows' bytes to shared memory by cp.async, then to tensor memory.
// A stage's four MMAs last 512 cycles, as the 4-bit kernel's do on twice the elements.
//
// Segments are not padded.  A tile starts at its segment's first row wherever that is (a
// TMA box may start at any row); the rows past the segment's end that it then holds are
// the next expert's, each row of a product depends on no other, and they are not stored:
// a lane of the epilogue holds columns of one row, and stores them or not, as whole sectors.
// (Boxes through shared memory take a stage's room.  Without them, and with a sixth stage:
// 1024 rows of 8 experts, 4096 -> 14336 SwiGLU in 8 bits, 156 us and 150; 2 rows of 2 of
// them 43.9 and 42.8; 8192 rows, 14336 -> 4096, 332 and 325; the largest bf16 product 2518
// and 2563.  fp32, four times the bytes, leaves by boxes: 32768 rows, 2048 -> 4096, silu,
// 211 to 236 us from one GPU to another, by lanes 262.)  For the same reason the scales of x
// are kept by rows and not in the tensor cores' 128-row tiles, which would begin at other rows
// than a segment: the scale warps form the tile (row r's four bytes as word r / 32 of lane
// r % 32) from 16 bytes a row, four stages' worth, in registers.
//
// W is kept in blocks of 128 rows x 128 elements, 16 KB each, a row block's one after the
// other along K, and its scales in the tensor cores' tiles of 512 bytes in the same order:
// a stage's scales of W are whole sectors, where 16 bytes a row for four stages left
// half of each unused (32768 rows, K = 4096, N = 14336, SwiGLU: 2460 us, by rows 2560).
//
// Few rows (decoding) are bound by W's bytes, and what they must not do is read x's few
// lines from every CTA more often than they have to: with 128 requests of every CTA for
// the scales of one row, and boxes of 128 rows for the four that there are, 2 rows of each
// of 2 experts (K = 4096, N = 14336, SwiGLU) took 145 us where they take 43.
//
// Tensor memory: two accumulators of 256 columns that overlap in 128, and buffers of 16
// columns of scales.
//
// What bounds it.  Large products: the power cap.  32768 rows of 8 experts, K = 4096,
// N = 14336, SwiGLU: about 2500 us, 3.1 PFLOP/s at 1440 MHz and 1.37 kW, where the tensor pipe
// is active 0.82 of the time; with operands of zeros, which draw less, the same launch held
// 2070 MHz and 4.0 PFLOP/s (1925 us).  There the MMAs alone took 1646 us, the loads added
// 5 %, the stores 4 %, the hand-over of the accumulator 2 %, the scales nothing.  Few rows:
// HBM, 6.9 TB/s of W (64 rows of 8 experts, the same product: 140 us).  In between the rows
// of a 256-row tile that a segment does not fill (2048 rows: 223 us).
#include <algorithm>
#include <cstring>

#include "kernels.h"
#include "mx8.cuh"
#include "mx_tc.cuh"

namespace moe {

namespace {

constexpr int BM = 128;                    // rows per CTA
constexpr int BK = 128;                    // elements, and bytes, of a row per stage
constexpr int QUAD = 4;                    // stages whose scales are 16 bytes of a row
constexpr int A_BYTES = BM * BK;
constexpr int NUM_EPI_WARPS = 8;
constexpr int NUM_SF_WARPS = 4;            // one per lane quarter of tensor memory
constexpr int NTHREADS = 64 + 32 * (NUM_EPI_WARPS + NUM_SF_WARPS);
constexpr int CTRL_BYTES = 1024;
constexpr int TMEM_COLS = 512;
constexpr int ACC1 = 128;                  // second accumulator's first column (a pair's overlap in 128-255)
constexpr int SF_COL = 384, SF_COLS = 16;  // buffers: 4 columns of x's scales, from the 8th on 4 or 8 of W's
constexpr int SF_QUAD = BM * 16;           // scale bytes of a quad: of 128 rows of x, or of a row block of W
constexpr int SF_AHEAD = 2, SF_SLOTS = SF_AHEAD + 1;     // in quads
constexpr int RASTER_ROWS = 4096;          // rows of x that pass over an expert's weights together

enum Out { OUT_F32, OUT_BF16, OUT_MX8 };

template <int CG, int OT> struct Ring {    // CG CTAs a tile: stages and their bytes per CTA
    static constexpr int BN = 128 * CG;    // accumulator columns (SwiGLU: half gate, half up)
    static constexpr int BYTES = A_BYTES + 128 * BK;
    static constexpr int STAGES = OT == OUT_F32 ? 5 : 6;
    static constexpr int STAGING = OT == OUT_F32 ? NUM_EPI_WARPS * 4096 : 0;   // fp32: a box a warp
    static constexpr int SF_BUFS = STAGES;               // see the scale warps
    static constexpr int SF_SLOT = 3 * SF_QUAD;          // x, and one or two row blocks of W
    static constexpr int SMEM = 1024 + STAGES * BYTES + STAGING + SF_SLOTS * SF_SLOT + CTRL_BYTES;
    static_assert(BYTES % 1024 == 0, "128B swizzle atoms");
    static_assert(SMEM <= 232448, "227 KB of dynamic shared memory");
    static_assert(STAGES <= 8 && SF_COL + SF_BUFS * SF_COLS <= TMEM_COLS, "barriers and tensor memory");
};

struct Mx8Params {
    CUtensorMap tmA, tmB0, tmB1, tmO;      // (tmO: fp32)
    const uint8_t *sa, *sb0, *sb1;         // scales of x (rows), and of the accumulator's two halves' W (tiles)
    uint8_t* out;
    uint8_t* out_scales;                   // OUT_MX8
    const int32_t* offsets;
    int* status;
    int64_t rows;
    int E, K, N, n_blocks, act;
    int wide;                              // rows of out are whole, aligned pieces of 32 bytes (else of 16)
    int w_blocks;                          // W's row blocks an expert
    int a_rows;                            // rows of x that a stage loads (one CTA: fewer where there are no more)
    int pitch, out_pitch;                  // bytes of a row of scales: of x, of out
    int ways;                              // CTAs of a cluster that may share a tile's K (single CTAs only)
    int max_tiles;                         // their grid
};

// kind::mxf8f6f4: e4m3 x e4m3, scales of 8 exponent bits for 32 elements; `ks` picks the
// byte of a scale word
__device__ __forceinline__ uint32_t idesc_mx8(int M, int N, int ks) {
    return ((uint32_t)ks << 4) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27) |
           ((uint32_t)ks << 29);
}
template <int CG>
__device__ __forceinline__ void mma_mx8(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n.reg .pred p;\n.reg .b64 da, db;\nsetp.ne.b32 p, %7, 0;\nmov.b64 da, {%1, %3};\nmov.b64 db, {%2, %3};\n"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], da, db, %4, [%5], [%6], p;\n}" ::"r"(d),
            "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate));
    else
        asm volatile(
            "{\n.reg .pred p;\n.reg .b64 da, db;\nsetp.ne.b32 p, %7, 0;\nmov.b64 da, {%1, %3};\nmov.b64 db, {%2, %3};\n"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], da, db, %4, [%5], [%6], p;\n}" ::"r"(d),
            "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate));
}
// words of this warp's 32 lanes, from column taddr on
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// silu for fp32 outputs, within a few units of fp32 down to the last denormals: z or z t over
// 1 + t with t = e^-|z| = 2^h (1 + l ln 2), where h + l is -|z| log2(e) in two parts, so that the
// product's rounding does not grow with z.  The divisor stays within 1..2.  (The quick form's
// error grows with z, and past -87.3 its divisor leaves the quick division's range: it gives 0
// for what is at most 1e-36.  By expf and a division the registers spilled: 32768 rows, K = 2048,
// N = 4096, silu 439 us, so 211 to 230 from one GPU to another.  The single CTA's SwiGLU spills a
// few registers in any form: its 64 values and a cluster's sums are more than 128 hold, off the
// path of W's bytes.)  Past 128 t is 0, and h and l are finite where z is not.
__device__ __forceinline__ float silu_fine(float z) {
    constexpr float L = 1.44269504f, L_LO = 1.92596303e-8f, LN2 = 0.693147181f;   // log2(e) in two parts
    const float c = fminf(fabsf(z), 128.f);
    const float h = -c * L, l = fmaf(-c, L_LO, fmaf(-c, L, -h));
    float e;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(h));
    const float t = fmaf(e, l * LN2, e);
    return __fdividef(z >= 0.f ? z : z * t, 1.f + t);
}

// A tile is CG * 128 rows x BN accumulator columns; tiles run over experts, then
// groups of RASTER_ROWS rows, columns, rows.
struct Mx8Tile { int e, m0, nb, end; };    // end: the segment's
template <int CG>
__device__ __forceinline__ Mx8Tile decode(const int* offs, const int* prefix, int E, int n_blocks, int tix) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= tix) lo = mid; else hi = mid - 1;
    }
    const int local = tix - prefix[lo];
    const int mt = (offs[lo + 1] - offs[lo] + CG * BM - 1) / (CG * BM);
    constexpr int RG = RASTER_ROWS / (CG * BM);
    const int grp = local / (RG * n_blocks), first = grp * RG, gm = min(RG, mt - first);
    const int r = local - grp * RG * n_blocks;
    const int m = first + r % gm;
    return {lo, offs[lo] + m * CG * BM, r / gm, offs[lo + 1]};
}

// W's row block that half h of the accumulator's columns multiplies by (SwiGLU: the half's
// own matrix'); past the last block that one again, for columns that are not stored
template <int CG, bool DUAL>
__device__ __forceinline__ int w_block(const Mx8Params& P, int nb, int h) {
    return min(DUAL ? (CG == 2 ? nb : nb >> 1) : nb * CG + h, P.w_blocks - 1);
}

template <int CG, int OT, bool DUAL>
__global__ void __launch_bounds__(NTHREADS, 1) mx8_grouped_kernel(const __grid_constant__ Mx8Params P) {
    using R = Ring<CG, OT>;
    constexpr int S = R::STAGES, SB = R::SF_BUFS, BN = R::BN;
    constexpr int OUT = DUAL ? BN / 2 : BN;              // output columns of a tile
    constexpr bool F32 = OT == OUT_F32;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sf_smem = base + S * R::BYTES + R::STAGING;
    uint8_t* ctrl = sf_smem + SF_SLOTS * R::SF_SLOT;
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

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(tfull), 1);
        mbar_init(smem_u32(tempty), CG * NUM_EPI_WARPS);
        for (int b = 0; b < SB; ++b) mbar_init(smem_u32(&sfull[b]), CG * NUM_SF_WARPS);
        mbar_init(smem_u32(drain), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        const CUtensorMap* maps[4] = {&P.tmA, &P.tmB0, &P.tmB1, &P.tmO};
        for (int i = 0; i < 4; ++i)
            if (i < 2 || (DUAL && i == 2) || (F32 && i == 3))
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
        // Each lane two segments: their tiles, and the tiles before them.  Segments lie in
        // 0..rows and ascend, so that no box starts at a negative row; others are recorded
        // and nothing is computed.
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
            ok = ok && lo[i] >= 0 && hi[i] >= lo[i] && hi[i] <= P.rows;
            n[i] = ((hi[i] - lo[i] + CG * BM - 1) / (CG * BM)) * P.n_blocks;
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
    const int nk = (P.K + BK - 1) / BK, nq = (nk + QUAD - 1) / QUAD;   // stages of a tile, and their quads
    // Few tiles: the CTAs of a cluster each take a share of one tile's quads, and the
    // first adds the others' sums.  Every CTA then has one tile at most, so the ring
    // is free to hold its sums once they are formed.
    const bool split = CG == 1 && P.ways > 1 && total * P.ways <= (int)gridDim.x;
    const int share = split ? (int)cluster_rank() : 0, ways = split ? P.ways : 1;
    const int unit = (int)blockIdx.x / (CG * ways), nunits = (int)gridDim.x / (CG * ways);
    const int kb0 = QUAD * (nq * share / ways), kb1 = min(nk, QUAD * (nq * (share + 1) / ways));

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------ TMA producer (each CTA)
        int it = 0;
        bool ok = live;
        for (int tix = unit; ok && tix < total; tix += nunits) {
            const Mx8Tile t = decode<CG>(offs, prefix, P.E, P.n_blocks, tix);
            const int am = t.m0 + (int)rank * BM;
            // its first row of W's 128-byte rows in memory
            const int wrow = (t.e * P.w_blocks + w_block<CG, DUAL>(P, t.nb, (int)rank)) * nk * 128 +
                             (DUAL && CG == 1 ? (t.nb & 1) * 64 : 0);
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % S;
                if (!wait_bar<1>(smem_u32(&empty[s]), ((uint32_t)(it / S) & 1u) ^ 1u, abort_flag, P.status)) {
                    ok = false;
                    break;
                }
                const uint32_t st = smem0 + s * R::BYTES;
                const uint32_t bar = CG == 1 ? smem_u32(&full[s]) : mapa_shared(smem_u32(&full[s]), 0);
                if (leader) mbar_expect_tx(smem_u32(&full[s]), CG * (R::BYTES - A_BYTES + P.a_rows * BK));   // every byte of a stage
                auto ld = [&](const CUtensorMap* m, uint32_t dst, int c0, int c1, int c2) {
                    if constexpr (CG == 1) tma_load3(m, dst, bar, c0, c1, c2);
                    else tma_load3_pair(m, dst, bar, c0, c1, c2);
                };
                ld(&P.tmA, st, kb * BK, am, 0);
                // this CTA's 128 rows of W: a pair's halves are gate and up, or columns;
                // one CTA has 64 of each
                if (DUAL && CG == 1) {
                    ld(&P.tmB0, st + A_BYTES, 0, wrow + kb * 128, 0);
                    ld(&P.tmB1, st + A_BYTES + 64 * BK, 0, wrow + kb * 128, 0);
                } else {
                    ld(DUAL && rank ? &P.tmB1 : &P.tmB0, st + A_BYTES, 0, wrow + kb * 128, 0);
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
        const uint32_t id0 = idesc_mx8(BM * CG, BN, 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const int tail = (P.K - (nk - 1) * BK) / 32;     // MMAs of a tile's last stage
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
                            mma_mx8<CG>(dt, al + ks * 2, bl + ks * 2, hi, id0 | ((uint32_t)ks << 4) | ((uint32_t)ks << 29),
                                        sf, sf + 8, kb > kb0 || ks > 0);
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
        // Thread i of the four warps copies 16 bytes of the scales of row i of x, and 16
        // bytes of the four tiles of each row block of W: a quad, four stages.  Quads are
        // copied SF_AHEAD ahead (cp.async).  Each warp then takes the words of every row to
        // registers, as the MMA reads its scales from every lane quarter, and writes a
        // stage's to its quarter of tensor memory.  A buffer there is free once the MMAs
        // SF_BUFS = STAGES stages back have read it, which is when that stage's "empty"
        // barrier completes.  (With more buffers than stages the barrier could pass that
        // phase and the next unseen.)
        constexpr int NB = CG == 2 || DUAL ? 2 : 1;      // row blocks of W
        const int i = (warp - 2 - NUM_EPI_WARPS) * 32 + lane;
        const uint32_t ta = tmem + ((uint32_t)((warp & 3) * 32) << 16) + SF_COL;
        const uint32_t bar0 = CG == 1 ? smem_u32(&sfull[0]) : mapa_shared(smem_u32(&sfull[0]), 0);
        const uint32_t dst = smem_u32(sf_smem) + i * 16;
        const int tiles = unit < total ? (total - 1 - unit) / nunits + 1 : 0;
        const int q0 = kb0 / QUAD, q1 = (kb1 + QUAD - 1) / QUAD;
        const int quads = tiles * (q1 - q0);
        int f_tix = unit, f_q = q0, f_slot = 0;          // the next quad to copy
        const uint8_t *pa = nullptr, *pb[NB] = {};       // its tile's first bytes
        uint32_t upper = 0, uppers = 0;                  // one CTA, SwiGLU: a tile is the upper or the lower 64
                                                         // rows of W's block; a bit per slot
        auto locate = [&]() {
            if (f_tix >= total) return;
            const Mx8Tile t = decode<CG>(offs, prefix, P.E, P.n_blocks, f_tix);
            // (the next segments' rows are not stored: any scale will do)
            const int row = t.m0 + (int)rank * BM + i;
            pa = row < t.end ? P.sa + (int64_t)row * P.pitch : nullptr;
#pragma unroll
            for (int h = 0; h < NB; ++h)
                pb[h] = (DUAL && h ? P.sb1 : P.sb0) +
                        ((int64_t)t.e * P.w_blocks + w_block<CG, DUAL>(P, t.nb, h)) * nk * 512 + i * 16;
            upper = t.nb & 1;
        };
        locate();
        auto copy = [&]() {                              // one group a quad, empty ones past the last
            if (f_tix < total) {
                const uint32_t d = dst + f_slot * R::SF_SLOT;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(pa ? pa + f_q * 16 : P.sa),
                             "r"(pa ? 16 : 0)
                             : "memory");
                const bool in = f_q * QUAD + i / 32 < nk;    // the row block has this tile
#pragma unroll
                for (int h = 0; h < NB; ++h)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d + (1 + h) * SF_QUAD),
                                 "l"(in ? pb[h] + f_q * SF_QUAD : P.sa), "r"(in ? 16 : 0)
                                 : "memory");
                if (DUAL && CG == 1) uppers = (uppers & ~(1u << f_slot)) | upper << f_slot;
                f_slot = f_slot + 1 == SF_SLOTS ? 0 : f_slot + 1;
                if (++f_q == q1) {
                    f_q = q0;
                    f_tix += nunits;
                    locate();
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        for (int k = 0; k < SF_AHEAD; ++k) copy();
        int slot = 0, buf = 0, kb = kb0;
        uint32_t ph = 1;                                 // of the "empty" barrier looked at
        bool ok = live;
        for (int q = 0; q < quads; ++q) {
            asm volatile("cp.async.wait_group %0;" ::"n"(SF_AHEAD - 1) : "memory");
            asm volatile("bar.sync 1, 128;" ::: "memory");   // every thread's rows are there
            uint4 a[4], b[NB][QUAD];
            const uint8_t* t = sf_smem + slot * R::SF_SLOT + lane * 16;
#pragma unroll
            for (int k = 0; k < 4; ++k) a[k] = *reinterpret_cast<const uint4*>(t + k * 512);
#pragma unroll
            for (int h = 0; h < NB; ++h)
#pragma unroll
                for (int k = 0; k < QUAD; ++k) b[h][k] = *reinterpret_cast<const uint4*>(t + (1 + h) * SF_QUAD + k * 512);
            if (DUAL && CG == 1) {                       // rows 0-63: the gate's, 64-127: up's
                const bool up = uppers >> slot & 1;
#pragma unroll
                for (int k = 0; k < QUAD; ++k) {
                    const uint4 g = b[0][k], u = b[NB - 1][k];
                    b[0][k] = up ? make_uint4(g.z, g.w, u.z, u.w) : make_uint4(g.x, g.y, u.x, u.y);
                }
            }
            copy();      // into the slot that the previous quad's reads, before the barrier, left
            const int n = min(QUAD, kb1 - kb);
            kb = kb + n == kb1 ? kb0 : kb + n;
#pragma unroll
            for (int st = 0; st < QUAD; ++st) {
                if (st >= n) break;
                ok = ok && warp_wait<1>(smem_u32(&empty[buf]), ph, abort_flag, P.status);
                if (ok) {    // (a warp that gave up still joins the barriers above)
                    auto w = [&](const uint4& v) { return st == 0 ? v.x : st == 1 ? v.y : st == 2 ? v.z : v.w; };
                    tc_fence_after();
                    tmem_st4(ta + buf * SF_COLS, w(a[0]), w(a[1]), w(a[2]), w(a[3]));
#pragma unroll
                    for (int h = 0; h < CG; ++h)
                        tmem_st4(ta + buf * SF_COLS + 8 + 4 * h, b[h][st].x, b[h][st].y, b[h][st].z, b[h][st].w);
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (CG == 1) mbar_arrive(bar0 + buf * 8);
                        else arrive_pair(bar0 + buf * 8);
                    }
                }
                if (++buf == SB) {
                    buf = 0;
                    ph ^= 1u;
                }
            }
            slot = slot + 1 == SF_SLOTS ? 0 : slot + 1;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else if (warp >= 2) {
        // ------------------------------------------------ epilogue (each CTA, its 128 rows)
        const int qd = warp & 3, half = (warp - 2) / 4;
        const uint32_t bar_te = CG == 1 ? smem_u32(tempty) : mapa_shared(smem_u32(tempty), 0);
        constexpr int ES = OT == OUT_F32 ? 4 : OT == OUT_BF16 ? 2 : 1;
        // 32 columns of this lane's row, from column col on: as many as lie before column N (N
        // is whole pieces)
        auto pieces = [&](uint8_t* dst, int col, const uint32_t (&w)[8 * ES]) {
#pragma unroll
            for (int i = 0; i < ES; ++i) {
                if (P.wide) {
                    if (col + i * (32 / ES) < P.N) store32(dst + i * 32, w + 8 * i);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (col + i * (32 / ES) + h * (16 / ES) < P.N)
                            *reinterpret_cast<uint4*>(dst + i * 32 + h * 16) =
                                make_uint4(w[8 * i + 4 * h], w[8 * i + 4 * h + 1], w[8 * i + 4 * h + 2], w[8 * i + 4 * h + 3]);
                }
            }
        };
        // fp32: 32 columns of the warp's rows as a box of 128-byte rows, 128-byte swizzle; all of
        // it by TMA, which leaves out columns past N, or the nv < 32 rows that are the segment's
        auto send_box = [&](const float (&o)[32], int col, int row, int nv) {
            uint8_t* box = base + S * R::BYTES + (warp - 2) * 4096;
            auto piece = [&](int r, int j) { return reinterpret_cast<float4*>(box + r * 128 + ((j ^ (r & 7)) << 4)); };
            if (lane == 0) bulk_wait_read<0>();          // the last box has been read
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) *piece(lane, j) = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            if (nv >= 32) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store3(&P.tmO, smem_u32(box), col, row, 0);
                    bulk_commit();
                }
                return;
            }
            __syncwarp();
            const int j = lane & 7;
            if (col + 4 * j < P.N)
                for (int r = lane >> 3; r < nv; r += 4)
                    *reinterpret_cast<float4*>(P.out + ((int64_t)(row + r) * P.N + col) * 4 + j * 16) = *piece(r, j);
            __syncwarp();
        };
        const bool silu = P.act == MOE_MX8_ACT_SILU;
        // The quick form is off by some 1e-6 of the value.  bf16 hides it; in 8 bits an element
        // near the middle of two codes takes the other one more often than by the sums' own
        // rounding (a prompt's outputs are 7.9e-5 from 64 bits, 4.2e-5 by the fine form; half a
        // step is 6e-2 of an element), where the fine form costs 8 % (32768 rows, 2048 -> 4096,
        // silu: 185 us and 201; two tokens, 4096 -> 14336 SwiGLU: 42.8 and 47.2).
        auto act = [](float z) { return F32 ? silu_fine(z) : silu_quick(z); };
        // 64 neighbouring columns of this lane's row, in two halves of 32; nv: rows of the
        // warp's 32 that are the segment's
        auto store = [&](const float (&o)[2][32], int col, int row, int nv) {
            if constexpr (F32) {
                if (nv <= 0) return;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (col + 32 * i < P.N) send_box(o[i], col + 32 * i, row, nv);
                return;
            }
            if (lane < nv && col < P.N) {
                const int64_t r = row + lane;
                uint8_t* dst = P.out + (r * P.N + col) * ES;
                uint32_t s[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t w[8 * ES];
                    if constexpr (OT == OUT_BF16) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            __nv_bfloat162 b2 = __floats2bfloat162_rn(o[i][2 * j], o[i][2 * j + 1]);
                            w[j] = *reinterpret_cast<uint32_t*>(&b2);
                        }
                    } else {                                 // a block
                        s[i] = mx8_scale_byte(amax_bits<32>(o[i]));
                        mx8_codes<32>(o[i], s[i], w);
                    }
                    pieces(dst + i * 32 * ES, col + 32 * i, w);
                }
                // (both bytes lie in the row's pitch; past the last block they stand for nothing)
                if constexpr (OT == OUT_MX8)
                    *reinterpret_cast<uint16_t*>(P.out_scales + r * P.out_pitch + col / 32) = (uint16_t)(s[0] | s[1] << 8);
            }
            __syncwarp();                                // (together again for tensor memory)
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
            const Mx8Tile t = decode<CG>(offs, prefix, P.E, P.n_blocks, tix);
            const int buf = tcount & 1;
            const int row = t.m0 + (int)rank * BM + qd * 32, nv = t.end - row;
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
                if (work) store(v, col0 + (DUAL ? 0 : half * 64), row, nv);
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
                store(v, col0 + c, row, nv);
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
                    store(v, col0 + ((buf == 0) == (h == 0) ? 128 : 0) + c, row, nv);
                }
            }
        }
        if (split && share == 0 && !joined) cluster_sync_all();   // (no tile, or given up)
        if (F32 && lane == 0) bulk_wait_all();
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
#define MX8_TRY(x)                   \
    do {                             \
        int _r = (x);                \
        if (_r != MOE_OK) return _r; \
    } while (0)

// rows of `bytes`: boxes of 128 bytes x `box_rows` rows
int codes_map(CUtensorMap* m, const void* p, int64_t rows, int bytes, int box_rows) {
    const uint64_t dims[3] = {(uint64_t)bytes, (uint64_t)rows, 1};
    const uint64_t st[2] = {(uint64_t)bytes, (uint64_t)bytes * rows};
    const uint32_t box[3] = {BK, (uint32_t)box_rows, 1};
    return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, dims, st, box);
}
template <int CG, int OT, bool DUAL>
int launch_mx8_t(const moe_mx8_product_config& c, const Mx8Params& P, cudaStream_t st) {
    static bool attr_done[64] = {};
    if (const int r = smem_attr_once(mx8_grouped_kernel<CG, OT, DUAL>, (Ring<CG, OT>::SMEM), attr_done)) return r;
    const int64_t mt = c.rows / (CG * BM) + c.E;         // a segment may round up
    const int64_t units = std::max<int64_t>(1, std::min<int64_t>(mt * P.n_blocks, num_sms() / CG));
    const int cluster = CG == 2 ? 2 : P.ways;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(P.ways > 1 ? P.ways * P.max_tiles : CG * units));
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = (Ring<CG, OT>::SMEM);
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
    void* args[] = {const_cast<Mx8Params*>(&P)};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(mx8_grouped_kernel<CG, OT, DUAL>), args);
    note_launch();
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

template <int CG, int OT>
int launch_mx8(const moe_mx8_product_config& c, const Mx8Params& P, cudaStream_t st) {
    return c.act == MOE_MX8_ACT_SWIGLU ? launch_mx8_t<CG, OT, true>(c, P, st) : launch_mx8_t<CG, OT, false>(c, P, st);
}
template <int CG>
int launch_mx8_out(const moe_mx8_product_config& c, const Mx8Params& P, cudaStream_t st) {
    switch (c.out_dtype) {
        case MOE_DTYPE_F32: return launch_mx8<CG, OUT_F32>(c, P, st);
        case MOE_DTYPE_BF16: return launch_mx8<CG, OUT_BF16>(c, P, st);
        default: return launch_mx8<CG, OUT_MX8>(c, P, st);
    }
}

}  // namespace

int launch_mx8_product(const moe_mx8_product_config& c, const void* xq, const void* xs, const int32_t* offsets,
                       const void* wq, const void* ws, const void* gq, const void* gs, void* out, void* out_scales,
                       cudaStream_t st) {
    Mx8Params P;
    memset(&P, 0, sizeof(P));
    const bool dual = c.act == MOE_MX8_ACT_SWIGLU;
    // A pair's tile is 256 rows x 256 columns, a single CTA's 128 x 128, which loads twice
    // the bytes for the same products: it serves where an expert has so few rows that W's
    // bytes are all that counts.  The host knows the experts' rows together (8 of them, us,
    // single and pair):     640 rows       768 rows       1024 rows
    //   4096 -> 14336 SwiGLU  148  153       200  154       211  156
    //   2048 -> 4096 silu      19  24         25  23         25  22
    //   14336 -> 4096          82  93        110  89        109  91
    // 8 and 64 experts part at the same place, by rows an expert (4096 -> 4096): where all have
    // as many rows single CTAs win by 10 % up to 128, pairs from 192 on (45 us and 33 for 8; 399
    // and 210 for 64); spread from none to twice the mean, pairs win from 96 on (38.2 and 31.2;
    // 252 and 208) and lose at 64 (28.6 and 30.9; 190 and 200).
    // Nor does a pair pay where the single CTAs' tiles fit the GPU at once (666 rows of 5 experts,
    // 1056 -> 1000: 8.0 and 9.1; 1024 of one, 4096 -> 1024 fp32: 12.8 and 15.3; two experts,
    // 2048 -> 4096, 96 rows each: 10.1 and 11.1).  In two turns they lose (600 of one, 4096 ->
    // 2048 SwiGLU: 26.2 and 16.2).
    const int64_t single = (c.rows / BM + c.E) * ((c.N + (dual ? 63 : 127)) / (dual ? 64 : 128));
    const bool pair = c.rows >= (int64_t)96 * c.E && single > num_sms();
    const int w_rows = dual && !pair ? 64 : 128;
    // (rows of x behind the last: what is left in shared memory serves as well)
    P.a_rows = pair ? BM : (int)std::min<int64_t>(BM, (c.rows + 7) / 8 * 8);
    MX8_TRY(codes_map(&P.tmA, xq, c.rows, c.K, P.a_rows));
    // the accumulator's first half is the gate's for SwiGLU
    P.w_blocks = (c.N + 127) / 128;
    const int64_t w_lines = (int64_t)c.E * P.w_blocks * ((c.K + BK - 1) / BK) * 128;
    MX8_TRY(codes_map(&P.tmB0, dual ? gq : wq, w_lines, BK, w_rows));
    if (dual) MX8_TRY(codes_map(&P.tmB1, wq, w_lines, BK, w_rows));
    P.sa = static_cast<const uint8_t*>(xs);
    P.sb0 = static_cast<const uint8_t*>(dual ? gs : ws);
    P.sb1 = static_cast<const uint8_t*>(ws);
    const bool f32 = c.out_dtype == MOE_DTYPE_F32, mx8 = c.out_dtype == MOE_DTYPE_MX8;
    const int64_t row_bytes = (int64_t)c.N * (f32 ? 4 : mx8 ? 1 : 2);
    if (f32) {
        const uint64_t dims[3] = {(uint64_t)c.N, (uint64_t)c.rows, 1};
        const uint64_t strides[2] = {(uint64_t)row_bytes, (uint64_t)row_bytes * c.rows};
        const uint32_t box[3] = {32, 32, 1};
        MX8_TRY(encode_map(&P.tmO, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, out, dims, strides, box));
    }
    P.wide = (reinterpret_cast<uintptr_t>(out) | (uintptr_t)row_bytes) % 32 == 0;
    P.out = static_cast<uint8_t*>(out);
    P.out_scales = static_cast<uint8_t*>(out_scales);
    P.offsets = offsets;
    P.status = device_status_ptr();
    P.rows = c.rows;
    P.E = c.E; P.K = c.K; P.N = c.N; P.act = c.act;
    P.pitch = (int)mx8_pitch(c.K);
    P.out_pitch = (int)mx8_pitch(c.N);
    const int cols = (pair ? 256 : 128) / (dual ? 2 : 1);       // output columns of a tile
    P.n_blocks = (c.N + cols - 1) / cols;
    // Few tiles (a token or two in decoding): the CTAs of a cluster share a tile's K where a
    // share is long enough, us with 1, 2 and 4 of them (one row of one expert):
    //   1024 -> 1024   6.0  7.2       2048 -> 1024   8.2  8.3  9.0
    //   4096 -> 1024  12.6 10.6 10.1  14336 -> 4096 36.5 22.9 19.3
    // The host knows how many experts rows can name, not how many they do: two share where
    // the tiles might fit the GPU so, and the kernel looks whether they do (2 tokens of
    // 8 experts, top-2, 14336 -> 4096: 25 where rows name two of them, 37 without; in
    // turns they lose: four experts 49 for 40).
    const int64_t tiles = (c.rows / BM + std::min<int64_t>(c.E, c.rows)) * P.n_blocks;
    const int nk = (c.K + BK - 1) / BK, sms = num_sms();
    P.ways = pair ? 1 : nk >= 64 && tiles * 4 <= sms ? 4 : nk >= 24 && tiles <= sms ? 2 : 1;
    P.max_tiles = (int)std::min<int64_t>(tiles, sms / P.ways);
    return pair ? launch_mx8_out<2>(c, P, st) : launch_mx8_out<1>(c, P, st);
}

}  // namespace moe
