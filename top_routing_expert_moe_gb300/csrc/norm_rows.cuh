// norm_rows.cuh -- rows of the residual stream's norms: the forward kernels, the ring that
// brings long batches, and the plan of a launch (norm.cu, norm_mx8.cu).
#pragma once
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "mx8.cuh"
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

// VEC neighbouring elements of z a lane, so that 32 / VEC neighbouring lanes hold a block of
// the 8-bit numbers (rows are whole blocks; all lanes come here, those past the row's end
// with elements that are not stored).  z is rounded once, from fp32.
template <int VEC>
__device__ __forceinline__ void store_mx8(uint8_t* codes, uint8_t* scales, int c, int nvec, const float (&v)[VEC]) {
    uint32_t m = amax_bits<VEC>(v);
#pragma unroll
    for (int o = 1; o < 32 / VEC; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t s = mx8_scale_byte(m);
    uint32_t w[VEC / 4];
    mx8_codes<VEC>(v, s, w);
    if (c >= nvec) return;
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(codes + c * VEC) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(codes + c * VEC) = w[0];
    if (c % (32 / VEC) == 0) scales[c / (32 / VEC)] = (uint8_t)s;
}

struct NormArgs {
    const void *x, *u, *gate, *dx_out, *dz;   // x: the stream (x_out in the backward)
    const float *w_post, *w_pre;
    void *x_out, *z, *dx, *du, *dgate;
    uint8_t *codes, *scales;                  // z in 8 bits (then z itself may be absent)
    int pitch;                                // bytes of a row of scales
    float *part;                              // [3][grid][d]: dw_pre, dw_post, dgate partials
    int T, d, leave, post, enter, gmode;
    float eps, ra, ob;
};

// Q8: z leaves in 8 bits, and in T too where it is asked for
template <typename T, int VEC, int EPT, int MAXT, bool Q8>
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
                if constexpr (Q8)
                    store_mx8<VEC>(a.codes + o, a.scales + (size_t)t * a.pitch, c, nvec, y[i]);
                if (!Q8 || a.z) store_vec<T, VEC>(static_cast<T*>(a.z) + o, c, nvec, y[i]);
            }
        }
        // buf[0] and buf[1] alternate unless only one of the norms is on
        if (a.post != a.enter && blockDim.x > 32) __syncthreads();
    }
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
constexpr int RE = 8;                      // elements of a row per thread (see RE8 for z in 8 bits)
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

// With z in 8 bits too a row costs its threads more instructions, and the kernel is bound by
// issuing them: twice the elements a thread halve what is once a row (the reductions, the
// ring, addresses) for bf16.
template <typename T> constexpr int RE8 = sizeof(T) == 2 ? 16 : RE;

// A thread's 2 NP elements of a row.  WIDE (rows of whole 16 bytes): one 16-byte
// piece of bf16, or one of each half of an fp32 row (or of a bf16 row where there are
// 16 elements), so that neighbouring threads' accesses stay neighbours.  Otherwise
// elements tid, tid + threads, ...
template <typename T>
__device__ __forceinline__ int part_of(int half) { return (threadIdx.x + half * blockDim.x) * (16 / (int)sizeof(T)); }
template <typename T, bool WIDE, int NP>
__device__ __forceinline__ void take(const T* p, int d, f2 (&v)[NP]) {
    constexpr int V = 16 / sizeof(T);
    if constexpr (!WIDE) {
        float f[2 * NP];
#pragma unroll
        for (int j = 0; j < 2 * NP; ++j) {
            const int c = threadIdx.x + j * blockDim.x;
            f[j] = c < d ? to_f<T>(p[c]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) v[i] = pk(f[2 * i], f[2 * i + 1]);
    } else if constexpr (sizeof(T) == 2 && 2 * NP == V) {
        // threads past the row's end read its last elements; sums and stores leave them out
        const uint4 u = *reinterpret_cast<const uint4*>(p + min((int)threadIdx.x * V, d - V));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < NP; ++i) v[i] = pk(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
#pragma unroll
        for (int h = 0; h < 2 * NP / V; ++h) {
            const int c = part_of<T>(h);
            const uint4 u = c < d ? *reinterpret_cast<const uint4*>(p + c) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                if constexpr (sizeof(T) == 2)
                    v[h * V / 2 + i] = pk(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
                else v[h * V / 2 + i] = pk(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
            }
        }
    }
}
// This thread's share of a sum: its own, or none where it has read again what belongs
// to others (other shares past the end are zeros).  Chosen, not multiplied by 0: the
// elements read again may be infinite, or their squares.
template <typename T, bool WIDE, int NP = RP>
__device__ __forceinline__ bool live(int d) {
    constexpr int V = 16 / sizeof(T);
    return !WIDE || sizeof(T) == 4 || 2 * NP != V || (int)threadIdx.x * V < d;
}
template <typename T, bool WIDE, int NP>
__device__ __forceinline__ void give(T* p, int d, const f2 (&v)[NP]) {
    if constexpr (!WIDE) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            float lo, hi;
            unpk(v[i], lo, hi);
            const int c = threadIdx.x + 2 * i * blockDim.x;
            if (c < d) p[c] = from_f<T>(lo);
            if (c + (int)blockDim.x < d) p[c + blockDim.x] = from_f<T>(hi);
        }
    } else {
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int h = 0; h < 2 * NP / V; ++h) {
            const int c = part_of<T>(h);
            float f[V];
#pragma unroll
            for (int j = 0; j < V / 2; ++j) unpk(v[h * V / 2 + j], f[2 * j], f[2 * j + 1]);
            if (c < d) store16_f<T>(p + c, f);
        }
    }
}
// in 8 bits, by the same split
template <typename T, int NP>
__device__ __forceinline__ void give_mx8(uint8_t* codes, uint8_t* scales, int d, const f2 (&v)[NP]) {
    constexpr int V = 16 / sizeof(T);
#pragma unroll
    for (int h = 0; h < 2 * NP / V; ++h) {
        float f[V];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) unpk(v[h * V / 2 + j], f[2 * j], f[2 * j + 1]);
        store_mx8<V>(codes, scales, part_of<T>(h) / V, d / V, f);
    }
}
// the fp32 channel vector's share that goes with it
template <typename T, bool WIDE, int NP>
__device__ __forceinline__ void channel(const float* p, int d, f2 (&v)[NP]) {
    constexpr int V = WIDE ? 16 / sizeof(T) : 1;
    float f[2 * NP];
#pragma unroll
    for (int j = 0; j < 2 * NP; ++j) {
        const int c = WIDE ? part_of<T>(j / V) + j % V : threadIdx.x + j * blockDim.x;
        f[j] = c < d ? __ldg(p + c) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) v[i] = pk(f[2 * i], f[2 * i + 1]);
}
template <int NP>
__device__ __forceinline__ void fill(f2 (&v)[NP], float x) {
#pragma unroll
    for (int i = 0; i < NP; ++i) v[i] = both(x);
}
template <int NP>
__device__ __forceinline__ float dot2(const f2 (&a)[NP], const f2 (&b)[NP]) {
    f2 s = a[0] * b[0];
#pragma unroll
    for (int i = 1; i < NP; ++i) s = fma2(a[i], b[i], s);
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
// With 16 elements a thread both norms want about 100 registers, where the compiler aimed
// at 64 and spilled: two CTAs of 256 threads are what the plan counts on.
template <int FORM, int MAXT> constexpr int FWD8_CTAS = FORM == FORM_BOTH || FORM == FORM_ANY ? (MAXT == 256 ? 2 : 1) : 0;
template <int FORM, int MAXT> constexpr int BWD_CTAS = (FORM == FORM_ADD || FORM == FORM_ENTER) && MAXT == 768 ? 1 : 0;

// in: x, u (leave), gate (full)
template <typename T, bool WIDE, int FORM, int MAXT, bool Q8>
__global__ void __launch_bounds__(MAXT, (Q8 && sizeof(T) == 2 ? FWD8_CTAS<FORM, MAXT> : FWD_CTAS<WIDE, FORM, MAXT>))
block_norm_ring_kernel(const __grid_constant__ RingArgs a) {
    __shared__ float buf[2][32];
    NORM_RING_SETUP();
    const Parts p = parts_of<FORM>(n);
    const int gmode = FORM == FORM_ADD || FORM == FORM_ENTER ? MOE_GATE_NONE : n.gmode;
    constexpr int NP = (Q8 ? RE8<T> : RE) / 2;
    const bool on = live<T, WIDE, NP>(d);
    f2 wq[NP], wz[NP];                     // g w_post, w_pre
    fill(wq, 1.f);
    if (p.post) channel<T, WIDE>(n.w_post, d, wq);
    if (gmode == MOE_GATE_CHANNEL) {
        channel<T, WIDE>(static_cast<const float*>(n.gate), d, wz);
#pragma unroll
        for (int i = 0; i < NP; ++i) wq[i] = wq[i] * wz[i];
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
        f2 y[NP], u[NP];
        take<T, WIDE>(in(0), d, y);
        if (p.leave) {
            take<T, WIDE>(in(1), d, u);
            const float s = p.post && on ? dot2(u, u) : 0.f;
            if (p.full) {
                f2 g[NP];
                take<T, WIDE>(in(2), d, g);
#pragma unroll
                for (int i = 0; i < NP; ++i) u[i] = u[i] * g[i];
            }
            if (p.post) {
                tok *= rsqrtf(row_sum(s, buf[0]) * invd + n.eps);
            }
            const f2 c = both(tok), ra = both(n.ra);
#pragma unroll
            for (int i = 0; i < NP; ++i) y[i] = fma2(c * wq[i], u[i], ra * y[i]);
            give<T, WIDE>(static_cast<T*>(n.x_out) + o, d, y);
        }
        if (p.enter) {
            const float s = on ? dot2(y, y) : 0.f;
            ring.wait_next(a, t);
            const f2 r = both(rsqrtf(row_sum(s, buf[p.leave ? 1 : par]) * invd + n.eps));
#pragma unroll
            for (int i = 0; i < NP; ++i) y[i] = y[i] * (r * wz[i]);
            if constexpr (Q8) give_mx8<T>(n.codes + o, n.scales + (size_t)t * n.pitch, d, y);
            if (!Q8 || n.z) give<T, WIDE>(static_cast<T*>(n.z) + o, d, y);
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
// `by_warp`: registers are counted as they are handed out, to whole warps from the quarter of
// the file that their scheduler has.
RingPlan ring_plan(const moe_norm_config& c, int nin, int regs, bool backward, int re = RE, bool by_warp = false) {
    RingPlan p = {0, 0, 0, 0};
    const int es = c.dtype == MOE_DTYPE_BF16 ? 2 : 4;
    p.threads = ((c.d + re - 1) / re + 31) / 32 * 32;
    if (p.threads > 1024 || !ring_pays(c, backward)) return p;
    const int stage = nin * (int)row_pitch(c.d * es);
    // CTAs an SM by registers and threads, fewer where they would not have three stages
    // each (228 KB an SM, 3 KB of it a CTA's fixed part)
    const int fit = by_warp ? 16384 / (32 * regs) * 4 / (p.threads / 32) : 65536 / (regs * p.threads);
    int per_sm = std::max(1, std::min(std::min(32, fit), 2048 / p.threads));
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
template <typename T, bool WIDE, int FORM, int MAXT, bool Q8>
int launch_fwd_ring_t(const RingPlan& p, const RingArgs& r, cudaStream_t st) {
    static bool done[64] = {};
    if (const int e = smem_attr_once(block_norm_ring_kernel<T, WIDE, FORM, MAXT, Q8>, 200 * 1024, done)) return e;
    MOE_LAUNCH((block_norm_ring_kernel<T, WIDE, FORM, MAXT, Q8>), p.grid, p.threads, p.smem, st, r);
    return MOE_OK;
}
template <typename T, bool WIDE, int FORM, bool Q8>
int launch_fwd_ring_f(const RingPlan& p, const RingArgs& r, cudaStream_t st) {
    if constexpr (Q8 && sizeof(T) == 2)
        if (p.threads <= 256) return launch_fwd_ring_t<T, WIDE, FORM, 256, Q8>(p, r, st);
    return p.threads <= 512 ? launch_fwd_ring_t<T, WIDE, FORM, 512, Q8>(p, r, st)
                            : launch_fwd_ring_t<T, WIDE, FORM, 1024, Q8>(p, r, st);
}
template <typename T, bool WIDE, bool Q8>
int launch_fwd_ring(const RingPlan& p, const RingArgs& r, cudaStream_t st) {
    switch (form_of(r.n, false)) {
        case FORM_BOTH: return launch_fwd_ring_f<T, WIDE, FORM_BOTH, Q8>(p, r, st);
        case FORM_ADD: return launch_fwd_ring_f<T, WIDE, FORM_ADD, Q8>(p, r, st);
        case FORM_ENTER: return launch_fwd_ring_f<T, WIDE, FORM_ENTER, Q8>(p, r, st);
        default: return launch_fwd_ring_f<T, WIDE, FORM_ANY, Q8>(p, r, st);
    }
}
template <typename T, int VEC, bool Q8 = false>
int launch_fwd(const moe_norm_config& c, const NormArgs& a, cudaStream_t st) {
    const bool heavy = c.post_norm || c.gate != MOE_GATE_NONE;
    // With 16 elements a thread the forms' registers differ (96 for both norms, 106 with the
    // run-time flags), and a CTA counted that does not fit costs a second wave (65536 x 2048, full
    // gate, 96 counted for all: 270 us, so 188; both norms at 1536 and 3584, where a scheduler's
    // quarter does not divide evenly, 172 and 416, so 121 and 315).
    constexpr bool by_warp = Q8 && sizeof(T) == 2;
    const int regs = by_warp ? (form_of(a, false) == FORM_ANY ? 112 : heavy ? 96 : 64) : heavy ? 64 : Q8 ? 48 : 40;
    const RingPlan p = ring_plan(c, fwd_inputs(c), regs, false, Q8 ? RE8<T> : RE, by_warp);
    if (p.stages) {
        RingArgs r = {};
        r.n = a;
        r.in[r.nin++] = a.x;
        if (c.leave) r.in[r.nin++] = a.u;
        if (c.gate == MOE_GATE_FULL) r.in[r.nin++] = a.gate;
        r.stages = p.stages;
        r.status = device_status_ptr();
        return launch_fwd_ring<T, (VEC > 1), Q8>(p, r, st);
    }
    const dim3 b = norm_block(c);
    const int grid = (int)std::min<int64_t>(((int64_t)c.T + b.y - 1) / b.y, (int64_t)num_sms() * 64);
    if (direct_ept(c) == 16) MOE_LAUNCH((block_norm_kernel<T, VEC, 16, 1024, Q8>), grid, b, 0, st, a);
    else if (b.x <= 256) MOE_LAUNCH((block_norm_kernel<T, VEC, 8, 256, Q8>), grid, b, 0, st, a);
    else MOE_LAUNCH((block_norm_kernel<T, VEC, 8, 1024, Q8>), grid, b, 0, st, a);
    return MOE_OK;
}
NormArgs base_args(const moe_norm_config& c) {
    NormArgs a = {};
    a.T = c.T; a.d = c.d; a.leave = c.leave; a.post = c.post_norm; a.enter = c.enter;
    a.gmode = c.gate; a.eps = c.eps; a.ra = c.res_scale; a.ob = c.out_scale;
    return a;
}

}  // namespace

}  // namespace moe
