// norm_mx8.cu -- the residual stream's norms with the next block's input in 8 bits
// (norm_rows.cuh's forward kernels; the numbers: mx8.cuh).
//
// z never passes through memory in 16 bits on its way to the 8-bit numbers: a block's 32
// elements are those of four (bf16) or eight (fp32) neighbouring lanes, which find its
// largest magnitude in two or three shuffles.
//
// As a graph, bf16: 16384 x 4096, both norms, channel gate, z beside its codes 96 us
// (6.3 TB/s); 65536 x 4096 380 (6.4), without z 332 (5.7).  Entering alone 65536 x 4096 174
// (4.7), with z 240 (5.6): 64 % of the issue slots are taken, with 28 warps an SM, and a warp
// that does not issue waits at the row's barrier or for shared memory as often as for its turn.
// With the run-time flags, without z: full gate 65536 x 2048 188 (6.5), 65536 x 4096 375 (6.5),
// 5120 wide 4.3 TB/s (one CTA of 320 threads an SM); channel gate without post norm 65536 x 2048
// 158 (6.0).  More than 512 threads a row (bf16 above 8192 wide, fp32 above 4096) have 64
// registers each at most, and spill where they want about 100: 16384 x 12288 both norms 380 us
// without z (3.7 TB/s) and 419 with it (4.3), 16384 x 16384 443 and 481; addition and norm, which
// do not spill, 214 (6.6) and 302 (6.3).  fp32: 65536 x 2048, addition and norm, without z 295
// (5.9); 16384 x 8192 both norms 263 (6.6), addition and norm 301, entering alone 170 (4.0: 32
// registers and a few spilled).
#include "norm_rows.cuh"

namespace moe {

int launch_block_norm_mx8(const moe_norm_config& c, const void* x, const void* u, const float* w_post,
                          const void* gate, const float* w_pre, void* x_out, void* z, void* codes,
                          void* scales, cudaStream_t st) {
    NormArgs a = base_args(c);
    a.x = x; a.u = u; a.w_post = w_post; a.gate = gate; a.w_pre = w_pre; a.x_out = x_out; a.z = z;
    a.codes = static_cast<uint8_t*>(codes);
    a.scales = static_cast<uint8_t*>(scales);
    a.pitch = (int)mx8_pitch(c.d);
    return c.dtype == MOE_DTYPE_BF16 ? launch_fwd<__nv_bfloat16, 8, true>(c, a, st) : launch_fwd<float, 4, true>(c, a, st);
}

}  // namespace moe
