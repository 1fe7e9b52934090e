// norm_mx8.cu -- the residual stream's norms with the next block's input in 8 bits
// (norm_rows.cuh's forward kernels; the numbers: mx8.cuh).
//
// z never passes through memory in 16 bits on its way to the 8-bit numbers: a block's 32
// elements are those of four (bf16) or eight (fp32) neighbouring lanes, which find its
// largest magnitude in two or three shuffles.
//
// As a graph, bf16: 16384 x 4096, both norms, channel gate, z beside its codes 96 us
// (6.3 TB/s); 65536 x 4096 380 (6.4), without z 332 (5.7), entering alone 174 (4.7: issue);
// 16384 x 12288 410 (4.4).  fp32: 65536 x 2048, addition and norm, without z 295 (5.9).
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
