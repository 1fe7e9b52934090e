// mx8_abi.cu -- the extern "C" entry points of the 8-bit operators: argument checks,
// then the launchers.
#include <algorithm>

#include "kernels.h"
#include "mx8.cuh"

using namespace moe;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_ptr(const void* p) { return p != nullptr && aligned16(p); }
// a pointer that is there exactly when `on`
bool ok_if(bool on, const void* p) { return on ? ok_ptr(p) : p == nullptr; }
bool is_dtype(int v) { return v == MOE_DTYPE_F32 || v == MOE_DTYPE_BF16; }
// a tensor of 8-bit numbers: rows, and a width that is whole blocks
int mx8_shape(int64_t rows, int K) {
    if (rows < 1 || K < 1) return MOE_ERR_INVALID_ARG;
    return K % 32 || K > (1 << 24) || rows > (1LL << 31) - 256 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
// expert weights: W's columns in whole 16-byte pieces, and the launches' grids (64-column
// tiles, experts); 128-byte rows of all blocks counted in 31 bits
int weight8_shape(int64_t E, int K, int N) {
    if (E < 1 || N < 1) return MOE_ERR_INVALID_ARG;
    const int r = mx8_shape(N, K);
    if (r) return r;
    if (N % 8 || N > (1 << 21) || E > 65535) return MOE_ERR_UNSUPPORTED;
    return E * ((N + 127) / 128) * ((K + 127) / 128) > (1LL << 31) / 128 - 1 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
int64_t rows_cap8(const moe_config& c) { return std::min<int64_t>((int64_t)c.T * c.k, (int64_t)c.E * capacity_of(c)); }
int permute8_config(const moe_config* c) {
    const int r = moe_check_config(c);
    if (r) return r;
    return c->d % 32 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

}  // namespace

extern "C" {

int moe_mx8_scale_pitch(int32_t K, int32_t* pitch) {
    const int r = mx8_shape(1, K);
    if (r) return r;
    if (!pitch) return MOE_ERR_INVALID_ARG;
    *pitch = (int32_t)mx8_pitch(K);
    return MOE_OK;
}

int moe_mx8_quantize(int32_t dtype, int64_t rows, int32_t K, const void* x, const int32_t* rows_used,
                     void* codes, void* scales, moe_stream_t stream) {
    if (!is_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    const int r = mx8_shape(rows, K);
    if (r) return r;
    // rows_used points into an offsets array, so 4-byte alignment is enough
    if (!ok_ptr(x) || (reinterpret_cast<uintptr_t>(rows_used) & 3u) || !ok_ptr(codes) || !ok_ptr(scales))
        return MOE_ERR_INVALID_ARG;
    return launch_mx8_quantize(dtype, rows, K, x, rows_used, codes, scales, (cudaStream_t)stream);
}

int moe_mx8_weight_bytes(int32_t E, int32_t K, int32_t N, size_t* codes, size_t* scales) {
    const int r = weight8_shape(E, K, N);
    if (r) return r;
    if (!codes || !scales) return MOE_ERR_INVALID_ARG;
    const size_t blocks = (size_t)E * ((N + 127) / 128) * ((K + 127) / 128);
    *codes = blocks * 16384;
    *scales = blocks * 512;
    return MOE_OK;
}

int moe_mx8_quantize_weight(int32_t dtype, int32_t E, int32_t K, int32_t N, const void* W,
                            void* codes, void* scales, moe_stream_t stream) {
    if (!is_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    const int r = weight8_shape(E, K, N);
    if (r) return r;
    if (!ok_ptr(W) || !ok_ptr(codes) || !ok_ptr(scales)) return MOE_ERR_INVALID_ARG;
    return launch_mx8_quantize_weight(dtype, E, K, N, W, codes, scales, (cudaStream_t)stream);
}

int moe_mx8_dequantize_weight(int32_t dtype, int32_t E, int32_t K, int32_t N, const void* codes,
                              const void* scales, void* out, moe_stream_t stream) {
    if (!is_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    const int r = weight8_shape(E, K, N);
    if (r) return r;
    if (!ok_ptr(codes) || !ok_ptr(scales) || !ok_ptr(out)) return MOE_ERR_INVALID_ARG;
    return launch_mx8_dequantize_weight(dtype, E, K, N, codes, scales, out, (cudaStream_t)stream);
}

int moe_mx8_dequantize(int32_t dtype, int64_t rows, int32_t K, const void* codes, const void* scales,
                       void* out, moe_stream_t stream) {
    if (!is_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    const int r = mx8_shape(rows, K);
    if (r) return r;
    if (!ok_ptr(codes) || !ok_ptr(scales) || !ok_ptr(out)) return MOE_ERR_INVALID_ARG;
    return launch_mx8_dequantize(dtype, rows, K, codes, scales, out, (cudaStream_t)stream);
}

int moe_mx8_rows_capacity(const moe_config* c, int64_t* rows) {
    const int r = moe_check_config(c);
    if (r) return r;
    if (!rows) return MOE_ERR_INVALID_ARG;
    *rows = rows_cap8(*c);
    return MOE_OK;
}

int moe_permute_mx8_workspace_size(const moe_config* c, size_t* bytes) {
    const int r = permute8_config(c);
    if (r) return r;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = permute_ws_bytes(*c);
    return MOE_OK;
}

int moe_permute_mx8(const moe_config* c, const void* codes, const void* scales, const int32_t* topk_idx,
                    void* codes_perm, void* scales_perm, int32_t* perm_token, int32_t* slot_of,
                    int32_t* kept, int32_t* offsets, float* stats, void* ws, moe_stream_t stream) {
    const int r = permute8_config(c);
    if (r) return r;
    if (!ok_ptr(codes) || !ok_ptr(scales) || !ok_ptr(topk_idx) || !ok_ptr(codes_perm) || !ok_ptr(scales_perm) ||
        !ok_ptr(perm_token) || !ok_ptr(slot_of) || !ok_ptr(kept) || !ok_ptr(offsets) || !aligned16(stats) ||
        !ok_ptr(ws))
        return MOE_ERR_INVALID_ARG;
    return launch_permute_mx8(*c, codes, scales, topk_idx, codes_perm, scales_perm, perm_token, slot_of, kept,
                              offsets, stats, ws, (cudaStream_t)stream);
}

int moe_block_norm_mx8(const moe_norm_config* c, const void* x, const void* u, const float* w_post,
                       const void* gate, const float* w_pre, void* x_out, void* z, void* codes,
                       void* scales, moe_stream_t stream) {
    const int r = moe_check_norm_config(c);
    if (r) return r;
    if (!c->enter) return MOE_ERR_INVALID_ARG;
    if (c->d % 32) return MOE_ERR_UNSUPPORTED;
    if (!ok_ptr(x) || !ok_if(c->leave, u) || !ok_if(c->post_norm, w_post) ||
        !ok_if(c->gate != MOE_GATE_NONE, gate) || !ok_ptr(w_pre) || !ok_if(c->leave, x_out) ||
        !aligned16(z) || !ok_ptr(codes) || !ok_ptr(scales))
        return MOE_ERR_INVALID_ARG;
    return launch_block_norm_mx8(*c, x, u, w_post, gate, w_pre, x_out, z, codes, scales, (cudaStream_t)stream);
}

int moe_check_mx8_product_config(const moe_mx8_product_config* c) {
    if (!c || c->N < 1 || c->E < 1) return MOE_ERR_INVALID_ARG;
    if (!is_dtype(c->out_dtype) && c->out_dtype != MOE_DTYPE_MX8) return MOE_ERR_INVALID_ARG;
    if (c->act < MOE_MX8_ACT_NONE || c->act > MOE_MX8_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
    const int r = mx8_shape(c->rows, c->K);
    if (r) return r;
    if (c->N % (c->out_dtype == MOE_DTYPE_MX8 ? 32 : 8) || c->N > (1 << 21) || c->E > 64 || c->rows > (1 << 30))
        return MOE_ERR_UNSUPPORTED;
    if (const int w = weight8_shape(c->E, c->K, c->N)) return w;
    // 32-bit tile counts, at the smallest tile's 64 columns
    if ((c->rows / 128 + c->E) * (((int64_t)c->N + 63) / 64) > (1LL << 30)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int moe_mx8_grouped_product(const moe_mx8_product_config* c, const void* x_codes, const void* x_scales,
                            const int32_t* offsets, const void* w_codes, const void* w_scales,
                            const void* wg_codes, const void* wg_scales, void* out, void* out_scales,
                            moe_stream_t stream) {
    const int r = moe_check_mx8_product_config(c);
    if (r) return r;
    const bool dual = c->act == MOE_MX8_ACT_SWIGLU;
    if (!ok_ptr(x_codes) || !ok_ptr(x_scales) || !ok_ptr(offsets) || !ok_ptr(w_codes) ||
        !ok_ptr(w_scales) || !ok_if(dual, wg_codes) || !ok_if(dual, wg_scales) || !ok_ptr(out) ||
        !ok_if(c->out_dtype == MOE_DTYPE_MX8, out_scales))
        return MOE_ERR_INVALID_ARG;
    return launch_mx8_product(*c, x_codes, x_scales, offsets, w_codes, w_scales, wg_codes, wg_scales, out,
                              out_scales, (cudaStream_t)stream);
}

}  // extern "C"
