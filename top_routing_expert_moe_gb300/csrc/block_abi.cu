// block_abi.cu -- the extern "C" entry points of the operators around the layer:
// argument checks, then the launchers.
#include <cmath>

#include "common.cuh"
#include "kernels.h"

using namespace moe;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_ptr(const void* p) { return p != nullptr && aligned16(p); }
// a pointer that is there exactly when `on`
bool ok_if(bool on, const void* p) { return on ? ok_ptr(p) : p == nullptr; }
bool is_flag(int v) { return v == 0 || v == 1; }
bool is_dtype(int v) { return v == MOE_DTYPE_F32 || v == MOE_DTYPE_BF16; }
// a tensor of 4-bit numbers: rows, and a width that is whole blocks
int mx4_shape(int64_t rows, int K) {
    if (rows < 1 || K < 1) return MOE_ERR_INVALID_ARG;
    return K % 32 || K > (1 << 24) || rows > (1LL << 31) - 256 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

}  // namespace

extern "C" {

int moe_check_norm_config(const moe_norm_config* c) {
    if (!c || c->T < 1 || c->d < 1) return MOE_ERR_INVALID_ARG;
    if (c->dtype != MOE_DTYPE_F32 && c->dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
    if (!is_flag(c->leave) || !is_flag(c->post_norm) || !is_flag(c->enter)) return MOE_ERR_INVALID_ARG;
    if (c->gate < MOE_GATE_NONE || c->gate > MOE_GATE_FULL) return MOE_ERR_INVALID_ARG;
    if (!c->leave && (c->post_norm || !c->enter || c->gate != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(c->eps) || !(c->eps > 0.f)) return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(c->res_scale) || !std::isfinite(c->out_scale)) return MOE_ERR_INVALID_ARG;
    if (c->d > MOE_NORM_MAX_D) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int moe_norm_workspace_size(const moe_norm_config* c, size_t* bytes) {
    const int r = moe_check_norm_config(c);
    if (r) return r;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = norm_ws_bytes(*c);
    return MOE_OK;
}

int moe_block_norm(const moe_norm_config* c, const void* x, const void* u, const float* w_post,
                   const void* gate, const float* w_pre, void* x_out, void* z, moe_stream_t stream) {
    const int r = moe_check_norm_config(c);
    if (r) return r;
    if (!ok_ptr(x) || !ok_if(c->leave, u) || !ok_if(c->post_norm, w_post) ||
        !ok_if(c->gate != MOE_GATE_NONE, gate) || !ok_if(c->enter, w_pre) ||
        !ok_if(c->leave, x_out) || !ok_if(c->enter, z))
        return MOE_ERR_INVALID_ARG;
    return launch_block_norm(*c, x, u, w_post, gate, w_pre, x_out, z, (cudaStream_t)stream);
}

int moe_block_norm_backward(const moe_norm_config* c, const void* x_out, const void* u,
                            const float* w_post, const void* gate, const float* w_pre,
                            const void* dx_out, const void* dz, void* dx, void* du, float* dw_post,
                            void* dgate, float* dw_pre, void* ws, moe_stream_t stream) {
    const int r = moe_check_norm_config(c);
    if (r) return r;
    const bool gated = c->gate != MOE_GATE_NONE;
    // u and x_out are read only where a norm or a gate needs them, dx_out may be zero (NULL)
    const bool u_ok = !c->leave ? u == nullptr : (c->post_norm || gated) ? ok_ptr(u) : aligned16(u);
    const bool y_ok = c->enter ? ok_ptr(x_out) : aligned16(x_out);
    const bool g_ok = c->enter ? aligned16(dx_out) : ok_ptr(dx_out);
    if (!y_ok || !u_ok || !g_ok || !ok_if(c->post_norm, w_post) || !ok_if(gated, gate) ||
        !ok_if(c->enter, w_pre) || !ok_if(c->enter, dz) || !ok_ptr(dx) || !ok_if(c->leave, du) ||
        !ok_if(c->post_norm, dw_post) || !ok_if(gated, dgate) || !ok_if(c->enter, dw_pre) || !ok_ptr(ws))
        return MOE_ERR_INVALID_ARG;
    return launch_block_norm_backward(*c, x_out, u, w_post, gate, w_pre, dx_out, dz, dx, du, dw_post,
                                      dgate, dw_pre, ws, (cudaStream_t)stream);
}

int moe_check_balance_config(const moe_balance_config* c) {
    if (!c || c->T < 1 || c->E < 1 || c->k < 1 || c->k > c->E || c->S < 1) return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(c->balance_coef) || !std::isfinite(c->z_coef)) return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(c->temperature) || c->temperature < 0.f) return MOE_ERR_INVALID_ARG;
    if (c->E > 256 || c->k > 16 || c->S > 65536 || c->T > (1 << 30)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int moe_balance_workspace_size(const moe_balance_config* c, size_t* bytes) {
    const int r = moe_check_balance_config(c);
    if (r) return r;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = balance_ws_bytes(*c);
    return MOE_OK;
}

int moe_balance_loss(const moe_balance_config* c, const float* logits, const int32_t* topk_idx,
                     const int32_t* seq_offsets, float* loss, int32_t* counts, float* pbar,
                     float* grad_w, void* ws, moe_stream_t stream) {
    const int r = moe_check_balance_config(c);
    if (r) return r;
    if (!ok_ptr(logits) || !ok_ptr(topk_idx) || !aligned16(seq_offsets) || !ok_ptr(loss) ||
        !ok_ptr(counts) || !ok_ptr(pbar) || !ok_ptr(grad_w) || !ok_ptr(ws))
        return MOE_ERR_INVALID_ARG;
    if (!seq_offsets && c->S != 1) return MOE_ERR_INVALID_ARG;
    return launch_balance_loss(*c, logits, topk_idx, seq_offsets, loss, counts, pbar, grad_w, ws,
                               (cudaStream_t)stream);
}

int moe_balance_loss_backward(const moe_balance_config* c, const float* logits,
                              const int32_t* topk_idx, const int32_t* seq_offsets,
                              const float* grad_w, const float* dloss, float* dlogits,
                              moe_stream_t stream) {
    const int r = moe_check_balance_config(c);
    if (r) return r;
    if (!ok_ptr(logits) || !ok_ptr(topk_idx) || !aligned16(seq_offsets) || !ok_ptr(grad_w) ||
        !aligned16(dloss) || !ok_ptr(dlogits))
        return MOE_ERR_INVALID_ARG;
    if (!seq_offsets && c->S != 1) return MOE_ERR_INVALID_ARG;
    return launch_balance_loss_backward(*c, logits, topk_idx, seq_offsets, grad_w, dloss, dlogits,
                                        (cudaStream_t)stream);
}

int moe_mx4_scale_bytes(int64_t rows, int32_t K, size_t* bytes) {
    const int r = mx4_shape(rows, K);
    if (r) return r;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = (size_t)((rows + 127) / 128) * ((K + 127) / 128) * 512;
    return MOE_OK;
}

int moe_mx4_quantize(int32_t dtype, int64_t rows, int32_t K, const void* x, const int32_t* rows_used,
                     void* codes, void* scales, moe_stream_t stream) {
    if (!is_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    const int r = mx4_shape(rows, K);
    if (r) return r;
    // rows_used points into an offsets array, so 4-byte alignment is enough
    if (!ok_ptr(x) || (reinterpret_cast<uintptr_t>(rows_used) & 3u) || !ok_ptr(codes) || !ok_ptr(scales))
        return MOE_ERR_INVALID_ARG;
    return launch_mx4_quantize(dtype, rows, K, x, rows_used, codes, scales, (cudaStream_t)stream);
}

int moe_mx4_quantize_weight(int32_t dtype, int32_t E, int32_t K, int32_t N, const void* W,
                            void* codes, void* scales, moe_stream_t stream) {
    if (!is_dtype(dtype) || E < 1) return MOE_ERR_INVALID_ARG;
    const int r = mx4_shape(N, K);
    if (r) return r;
    // (the launch's grid: 64-column tiles and experts)
    if (N % 8 || N > (1 << 21) || E > 65535) return MOE_ERR_UNSUPPORTED;
    if (!ok_ptr(W) || !ok_ptr(codes) || !ok_ptr(scales)) return MOE_ERR_INVALID_ARG;
    return launch_mx4_quantize_weight(dtype, E, K, N, W, codes, scales, (cudaStream_t)stream);
}

int moe_mx4_dequantize(int32_t dtype, int32_t sets, int64_t rows, int32_t K, const void* codes,
                       const void* scales, void* out, moe_stream_t stream) {
    if (!is_dtype(dtype) || sets < 1) return MOE_ERR_INVALID_ARG;
    const int r = mx4_shape(rows, K);
    if (r) return r;
    if ((rows + 127) / 128 * sets > (1 << 26)) return MOE_ERR_UNSUPPORTED;   // 32-bit tile counts
    if (!ok_ptr(codes) || !ok_ptr(scales) || !ok_ptr(out)) return MOE_ERR_INVALID_ARG;
    return launch_mx4_dequantize(dtype, sets, rows, K, codes, scales, out, (cudaStream_t)stream);
}

int moe_check_mx4_product_config(const moe_mx4_product_config* c) {
    if (!c || c->N < 1 || c->E < 1 || !is_dtype(c->out_dtype)) return MOE_ERR_INVALID_ARG;
    if (c->act < MOE_MX4_ACT_NONE || c->act > MOE_MX4_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
    const int r = mx4_shape(c->rows, c->K);
    if (r) return r;
    if (c->N % 8 || c->N > (1 << 21) || c->E > 64 || c->rows > (1 << 30)) return MOE_ERR_UNSUPPORTED;
    // 32-bit tile counts, at the smallest tile's 64 columns
    if ((c->rows / 128 + c->E) * (((int64_t)c->N + 63) / 64) > (1LL << 30)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int moe_mx4_grouped_product(const moe_mx4_product_config* c, const void* x_codes, const void* x_scales,
                            const int32_t* offsets, const void* w_codes, const void* w_scales,
                            const void* wg_codes, const void* wg_scales, void* out,
                            moe_stream_t stream) {
    const int r = moe_check_mx4_product_config(c);
    if (r) return r;
    const bool dual = c->act == MOE_MX4_ACT_SWIGLU;
    if (!ok_ptr(x_codes) || !ok_ptr(x_scales) || !ok_ptr(offsets) || !ok_ptr(w_codes) ||
        !ok_ptr(w_scales) || !ok_if(dual, wg_codes) || !ok_if(dual, wg_scales) || !ok_ptr(out))
        return MOE_ERR_INVALID_ARG;
    return launch_mx4_product(*c, x_codes, x_scales, offsets, w_codes, w_scales, wg_codes, wg_scales,
                              out, (cudaStream_t)stream);
}

}  // extern "C"
