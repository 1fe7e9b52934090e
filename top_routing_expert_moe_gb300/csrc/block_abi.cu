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

}  // extern "C"
