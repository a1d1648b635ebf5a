// backward_api.cu -- the C ABI of the backward pass and of gradient clipping
// (declared in include/moe.h): argument checks, workspace layout, launches.
#include "api.h"

namespace moe {
namespace {

// Workspace of moe_backward (256-byte aligned sub-buffers).
struct BwdLayout {
    size_t dy_perm, dx_perm, x_perm, dw, dlogits, experts, route, total;
};

size_t es(const Shape &s) { return s.bf16 ? 2 : 4; }

size_t experts_scratch_bytes(const Shape &s) {
    return s.bf16 ? experts_backward_tc_scratch_bytes(s) : 4 * (size_t)s.P() * 2 * s.f;
}

BwdLayout bwd_layout(const Shape &s) {
    BwdLayout L;
    const size_t P = (size_t)s.P();
    size_t o = 0;
    L.dy_perm = o; o = up256(o + es(s) * P * s.d);
    L.dx_perm = o; o = up256(o + es(s) * P * s.d);
    L.x_perm = o;
    if (ws_layout(s).x_perm == MOE_WS_ABSENT) o = up256(o + es(s) * P * s.d);
    L.dw = o; o = up256(o + 4 * P);
    L.dlogits = o; o = up256(o + 4 * (size_t)s.T * s.E);
    L.experts = o; o = up256(o + experts_scratch_bytes(s));
    L.route = o; o = up256(o + route_backward_scratch_bytes(s));
    L.total = o;
    return L;
}

moe_status_t run_experts_backward(const Shape &s, const ExpertsBwd &a, const DevStatus &ds,
                                  cudaStream_t st) {
    return from_cuda(s.bf16 ? launch_experts_backward_tc(s, a, ds, st)
                            : launch_experts_backward_f32(s, a, st),
                     "grouped SwiGLU gradient launch");
}

moe_status_t check_ws(size_t have, size_t need) {
    if (have >= need) return MOE_OK;
    set_error_message("workspace %zu bytes < %zu needed", have, need);
    return MOE_ERR_WORKSPACE;
}

// Weight gradients of an empty batch.
moe_status_t clear(void *p, size_t bytes, cudaStream_t st) {
    return p ? from_cuda(cudaMemsetAsync(p, 0, bytes, st), "clearing a gradient") : MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_combine_backward(const moe_config_t *cfg, const void *dout, const void *y_perm,
                                  const int32_t *pos, const float *topk_w, void *dy_perm,
                                  float *dtopk_w, void *stream) {
    set_error_message("");
    Shape s;
    moe_status_t st = check_cfg(cfg, &s);
    if (st != MOE_OK) return st;
    if (s.T == 0) return MOE_OK;  // empty batch: nothing to check or launch
    if ((st = check_ptrs({dout, pos, dy_perm})) != MOE_OK) return st;
    if (!s.scale_inputs && (st = check_ptrs({y_perm, topk_w, dtopk_w})) != MOE_OK) return st;
    DevStatus ds;
    if ((st = device_status(&ds)) != MOE_OK) return st;
    const bool w = !s.scale_inputs;
    return from_cuda(launch_scatter_rows(s, dout, w ? y_perm : nullptr, pos, w ? topk_w : nullptr,
                                         dy_perm, w ? dtopk_w : nullptr,
                                         static_cast<cudaStream_t>(stream)),
                     "combine gradient launch");
}

moe_status_t moe_dispatch_backward(const moe_config_t *cfg, const void *dx_perm,
                                   const int32_t *pos, const float *topk_w, const void *x, void *dx,
                                   float *dtopk_w, void *stream) {
    set_error_message("");
    Shape s;
    moe_status_t st = check_cfg(cfg, &s);
    if (st != MOE_OK) return st;
    if (s.T == 0) return MOE_OK;  // empty batch: nothing to check or launch
    if ((st = check_ptrs({dx_perm, pos, dx})) != MOE_OK) return st;
    if (s.scale_inputs && (st = check_ptrs({topk_w, x, dtopk_w})) != MOE_OK) return st;
    DevStatus ds;
    if ((st = device_status(&ds)) != MOE_OK) return st;
    const bool w = s.scale_inputs;
    return from_cuda(launch_dispatch_backward(s, dx_perm, pos, w ? topk_w : nullptr,
                                              w ? x : nullptr, dx, w ? dtopk_w : nullptr,
                                              static_cast<cudaStream_t>(stream)),
                     "dispatch gradient launch");
}

size_t moe_grouped_swiglu_backward_workspace_size(const moe_config_t *cfg) {
    Shape s;
    if (check_cfg(cfg, &s) != MOE_OK || s.T == 0) return 0;
    return experts_scratch_bytes(s);
}

moe_status_t moe_grouped_swiglu_backward(const moe_config_t *cfg, const void *x_perm,
                                         const int32_t *offsets, const void *W_gate_up,
                                         const void *W_down, const void *h_perm,
                                         const void *dy_perm, void *dx_perm, void *dW_gate_up,
                                         void *dW_down, void *ws, size_t ws_bytes, void *stream) {
    set_error_message("");
    Shape s;
    moe_status_t st = check_cfg(cfg, &s);
    if (st != MOE_OK) return st;
    if ((st = check_ptrs({dW_gate_up, dW_down})) != MOE_OK) return st;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    DevStatus ds;
    if (s.T == 0) {
        const size_t n = es(s) * (size_t)s.E * s.d * s.f;
        if ((st = device_status(&ds)) != MOE_OK || (st = clear(dW_gate_up, 2 * n, cs)) != MOE_OK)
            return st;
        return clear(dW_down, n, cs);
    }
    if ((st = check_ptrs({x_perm, offsets, W_gate_up, W_down, h_perm, dy_perm, dx_perm, ws})) !=
        MOE_OK)
        return st;
    if ((st = check_ws(ws_bytes, experts_scratch_bytes(s))) != MOE_OK) return st;
    if ((st = device_status(&ds)) != MOE_OK) return st;
    return run_experts_backward(s, {x_perm, offsets, W_gate_up, W_down, h_perm, dy_perm, dx_perm,
                                    dW_gate_up, dW_down, ws}, ds, cs);
}

size_t moe_route_backward_workspace_size(const moe_config_t *cfg) {
    Shape s;
    if (check_cfg(cfg, &s) != MOE_OK || s.T == 0) return 0;
    return route_backward_scratch_bytes(s);
}

moe_status_t moe_route_backward(const moe_config_t *cfg, const void *x, const float *Wr,
                                const float *logits, const int32_t *topk_idx, const float *topk_w,
                                const float *dtopk_w, const void *dx_in, float *dlogits, float *dWr,
                                float *dlogit_bias, void *dx, void *ws, size_t ws_bytes,
                                void *stream) {
    set_error_message("");
    Shape s;
    moe_status_t st = check_cfg(cfg, &s);
    if (st != MOE_OK) return st;
    if ((st = check_ptrs({dWr})) != MOE_OK) return st;
    if (dlogit_bias && !aligned16(dlogit_bias)) {
        set_error_message("dlogit_bias is not 16-byte aligned");
        return MOE_ERR_INVALID_ARG;
    }
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    DevStatus ds;
    if (s.T == 0) {
        if ((st = device_status(&ds)) != MOE_OK ||
            (st = clear(dWr, 4 * (size_t)s.E * s.d, cs)) != MOE_OK)
            return st;
        return clear(dlogit_bias, 4 * (size_t)s.E, cs);
    }
    if ((st = check_ptrs({x, Wr, topk_idx, topk_w, dtopk_w, dlogits, dx, ws})) != MOE_OK) return st;
    if (!s.renorm && (st = check_ptrs({logits})) != MOE_OK) return st;
    if (dx_in && !aligned16(dx_in)) {
        set_error_message("dx_in is not 16-byte aligned");
        return MOE_ERR_INVALID_ARG;
    }
    if ((st = check_ws(ws_bytes, route_backward_scratch_bytes(s))) != MOE_OK) return st;
    if ((st = device_status(&ds)) != MOE_OK) return st;
    return from_cuda(launch_route_backward(s, {x, Wr, logits, topk_idx, topk_w, dtopk_w, dx_in,
                                               dlogits, dWr, dlogit_bias, dx, ws}, ds, cs),
                     "router gradient launch");
}

size_t moe_backward_workspace_size(const moe_config_t *cfg) {
    Shape s;
    if (check_cfg(cfg, &s) != MOE_OK || s.T == 0) return 0;
    return bwd_layout(s).total;
}

moe_status_t moe_backward(const moe_config_t *cfg, const void *x, const float *Wr,
                          const void *W_gate_up, const void *W_down, const void *fwd_ws,
                          size_t fwd_ws_bytes, const void *dout, void *dx, float *dWr,
                          float *dlogit_bias, void *dW_gate_up, void *dW_down, void *ws,
                          size_t ws_bytes, void *stream) {
    set_error_message("");
    Shape s;
    moe_status_t st = check_cfg(cfg, &s);
    if (st != MOE_OK) return st;
    if (s.T == 0) {  // clears the weight gradients
        if ((st = moe_route_backward(cfg, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                     nullptr, nullptr, dWr, dlogit_bias, nullptr, nullptr, 0,
                                     stream)) != MOE_OK)
            return st;
        return moe_grouped_swiglu_backward(cfg, nullptr, nullptr, nullptr, nullptr, nullptr,
                                           nullptr, nullptr, dW_gate_up, dW_down, nullptr, 0,
                                           stream);
    }
    if ((st = check_ptrs({x, Wr, W_gate_up, W_down, fwd_ws, dout, dx, dWr, dW_gate_up, dW_down,
                          ws})) != MOE_OK)
        return st;
    if (dlogit_bias && !aligned16(dlogit_bias)) {
        set_error_message("dlogit_bias is not 16-byte aligned");
        return MOE_ERR_INVALID_ARG;
    }
    const WsLayout F = ws_layout(s);
    const BwdLayout L = bwd_layout(s);
    if (fwd_ws_bytes < F.total) {
        set_error_message("forward workspace %zu bytes < %zu needed", fwd_ws_bytes, F.total);
        return MOE_ERR_WORKSPACE;
    }
    if (fwd_ws == ws) {
        set_error_message("ws is the forward workspace");
        return MOE_ERR_INVALID_ARG;
    }
    if ((st = check_ws(ws_bytes, L.total)) != MOE_OK) return st;
    DevStatus ds;
    if ((st = device_status(&ds)) != MOE_OK) return st;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const int32_t *pos = at<int32_t>(fwd_ws, F.pos);
    const float *w = at<float>(fwd_ws, F.w);
    void *dy_perm = at<uint8_t>(ws, L.dy_perm), *dx_perm = at<uint8_t>(ws, L.dx_perm);
    float *dw = at<float>(ws, L.dw);
    const bool scale = s.scale_inputs;
    if ((st = from_cuda(launch_scatter_rows(s, dout, scale ? nullptr : at<uint8_t>(fwd_ws, F.y_perm),
                                            pos, scale ? nullptr : w, dy_perm,
                                            scale ? nullptr : dw, cs),
                        "combine gradient launch")) != MOE_OK)
        return st;
    const void *x_perm;
    if (F.x_perm == MOE_WS_ABSENT) {
        x_perm = at<uint8_t>(ws, L.x_perm);
        st = from_cuda(launch_scatter_rows(s, x, nullptr, pos, scale ? w : nullptr,
                                           at<uint8_t>(ws, L.x_perm), nullptr, cs),
                       "row copy launch");
        if (st != MOE_OK) return st;
    } else {
        x_perm = at<uint8_t>(fwd_ws, F.x_perm);
    }
    if ((st = run_experts_backward(s, {x_perm, at<int32_t>(fwd_ws, F.offsets), W_gate_up, W_down,
                                       at<uint8_t>(fwd_ws, F.h_perm), dy_perm, dx_perm, dW_gate_up,
                                       dW_down, at<uint8_t>(ws, L.experts)}, ds, cs)) != MOE_OK)
        return st;
    if ((st = from_cuda(launch_dispatch_backward(s, dx_perm, pos, scale ? w : nullptr,
                                                 scale ? x : nullptr, dx, scale ? dw : nullptr, cs),
                        "dispatch gradient launch")) != MOE_OK)
        return st;
    return from_cuda(launch_route_backward(s, {x, Wr, at<float>(fwd_ws, F.logits),
                                               at<int32_t>(fwd_ws, F.idx), w, dw, dx,
                                               at<float>(ws, L.dlogits), dWr, dlogit_bias, dx,
                                               at<uint8_t>(ws, L.route)}, ds, cs),
                     "router gradient launch");
}

size_t moe_clip_grad_norm_workspace_size(void) { return clip_scratch_bytes(); }

moe_status_t moe_clip_grad_norm(const moe_grad_t *grads, int64_t n, float max_norm, float *norm,
                                void *ws, size_t ws_bytes, void *stream) {
    set_error_message("");
    if (n < 0 || (n > 0 && !grads)) {
        set_error_message("grads is NULL or n = %lld is negative", (long long)n);
        return MOE_ERR_INVALID_ARG;
    }
    if (!(max_norm >= 0.f)) {
        set_error_message("max_norm %g is not a non-negative number", (double)max_norm);
        return MOE_ERR_INVALID_ARG;
    }
    moe_status_t st;
    if ((st = check_ptrs({ws})) != MOE_OK) return st;
    if (!norm || (reinterpret_cast<uintptr_t>(norm) & 3u)) {
        set_error_message("norm is NULL or not 4-byte aligned");
        return MOE_ERR_INVALID_ARG;
    }
    if ((st = check_ws(ws_bytes, clip_scratch_bytes())) != MOE_OK) return st;
    int64_t units = 0;
    for (int64_t i = 0; i < n; ++i) {
        const moe_grad_t &g = grads[i];
        if (g.dtype != MOE_F32 && g.dtype != MOE_BF16) {
            set_error_message("tensor %lld: unknown dtype %d", (long long)i, g.dtype);
            return MOE_ERR_UNSUPPORTED;
        }
        const uintptr_t mask = g.dtype == MOE_BF16 ? 1u : 3u;
        if (g.numel < 0 || (g.numel > 0 && !g.grad) ||
            ((reinterpret_cast<uintptr_t>(g.grad) | reinterpret_cast<uintptr_t>(g.out)) & mask)) {
            set_error_message("tensor %lld: negative size, NULL or misaligned", (long long)i);
            return MOE_ERR_INVALID_ARG;
        }
        if (g.numel > 0) units += (g.numel - 1) / clip_chunk() + 1;
        if (units > INT32_MAX / 2) {
            set_error_message("the tensors together hold too many elements");
            return MOE_ERR_INVALID_ARG;
        }
    }
    DevStatus ds;
    if ((st = device_status(&ds)) != MOE_OK) return st;
    return from_cuda(launch_clip(grads, n, max_norm, norm, ws, static_cast<cudaStream_t>(stream)),
                     "gradient clipping launch");
}

}  // extern "C"
