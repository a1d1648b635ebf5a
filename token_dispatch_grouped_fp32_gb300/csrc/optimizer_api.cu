// optimizer_api.cu -- the C ABI of AdamW and of the balance bias's update
// (declared in include/moe.h): argument checks and launches.
#include <cfloat>
#include <cmath>

#include "api.h"

namespace moe {
namespace {

bool aligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

moe_status_t invalid(const char *what) {
    set_error_message("%s", what);
    return MOE_ERR_INVALID_ARG;
}

moe_status_t check_hyper(const moe_adamw_hyper_t *h) {
    if (!h) return invalid("hyper is NULL");
    // (as floats: finite, and eps no subnormal, which a reciprocal takes for 0)
    const float lr = (float)h->lr, eps = (float)h->eps;
    if (!(lr >= 0.f) || !(eps == 0.f || eps >= FLT_MIN) || !std::isfinite(lr) || !std::isfinite(eps) ||
        (eps == 0.f && h->eps != 0.0) ||
        !(h->beta1 >= 0.0 && h->beta1 < 1.0) || !(h->beta2 >= 0.0 && h->beta2 < 1.0)) {
        set_error_message("lr %g, beta1 %g, beta2 %g or eps %g out of range", h->lr, h->beta1, h->beta2,
                          h->eps);
        return MOE_ERR_INVALID_ARG;
    }
    if (h->step < 1) return invalid("the step is counted from 1");
    return MOE_OK;
}

moe_adamw_scalars_t scalars_of(const moe_adamw_hyper_t &h) {
    moe_adamw_scalars_t s = {};
    s.lr = (float)h.lr;
    s.step_size = (float)(h.lr / (1.0 - std::pow(h.beta1, (double)h.step)));
    s.inv_sqrt_bc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(h.beta2, (double)h.step)));
    s.seed_lo = (uint32_t)h.seed;
    s.seed_hi = (uint32_t)(h.seed >> 32);
    return s;
}

moe_status_t check_tensor(const moe_adamw_tensor_t &t, long long i) {
    const bool small = t.state_dtype == MOE_E4M3;
    if ((t.param_dtype != MOE_F32 && t.param_dtype != MOE_BF16) ||
        (t.grad_dtype != MOE_F32 && t.grad_dtype != MOE_BF16) ||
        (t.state_dtype != MOE_F32 && !small)) {
        set_error_message("tensor %lld: unsupported dtypes (parameter %d, gradient %d, states %d)", i,
                          t.param_dtype, t.grad_dtype, t.state_dtype);
        return MOE_ERR_UNSUPPORTED;
    }
    if (t.numel < 0 || !std::isfinite(t.weight_decay)) {
        set_error_message("tensor %lld: negative size or a weight decay that is not finite", i);
        return MOE_ERR_INVALID_ARG;
    }
    if (t.master && t.param_dtype != MOE_BF16) {
        set_error_message("tensor %lld: a master copy beside an fp32 parameter", i);
        return MOE_ERR_INVALID_ARG;
    }
    if (!small && (t.exp_avg_scale || t.exp_avg_sq_scale)) {
        set_error_message("tensor %lld: scales beside fp32 states", i);
        return MOE_ERR_INVALID_ARG;
    }
    if (t.numel == 0) return MOE_OK;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq ||
        (small && (!t.exp_avg_scale || !t.exp_avg_sq_scale)) ||
        !aligned(t.param, t.param_dtype == MOE_BF16 ? 2 : 4) ||
        !aligned(t.grad, t.grad_dtype == MOE_BF16 ? 2 : 4) || !aligned(t.master, 4) ||
        !aligned(t.exp_avg_scale, 4) || !aligned(t.exp_avg_sq_scale, 4) ||
        (!small && (!aligned(t.exp_avg, 4) || !aligned(t.exp_avg_sq, 4)))) {
        set_error_message("tensor %lld: a NULL or misaligned pointer", i);
        return MOE_ERR_INVALID_ARG;
    }
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_adamw_scalars(const moe_adamw_hyper_t *hyper, moe_adamw_scalars_t *out) {
    set_error_message("");
    const moe_status_t st = check_hyper(hyper);
    if (st != MOE_OK) return st;
    if (!out) return invalid("out is NULL");
    *out = scalars_of(*hyper);
    return MOE_OK;
}

moe_status_t moe_adamw_step(const moe_adamw_tensor_t *tensors, int64_t n,
                            const moe_adamw_hyper_t *hyper, const float *norm,
                            const moe_adamw_scalars_t *scalars, void *stream) {
    set_error_message("");
    if (n < 0 || (n > 0 && !tensors)) {
        set_error_message("tensors is NULL or n = %lld is negative", (long long)n);
        return MOE_ERR_INVALID_ARG;
    }
    moe_status_t st = check_hyper(hyper);
    if (st != MOE_OK) return st;
    if (!aligned(norm, 4) || !aligned(scalars, 16)) return invalid("norm or scalars is misaligned");
    if (norm && !(hyper->max_norm >= 0.f)) {
        set_error_message("max_norm %g is not a non-negative number", (double)hyper->max_norm);
        return MOE_ERR_INVALID_ARG;
    }
    int64_t units = 0;
    for (int64_t i = 0; i < n; ++i) {
        if ((st = check_tensor(tensors[i], (long long)i)) != MOE_OK) return st;
        if (tensors[i].numel > 0) units += (tensors[i].numel - 1) / adamw_chunk() + 1;
        if (units > INT32_MAX / 2) return invalid("the tensors together hold too many elements");
    }
    DevStatus ds;
    if ((st = device_status(&ds)) != MOE_OK) return st;
    return from_cuda(launch_adamw(tensors, n, scalars_of(*hyper), scalars, *hyper, norm,
                                  static_cast<cudaStream_t>(stream)),
                     "AdamW launch");
}

moe_status_t moe_update_balance_bias(const int32_t *counts, int64_t layers, int32_t E, float rate,
                                     float *balance_bias, float *imbalance, void *stream) {
    set_error_message("");
    if (layers < 0 || E < 1 || !std::isfinite(rate)) {
        set_error_message("bad sizes: layers=%lld E=%d, or a rate that is not finite",
                          (long long)layers, E);
        return MOE_ERR_INVALID_ARG;
    }
    if (E > 1024 || layers > INT32_MAX) {
        set_error_message("unsupported E=%d layers=%lld (E <= 1024, layers < 2^31)", E,
                          (long long)layers);
        return MOE_ERR_UNSUPPORTED;
    }
    if (layers == 0) return MOE_OK;
    if (!counts || !balance_bias || !aligned(counts, 4) || !aligned(balance_bias, 4) ||
        !aligned(imbalance, 4))
        return invalid("counts or balance_bias is NULL, or a pointer is misaligned");
    DevStatus ds;
    const moe_status_t st = device_status(&ds);
    if (st != MOE_OK) return st;
    return from_cuda(launch_balance(counts, layers, E, rate, balance_bias, imbalance,
                                    static_cast<cudaStream_t>(stream)),
                     "balance bias launch");
}

}  // extern "C"
