// api.h -- what the C ABI's translation units share: argument checks, the
// device's state and the layout of moe_forward's workspace (internal to the
// library; defined in moe_api.cu).
#pragma once

#include <initializer_list>

#include "moe.h"
#include "common.cuh"
#include "kernels.h"

namespace moe {

// Architecture check and error word of the current device (cached).
moe_status_t device_status(DevStatus *out);

bool aligned16(const void *p);
// Sizes and types of `cfg`, checked, as a Shape.
moe_status_t check_cfg(const moe_config_t *cfg, Shape *s);
// Every pointer given and 16-byte aligned.
moe_status_t check_ptrs(std::initializer_list<const void *> ptrs);
moe_status_t from_cuda(cudaError_t e, const char *what);

// moe_forward's workspace: offsets of its 256-byte aligned sub-buffers.
struct WsLayout {
    size_t logits, idx, w, counts, offsets, pos, src, hist, route, row_scale, x_perm, h_perm,
        y_perm, total;
};
WsLayout ws_layout(const Shape &s);

inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

template <typename T> T *at(void *ws, size_t off) {
    return reinterpret_cast<T *>(static_cast<uint8_t *>(ws) + off);
}
template <typename T> const T *at(const void *ws, size_t off) {
    return reinterpret_cast<const T *>(static_cast<const uint8_t *>(ws) + off);
}

}  // namespace moe
