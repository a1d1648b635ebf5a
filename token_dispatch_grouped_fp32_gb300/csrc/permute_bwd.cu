// permute_bwd.cu -- gradients of the two permutations of the layer: the
// weighted combine and the token dispatch.
//
// With q = t*k + j the pair of token t's slot j, r = pos[q] its row:
//   combine   out[t] = sum_j w[q] y_perm[r]
//             dy_perm[r] = w[q] dout[t],   dw[q] = <dout[t], y_perm[r]>
//   dispatch  x_perm[r] = (w[q]) x[t]
//             dx[t] = sum_j (w[q]) dx_perm[r],   dw[q] = <x[t], dx_perm[r]>
// All sums are fp32 in a fixed order, rounded once to the act dtype.  A pair
// that the dispatch dropped (pos -1) has no row and a zero weight gradient.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One warp per pair: the token's row of dout times the pair's weight, to the
// pair's row; DOT: its dot product with the row of y_perm on the way.
template <typename TA, bool DOT>
__global__ void __launch_bounds__(kThreads)
scatter_rows_kernel(const TA *__restrict__ src, const TA *__restrict__ y_perm,
                    const int32_t *__restrict__ pos, const float *__restrict__ w, int64_t P, int k,
                    int d, TA *__restrict__ dst, float *__restrict__ dw) {
    pdl_entry();
    constexpr int EPV = 16 / sizeof(TA);
    const int lane = threadIdx.x & 31;
    const int64_t q = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (q >= P) return;
    const int row = pos[q];
    if (row < 0) {
        if (DOT && lane == 0) dw[q] = 0.f;
        return;
    }
    const TA *s = src + q / k * d;
    const float wq = w ? w[q] : 1.f;
    float dot = 0.f;
    for (int v = lane; v < d / EPV; v += 32) {
        float g[EPV], y[EPV];
        unpack16(ldg16(s + (int64_t)v * EPV), g, static_cast<const TA *>(nullptr));
        if (DOT) {
            unpack16(ldg16(y_perm + (int64_t)row * d + (int64_t)v * EPV), y,
                     static_cast<const TA *>(nullptr));
#pragma unroll
            for (int i = 0; i < EPV; ++i) dot = fmaf(g[i], y[i], dot);
        }
#pragma unroll
        for (int i = 0; i < EPV; ++i) g[i] *= wq;
        stg16(dst + (int64_t)row * d + (int64_t)v * EPV, pack16(g, static_cast<const TA *>(nullptr)));
    }
    if (DOT) {
        dot = warp_sum(dot);
        if (lane == 0) dw[q] = dot;
    }
}

// One warp per token: the weighted sum of its rows of dx_perm, and each
// row's dot product with the token's row of x (the partial of slot j is
// summed over the warp per chunk and kept by lane j).
template <typename TA>
__global__ void __launch_bounds__(kThreads)
gather_rows_scaled_kernel(const TA *__restrict__ dx_perm, const int32_t *__restrict__ pos,
                          const float *__restrict__ w, const TA *__restrict__ x, int64_t T, int k,
                          int d, TA *__restrict__ dx, float *__restrict__ dw) {
    pdl_entry();
    constexpr int EPV = 16 / sizeof(TA);
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= T) return;
    int my_pos = -1;
    float my_w = 0.f, my_dot = 0.f;
    if (lane < k) {
        my_pos = pos[t * k + lane];
        my_w = w[t * k + lane];
    }
    const int nvec = d / EPV;
    for (int v0 = 0; v0 < nvec; v0 += 32) {
        const int v = v0 + lane;
        float acc[EPV], xv[EPV];
#pragma unroll
        for (int i = 0; i < EPV; ++i) acc[i] = xv[i] = 0.f;
        if (v < nvec)
            unpack16(ldg16(x + t * d + (int64_t)v * EPV), xv, static_cast<const TA *>(nullptr));
        for (int j = 0; j < k; ++j) {
            const int row = __shfl_sync(0xffffffffu, my_pos, j);
            const float wj = __shfl_sync(0xffffffffu, my_w, j);
            if (row < 0) continue;  // warp-uniform
            float part = 0.f;
            if (v < nvec) {
                float r[EPV];
                unpack16(ldg16(dx_perm + (int64_t)row * d + (int64_t)v * EPV), r,
                         static_cast<const TA *>(nullptr));
#pragma unroll
                for (int i = 0; i < EPV; ++i) {
                    acc[i] = fmaf(wj, r[i], acc[i]);
                    part = fmaf(xv[i], r[i], part);
                }
            }
            part = warp_sum(part);
            if (lane == j) my_dot += part;
        }
        if (v < nvec)
            stg16(dx + t * d + (int64_t)v * EPV, pack16(acc, static_cast<const TA *>(nullptr)));
    }
    if (lane < k) dw[t * k + lane] = my_dot;
}

template <typename TA>
cudaError_t launch_scatter_t(const Shape &s, const void *src, const void *y_perm,
                             const int32_t *pos, const float *w, void *dst, float *dw,
                             cudaStream_t st) {
    const dim3 grid((unsigned)((s.P() + kWarps - 1) / kWarps));
    const TA *x = static_cast<const TA *>(src), *y = static_cast<const TA *>(y_perm);
    TA *o = static_cast<TA *>(dst);
    if (dw)
        launch_pdl(scatter_rows_kernel<TA, true>, grid, dim3(kThreads), 0, st, x, y, pos, w, s.P(),
                   s.k, s.d, o, dw);
    else
        launch_pdl(scatter_rows_kernel<TA, false>, grid, dim3(kThreads), 0, st, x, y, pos, w,
                   s.P(), s.k, s.d, o, dw);
    return cudaGetLastError();
}

template <typename TA>
cudaError_t launch_gather_t(const Shape &s, const void *dx_perm, const int32_t *pos,
                            const float *w, const void *x, void *dx, float *dw, cudaStream_t st) {
    launch_pdl(gather_rows_scaled_kernel<TA>, dim3((unsigned)((s.T + kWarps - 1) / kWarps)),
               dim3(kThreads), 0, st, static_cast<const TA *>(dx_perm), pos, w,
               static_cast<const TA *>(x), s.T, s.k, s.d, static_cast<TA *>(dx), dw);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scatter_rows(const Shape &s, const void *src, const void *y_perm,
                                const int32_t *pos, const float *w, void *dst, float *dw,
                                cudaStream_t st) {
    return s.bf16 ? launch_scatter_t<__nv_bfloat16>(s, src, y_perm, pos, w, dst, dw, st)
                  : launch_scatter_t<float>(s, src, y_perm, pos, w, dst, dw, st);
}

cudaError_t launch_dispatch_backward(const Shape &s, const void *dx_perm, const int32_t *pos,
                                     const float *w, const void *x, void *dx, float *dw,
                                     cudaStream_t st) {
    if (!w) return launch_combine(s, dx_perm, pos, nullptr, dx, st);
    return s.bf16 ? launch_gather_t<__nv_bfloat16>(s, dx_perm, pos, w, x, dx, dw, st)
                  : launch_gather_t<float>(s, dx_perm, pos, w, x, dx, dw, st);
}

}  // namespace moe
