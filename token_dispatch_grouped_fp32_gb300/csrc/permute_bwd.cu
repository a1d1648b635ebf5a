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

// Both kernels: a group of TPT threads (a warp or the block) per token, each
// thread holding U 16-byte vectors of the token's row, TPT apart; SG slots'
// rows are loaded at once.  Rows of more than TPT*U vectors are walked in
// chunks.  The token's own row is read once, whatever k, and a slot's dot
// product is summed over each warp, then over the group's warps in order.
// Bound by HBM: T = d = 4096, k = 2, bf16 (168 MB) 27.2 us, 0.91 of the copy
// rate.  A warp per pair, which reads the token's row k times, took 28.2; for
// the weighted sum a warp per token with the slots one after another 12.7 us
// at T = 777, d = 1000, k = 4 in fp32, where the group takes 4.1.
constexpr int kThreads = 128;
constexpr int kMaxK = 32;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Per-warp sums of the slots' dot products.
struct Dots {
    float s[kThreads / 32][kMaxK];
};
__device__ __forceinline__ void dots_clear(Dots &d) { d.s[threadIdx.x >> 5][threadIdx.x & 31] = 0.f; }
__device__ __forceinline__ void dots_add(Dots &d, int j, float part) {
    part = warp_sum(part);
    if ((threadIdx.x & 31) == 0) d.s[threadIdx.x >> 5][j] += part;
}
// dw[j] of the group's token, by its thread j (all threads of the group call).
template <int TPT> __device__ __forceinline__ void dots_store(const Dots &d, int k, float *dw) {
    if (TPT == 32) __syncwarp();
    else __syncthreads();
    const int j = threadIdx.x % TPT, w0 = threadIdx.x / TPT * (TPT / 32);
    if (j >= k) return;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < TPT / 32; ++w) s += d.s[w0 + w][j];
    dw[j] = s;
}

// dst[pos] = w * src row of every slot; DOT: dw = <src row, y_perm[pos]>.
template <typename TA, int TPT, int U, int SG, bool DOT>
__global__ void __launch_bounds__(kThreads)
scatter_rows_kernel(const TA *__restrict__ src, const TA *__restrict__ y_perm,
                    const int32_t *__restrict__ pos, const float *__restrict__ w, int64_t T, int k,
                    int d, TA *__restrict__ dst, float *__restrict__ dw) {
    pdl_wait();
    constexpr int EPV = 16 / sizeof(TA);
    __shared__ Dots dots;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / TPT) + threadIdx.x / TPT;
    const int nvec = d / EPV;
    if (DOT) {
        dots_clear(dots);
        __syncwarp();
    }
    if (t >= T) return;  // whole groups; TPT = block: the block
    for (int v0 = threadIdx.x % TPT; v0 - (int)(threadIdx.x % TPT) < nvec; v0 += TPT * U) {
        uint4 g[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v0 + u * TPT < nvec) g[u] = ldg16(src + t * d + (int64_t)(v0 + u * TPT) * EPV);
        for (int j0 = 0; j0 < k; j0 += SG) {
            int row[SG];
            float wj[SG];
            uint4 y[SG][U];
#pragma unroll
            for (int s = 0; s < SG; ++s) {
                row[s] = j0 + s < k ? __ldg(pos + t * k + j0 + s) : -1;
                wj[s] = w && j0 + s < k ? __ldg(w + t * k + j0 + s) : 1.f;
            }
            if (DOT)
#pragma unroll
                for (int s = 0; s < SG; ++s)
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (row[s] >= 0 && v0 + u * TPT < nvec)
                            y[s][u] = ldg16(y_perm + (int64_t)row[s] * d + (int64_t)(v0 + u * TPT) * EPV);
#pragma unroll
            for (int s = 0; s < SG; ++s) {
                if (row[s] < 0) continue;  // the same for the whole group
                float part = 0.f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (v0 + u * TPT >= nvec) continue;
                    float a[EPV], b[EPV];
                    unpack16(g[u], a, static_cast<const TA *>(nullptr));
                    if (DOT) {
                        unpack16(y[s][u], b, static_cast<const TA *>(nullptr));
#pragma unroll
                        for (int i = 0; i < EPV; ++i) part = fmaf(a[i], b[i], part);
                    }
#pragma unroll
                    for (int i = 0; i < EPV; ++i) a[i] *= wj[s];
                    stg16(dst + (int64_t)row[s] * d + (int64_t)(v0 + u * TPT) * EPV,
                          pack16(a, static_cast<const TA *>(nullptr)));
                }
                if (DOT) dots_add(dots, j0 + s, part);
            }
        }
    }
    if (DOT) dots_store<TPT>(dots, k, dw + t * k);
}

// dx = the sum of w * row over a token's slots; DOT: dw = <x row, row>, else x
// (if given) is added to dx.
template <typename TA, int TPT, int U, int SG, bool DOT>
__global__ void __launch_bounds__(kThreads)
gather_rows_scaled_kernel(const TA *__restrict__ dx_perm, const int32_t *__restrict__ pos,
                          const float *__restrict__ w, const TA *x, int64_t T, int k, int d, TA *dx,
                          float *__restrict__ dw) {
    pdl_wait();
    constexpr int EPV = 16 / sizeof(TA);
    __shared__ Dots dots;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / TPT) + threadIdx.x / TPT;
    const int nvec = d / EPV;
    if (DOT) {
        dots_clear(dots);
        __syncwarp();
    }
    if (t >= T) return;  // whole groups; TPT = block: the block
    for (int v0 = threadIdx.x % TPT; v0 - (int)(threadIdx.x % TPT) < nvec; v0 += TPT * U) {
        uint4 xv[U];
        float acc[U][EPV];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if ((DOT || x) && v0 + u * TPT < nvec)
                xv[u] = *reinterpret_cast<const uint4 *>(x + t * d + (int64_t)(v0 + u * TPT) * EPV);
#pragma unroll
            for (int i = 0; i < EPV; ++i) acc[u][i] = 0.f;
        }
        for (int j0 = 0; j0 < k; j0 += SG) {
            int row[SG];
            float wj[SG];
            uint4 r[SG][U];
#pragma unroll
            for (int s = 0; s < SG; ++s) {
                row[s] = j0 + s < k ? __ldg(pos + t * k + j0 + s) : -1;
                wj[s] = j0 + s < k ? __ldg(w + t * k + j0 + s) : 0.f;
            }
#pragma unroll
            for (int s = 0; s < SG; ++s)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (row[s] >= 0 && v0 + u * TPT < nvec)
                        r[s][u] = ldg16(dx_perm + (int64_t)row[s] * d + (int64_t)(v0 + u * TPT) * EPV);
#pragma unroll
            for (int s = 0; s < SG; ++s) {
                if (row[s] < 0) continue;  // the same for the whole group
                float part = 0.f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (v0 + u * TPT >= nvec) continue;
                    float a[EPV], b[EPV];
                    unpack16(r[s][u], b, static_cast<const TA *>(nullptr));
                    if (DOT) {
                        unpack16(xv[u], a, static_cast<const TA *>(nullptr));
#pragma unroll
                        for (int i = 0; i < EPV; ++i) part = fmaf(a[i], b[i], part);
                    }
#pragma unroll
                    for (int i = 0; i < EPV; ++i) acc[u][i] = fmaf(wj[s], b[i], acc[u][i]);
                }
                if (DOT) dots_add(dots, j0 + s, part);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (v0 + u * TPT >= nvec) continue;
            if (!DOT && x) {
                float a[EPV];
                unpack16(xv[u], a, static_cast<const TA *>(nullptr));
#pragma unroll
                for (int i = 0; i < EPV; ++i) acc[u][i] += a[i];
            }
            stg16(dx + t * d + (int64_t)(v0 + u * TPT) * EPV,
                  pack16(acc[u], static_cast<const TA *>(nullptr)));
        }
    }
    if (DOT) dots_store<TPT>(dots, k, dw + t * k);
}

unsigned blocks(int64_t T, int tpt) {
    const int per = kThreads / tpt;
    return (unsigned)((T + per - 1) / per);
}

template <typename TA, int TPT, int U, int SG>
cudaError_t launch_scatter_v(const Shape &s, const void *src, const void *y_perm,
                             const int32_t *pos, const float *w, void *dst, float *dw,
                             cudaStream_t st) {
    const TA *x = static_cast<const TA *>(src), *y = static_cast<const TA *>(y_perm);
    TA *o = static_cast<TA *>(dst);
    const dim3 grid(blocks(s.T, TPT));
    if (dw)
        launch_pdl(scatter_rows_kernel<TA, TPT, U, SG, true>, grid, dim3(kThreads), 0, st, x, y, pos,
                   w, s.T, s.k, s.d, o, dw);
    else
        launch_pdl(scatter_rows_kernel<TA, TPT, U, SG, false>, grid, dim3(kThreads), 0, st, x, y, pos,
                   w, s.T, s.k, s.d, o, dw);
    return cudaGetLastError();
}

template <typename TA, int TPT, int U, int SG>
cudaError_t launch_gather_v(const Shape &s, const void *dx_perm, const int32_t *pos,
                            const float *w, const void *x, void *dx, float *dw, cudaStream_t st) {
    const dim3 grid(blocks(s.T, TPT));
    const TA *r = static_cast<const TA *>(dx_perm), *xs = static_cast<const TA *>(x);
    TA *o = static_cast<TA *>(dx);
    if (dw)
        launch_pdl(gather_rows_scaled_kernel<TA, TPT, U, SG, true>, grid, dim3(kThreads), 0, st, r, pos,
                   w, xs, s.T, s.k, s.d, o, dw);
    else
        launch_pdl(gather_rows_scaled_kernel<TA, TPT, U, SG, false>, grid, dim3(kThreads), 0, st, r, pos,
                   w, xs, s.T, s.k, s.d, o, dw);
    return cudaGetLastError();
}

// Short rows: a warp per token; else a block, with as many vectors a thread
// as the row needs (up to 4: then 2 slots at a time keep the registers).
template <typename TA, typename... Args>
cudaError_t launch_scatter_t(const Shape &s, Args... args) {
    const int nvec = s.d / (16 / (int)sizeof(TA));
    if (nvec <= 32) return launch_scatter_v<TA, 32, 1, 4>(s, args...);
    if (nvec <= 128) return launch_scatter_v<TA, 128, 1, 4>(s, args...);
    if (nvec <= 256) return launch_scatter_v<TA, 128, 2, 4>(s, args...);
    return launch_scatter_v<TA, 128, 4, 2>(s, args...);
}
template <typename TA, typename... Args>
cudaError_t launch_gather_t(const Shape &s, Args... args) {
    const int nvec = s.d / (16 / (int)sizeof(TA));
    if (nvec <= 32) return launch_gather_v<TA, 32, 1, 4>(s, args...);
    if (nvec <= 128) return launch_gather_v<TA, 128, 1, 4>(s, args...);
    if (nvec <= 256) return launch_gather_v<TA, 128, 2, 4>(s, args...);
    return launch_gather_v<TA, 128, 4, 2>(s, args...);
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

cudaError_t launch_gather_sum_f32(const Shape &s, const float *rows, const int32_t *idx,
                                  const float *w, const float *add, float *out, cudaStream_t st) {
    return launch_gather_t<float>(s, (const void *)rows, idx, w, (const void *)add, (void *)out,
                                  (float *)nullptr, st);
}

}  // namespace moe
