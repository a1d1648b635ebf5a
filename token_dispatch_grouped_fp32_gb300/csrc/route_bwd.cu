// route_bwd.cu -- gradient of the router.
//
// With dw the gradient of the chosen experts' weights, S = sum_i w_i dw_i:
//   renormalised weights are a softmax over the chosen logits alone, so
//     dl[idx_j] = w_j (dw_j - S), every other logit's gradient is zero;
//   plain softmax weights: dl[e] = p_e (g_e - S), g_e = dw_j where e = idx_j
//     and 0 elsewhere, p = softmax over all E logits.
//   dWr = dl^T x,   dbias = sum_t dl,   dx = dx_in + dl Wr.
#include "common.cuh"
#include "kernels.h"
#include "simt_gemm.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
using Tl = simt::Tile<64, 64, 16, 4, 4>;

template <bool MAX> __device__ __forceinline__ float warp_all(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    return v;
}

// One warp per token.
__global__ void __launch_bounds__(kThreads)
dlogits_kernel(const float *__restrict__ logits, const int32_t *__restrict__ idx,
               const float *__restrict__ w, const float *__restrict__ dw, int64_t T, int E, int k,
               int renorm, float *__restrict__ dl, DevStatus ds) {
    pdl_entry();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= T) return;
    int e = -1;
    float wj = 0.f, dj = 0.f;
    if (lane < k) {
        e = idx[t * k + lane];
        wj = w[t * k + lane];
        dj = dw[t * k + lane];
        if ((unsigned)e >= (unsigned)E) {
            raise_error(ds, kErrBadRouting);
            e = -1;
            wj = dj = 0.f;
        }
    }
    const float S = warp_all<false>(wj * dj);
    float m = 0.f, inv = 0.f;
    if (!renorm) {
        m = -INFINITY;
        for (int i = lane; i < E; i += 32) m = fmaxf(m, logits[t * E + i]);
        m = warp_all<true>(m);
        float z = 0.f;
        for (int i = lane; i < E; i += 32) z += expf(logits[t * E + i] - m);
        inv = 1.f / warp_all<false>(z);
    }
    for (int i = lane; i < E; i += 32)
        dl[t * E + i] = renorm ? 0.f : expf(logits[t * E + i] - m) * inv * (0.f - S);
    __syncwarp();  // the zeros and unchosen terms above come before the chosen ones
    if (e >= 0) {
        const float p = renorm ? wj : expf(logits[t * E + e] - m) * inv;
        dl[t * E + e] = p * (dj - S);
    }
}

// Partial sums over the tokens of one split: part[split][e][n] with n < d
// dWr's columns and n == d the bias (a column of ones beside x).
template <typename TA>
__global__ void __launch_bounds__(simt::kThreads)
dwr_kernel(const float *__restrict__ dl, const TA *__restrict__ x, int64_t T, int E, int d,
           int tokens, float *__restrict__ part) {
    pdl_entry();
    __shared__ Tl::Smem sm;
    const int n0 = blockIdx.x * Tl::BN, e0 = blockIdx.y * Tl::BM;
    const int64_t t0 = (int64_t)blockIdx.z * tokens;
    const int K = (int)min((int64_t)tokens, T - t0);
    float acc[Tl::TM][Tl::TN];
    Tl::zero(acc);
    Tl::product<false, false>(
        sm, K, [&](int m, int k) { return e0 + m < E ? dl[(t0 + k) * E + e0 + m] : 0.f; },
        [&](int k, int n) {
            return n0 + n < d ? Act<TA>::to_f(x[(t0 + k) * d + n0 + n]) : n0 + n == d ? 1.f : 0.f;
        }, acc);
#pragma unroll
    for (int i = 0; i < Tl::TM; ++i)
#pragma unroll
        for (int j = 0; j < Tl::TN; ++j) {
            const int e = e0 + Tl::row(i), n = n0 + Tl::col(j);
            if (e < E && n <= d)
                part[((int64_t)blockIdx.z * E + e) * (d + 1) + n] = acc[i][j];
        }
}

__global__ void __launch_bounds__(kThreads)
dwr_sum_kernel(const float *__restrict__ part, int splits, int E, int d, float *__restrict__ dWr,
               float *__restrict__ dbias) {
    pdl_entry();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, n = (int64_t)E * (d + 1);
    if (i >= n) return;
    float s = 0.f;
    for (int z = 0; z < splits; ++z) s += part[z * n + i];
    const int64_t e = i / (d + 1), c = i % (d + 1);
    if (c < d) dWr[e * d + c] = s;
    else if (dbias) dbias[e] = s;
}

template <typename TA>
__global__ void __launch_bounds__(simt::kThreads)
route_dx_kernel(const float *__restrict__ dl, const float *__restrict__ Wr, const TA *dx_in,
                int64_t T, int E, int d, TA *dx) {
    pdl_entry();
    __shared__ Tl::Smem sm;
    const int64_t t0 = (int64_t)blockIdx.x * Tl::BM;
    const int n0 = blockIdx.y * Tl::BN;
    float acc[Tl::TM][Tl::TN];
    Tl::zero(acc);
    Tl::product<true, false>(
        sm, E, [&](int m, int k) { return t0 + m < T ? dl[(t0 + m) * E + k] : 0.f; },
        [&](int k, int n) { return n0 + n < d ? Wr[(int64_t)k * d + n0 + n] : 0.f; }, acc);
#pragma unroll
    for (int i = 0; i < Tl::TM; ++i)
#pragma unroll
        for (int j = 0; j < Tl::TN; ++j) {
            const int64_t t = t0 + Tl::row(i);
            const int n = n0 + Tl::col(j);
            if (t >= T || n >= d) continue;
            float v = acc[i][j];
            if (dx_in) v += Act<TA>::to_f(dx_in[t * d + n]);
            dx[t * d + n] = Act<TA>::from_f(v);
        }
}

struct Plan {
    int splits, tokens;  // splits of the token axis in dWr's sum
};
Plan plan(const Shape &s) {
    const int64_t tiles = (int64_t)((s.E + 63) / 64) * ((s.d + 64) / 64);
    int64_t want = (2 * 152 + tiles - 1) / tiles;
    const int64_t most = (s.T + 63) / 64;
    want = want < 1 ? 1 : want > most ? most : want;
    Plan p;
    p.tokens = (int)((s.T + want - 1) / want);
    p.splits = (int)((s.T + p.tokens - 1) / p.tokens);
    return p;
}

template <typename TA>
cudaError_t launch_t(const Shape &s, const RouteBwd &a, const DevStatus &ds, cudaStream_t st) {
    const Plan p = plan(s);
    float *part = static_cast<float *>(a.ws);
    launch_pdl(dlogits_kernel, dim3((unsigned)((s.T + kWarps - 1) / kWarps)), dim3(kThreads), 0, st,
               a.logits, a.idx, a.w, a.dw, s.T, s.E, s.k, s.renorm ? 1 : 0, a.dlogits, ds);
    launch_pdl(dwr_kernel<TA>, dim3((s.d + 64) / 64, (s.E + 63) / 64, p.splits), dim3(simt::kThreads),
               0, st, (const float *)a.dlogits, static_cast<const TA *>(a.x), s.T, s.E, s.d,
               p.tokens, part);
    launch_pdl(dwr_sum_kernel, dim3((unsigned)(((int64_t)s.E * (s.d + 1) + kThreads - 1) / kThreads)),
               dim3(kThreads), 0, st, (const float *)part, p.splits, s.E, s.d, a.dWr, a.dbias);
    launch_pdl(route_dx_kernel<TA>, dim3((unsigned)((s.T + 63) / 64), (s.d + 63) / 64),
               dim3(simt::kThreads), 0, st, (const float *)a.dlogits, a.Wr,
               static_cast<const TA *>(a.dx_in), s.T, s.E, s.d, static_cast<TA *>(a.dx));
    return cudaGetLastError();
}

}  // namespace

size_t route_backward_scratch_bytes(const Shape &s) {
    return 4 * (size_t)plan(s).splits * s.E * (s.d + 1);
}

cudaError_t launch_route_backward(const Shape &s, const RouteBwd &a, const DevStatus &ds,
                                  cudaStream_t st) {
    return s.bf16 ? launch_t<__nv_bfloat16>(s, a, ds, st) : launch_t<float>(s, a, ds, st);
}

}  // namespace moe
