// route_scored_grad.cu -- the gradient of a scored router's weights with respect to the
// logits, and the balance bias's update.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp2_fast(float x) {  // 2 ulp
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ------------------------- gradient to the logits --------------------------
//   softmax, renormalised:  dl[idx_j] = w_j (d_j - S/c)
//   softmax:                dl[e]     = s_e (c g_e - S),  g_e = d_j where e = idx_j
//   sigmoid, renormalised:  dl[idx_j] = w_j (d_j - S/c) (1 - s_j)
//   sigmoid:                dl[idx_j] = w_j d_j (1 - s_j)
// with S = sum_j w_j d_j.  LANES lanes per token: its row's chosen entries in shared
// memory, zero elsewhere, then written whole, W columns a lane at a time (four where
// E allows it).  The fewer lanes a token, the fewer steps its sums take: with eight
// columns a lane, 16 lanes for E = 128, T = 131072 (softmax, all logits) takes 21.7 us
// against 34.7 with 32 lanes, the time of its bytes at the copy rate.
constexpr int kGradThreads = 256;

struct GradArgs {
    const float *logits;
    const int32_t *idx;
    const float *w, *dw;
    int64_t T;
    int E, k;
    ScoreGrad f;
    float *dl;
};

template <int LANES> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

template <int W> struct Columns;
template <> struct Columns<4> { using V = float4; };
template <> struct Columns<1> { using V = float; };

// DENSE: softmax that is not renormalised, N times W columns a lane
template <bool DENSE, int W, int LANES, int N>
__global__ void __launch_bounds__(kGradThreads)
logits_grad_kernel(const GradArgs a, DevStatus ds) {
    pdl_wait();
    using V = typename Columns<W>::V;
    extern __shared__ __align__(16) float rows[];
    const int E = a.E, l = threadIdx.x % LANES, own = threadIdx.x / LANES;
    const int stride = (E + 3) & ~3;
    const int64_t t = (int64_t)blockIdx.x * (kGradThreads / LANES) + own;
    const bool there = t < a.T;
    float *row = rows + own * stride;
    for (int c = W * l; c < E; c += W * LANES)
#pragma unroll
        for (int i = 0; i < W; ++i) row[c + i] = 0.f;
    const float *L = a.logits + t * E;
    float *o = a.dl + t * E;
    // the logits first: nothing waits for them but the last sums
    float v[N][W];
    if constexpr (DENSE) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = (l + LANES * n) * W;
            if (there && c < E) {
                *reinterpret_cast<V *>(v[n]) = *reinterpret_cast<const V *>(L + c);
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i) v[n][i] = -INFINITY;
            }
        }
    }
    float S = 0.f;
    int e[32 / LANES];  // this lane's slots l, l + LANES, ...
    float wj[32 / LANES], dj[32 / LANES];
#pragma unroll
    for (int q = 0; q < 32 / LANES; ++q) {
        const int j = l + LANES * q;
        e[q] = -1;
        wj[q] = dj[q] = 0.f;
        if (there && j < a.k) {
            e[q] = a.idx[t * a.k + j];
            wj[q] = a.w[t * a.k + j];
            dj[q] = a.dw[t * a.k + j];
            if ((unsigned)e[q] >= (unsigned)E) {
                raise_error(ds, kErrBadRouting);
                e[q] = -1;
                wj[q] = dj[q] = 0.f;
            }
        }
        S += wj[q] * dj[q];
    }
    S = lanes_sum<LANES>(S);
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 32 / LANES; ++q)
        if (e[q] >= 0)
            row[e[q]] = DENSE ? a.f.scale * dj[q]
                              : a.f.chosen(wj[q], dj[q], S, a.f.sigmoid ? L[e[q]] : 0.f);
    __syncwarp();
    if constexpr (!DENSE) {
        if (there)
            for (int c = W * l; c < E; c += W * LANES)
                *reinterpret_cast<V *>(o + c) = *reinterpret_cast<const V *>(row + c);
    } else {
        float m = -INFINITY, z = 0.f;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < W; ++i) m = fmaxf(m, v[n][i]);
#pragma unroll
        for (int q = LANES / 2; q >= 1; q >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, q));
        if (m == -INFINITY) m = 0.f;  // all masked: exponentials of 0, and no scores
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < W; ++i) {
                v[n][i] = exp2_fast((v[n][i] - m) * kLog2e);
                z += v[n][i];
            }
        z = lanes_sum<LANES>(z);
        const float inv = z > 0.f || isnan(z) ? 1.f / z : 0.f;
        if (!there) return;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = (l + LANES * n) * W;
            if (c >= E) continue;
            float g[W];
            *reinterpret_cast<V *>(g) = *reinterpret_cast<const V *>(row + c);
#pragma unroll
            for (int i = 0; i < W; ++i) g[i] = v[n][i] * inv * (g[i] - S);
            *reinterpret_cast<V *>(o + c) = *reinterpret_cast<const V *>(g);
        }
    }
}

template <bool DENSE, int W, int LANES, int N>
cudaError_t launch_grad(const GradArgs &a, const DevStatus &ds, cudaStream_t st) {
    constexpr int kTokens = kGradThreads / LANES;
    const dim3 grid((unsigned)((a.T + kTokens - 1) / kTokens));
    const size_t smem = sizeof(float) * kTokens * (size_t)((a.E + 3) & ~3);
    return launch_pdl(logits_grad_kernel<DENSE, W, LANES, N>, grid, dim3(kGradThreads), smem, st, a, ds);
}

template <bool DENSE> cudaError_t launch_grad_any(const GradArgs &a, const DevStatus &ds, cudaStream_t st) {
    if (a.E % 4 == 0) {  // two float4 a lane, and from E = 257 on more
        if (a.E <= 64) return launch_grad<DENSE, 4, 8, 2>(a, ds, st);
        if (a.E <= 128) return launch_grad<DENSE, 4, 16, 2>(a, ds, st);
        if (a.E <= 256 || !DENSE) return launch_grad<DENSE, 4, 32, 2>(a, ds, st);
        if (a.E <= 512) return launch_grad<DENSE, 4, 32, 4>(a, ds, st);
        return launch_grad<DENSE, 4, 32, 8>(a, ds, st);
    }
    if (a.E <= 64) return launch_grad<DENSE, 1, 8, 8>(a, ds, st);
    if (a.E <= 128) return launch_grad<DENSE, 1, 16, 8>(a, ds, st);
    if (a.E <= 256 || !DENSE) return launch_grad<DENSE, 1, 32, 8>(a, ds, st);
    if (a.E <= 512) return launch_grad<DENSE, 1, 32, 16>(a, ds, st);
    return launch_grad<DENSE, 1, 32, 32>(a, ds, st);
}

// ------------------------------ balance bias -------------------------------
//   b_e += rate * sign(sum_i n_i - E n_e),  imbalance = E max n / sum n
// A block per layer; whole numbers are compared, so that an expert at the mean
// keeps its bias.
constexpr int kBalanceThreads = 256;

__global__ void __launch_bounds__(kBalanceThreads)
balance_kernel(const int32_t *__restrict__ counts, int E, float rate, float *__restrict__ bias,
               float *__restrict__ imbalance) {
    pdl_wait();
    __shared__ long long s_sum[kBalanceThreads / 32];
    __shared__ int s_max[kBalanceThreads / 32];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int32_t *n = counts + (int64_t)blockIdx.x * E;
    float *b = bias + (int64_t)blockIdx.x * E;
    long long sum = 0;
    int most = 0;
    for (int e = threadIdx.x; e < E; e += kBalanceThreads) {
        sum += n[e];
        most = max(most, n[e]);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    most = __reduce_max_sync(kAll, most);
    if (lane == 0) {
        s_sum[wid] = sum;
        s_max[wid] = most;
    }
    __syncthreads();
    sum = 0;
    most = 0;
    for (int i = 0; i < kBalanceThreads / 32; ++i) {
        sum += s_sum[i];
        most = max(most, s_max[i]);
    }
    for (int e = threadIdx.x; e < E; e += kBalanceThreads) {
        const long long d = sum - (long long)E * n[e];
        if (d != 0) b[e] += d > 0 ? rate : -rate;
    }
    if (imbalance != nullptr && threadIdx.x == 0)
        imbalance[blockIdx.x] = (float)((long long)E * most) / (float)max(sum, 1ll);
}

}  // namespace

cudaError_t launch_logits_grad(const Shape &s, const ScoreGrad &f, const float *logits,
                               const int32_t *idx, const float *w, const float *dw, float *dlogits,
                               const DevStatus &ds, cudaStream_t st) {
    const GradArgs a = {logits, idx, w, dw, s.T, s.E, s.k, f, dlogits};
    const cudaError_t e = f.dense ? launch_grad_any<true>(a, ds, st) : launch_grad_any<false>(a, ds, st);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_balance(const int32_t *counts, int64_t layers, int E, float rate, float *bias,
                           float *imbalance, cudaStream_t st) {
    const cudaError_t e = launch_pdl(balance_kernel, dim3((unsigned)layers), dim3(kBalanceThreads), 0,
                                     st, counts, E, rate, bias, imbalance);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
