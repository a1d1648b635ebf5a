// experts_bwd_f32.cu -- gradient of the grouped SwiGLU experts on the CUDA
// cores.
//
// For expert e and row r of its segment, with g, u = x[r] Wgu[e] recomputed,
// s = sigmoid(g) and dh = dy[r] Wd[e]^T:
//   dg = dh u s (1 + g (1 - s)),   du = dh g s          (rows_kernel -> dgu)
//   dx[r] = [dg du] Wgu[e]^T                            (dx_kernel)
//   dWd[e] = h^T dy,  dWgu[e] = x^T [dg du]             (weights_kernel)
// over the rows of the segment; an expert with no rows gets zero weight
// gradients.  Every sum is fp32 in a fixed order.
#include "common.cuh"
#include "kernels.h"
#include "simt_gemm.cuh"

namespace moe {
namespace {

using Tl = simt::Tile<64, 64, 16, 4, 4>;

// Warp 0: s_off = offsets, s_tile[e] = sum over e' < e of ceil(count_e' / BM).
__device__ void tile_prefix(const int32_t *__restrict__ offsets, int E, int *s_off, int *s_tile) {
    for (int e = threadIdx.x; e <= E; e += blockDim.x) s_off[e] = offsets[e];
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int per = (E + 31) / 32;
        const int e0 = min(E, lane * per), e1 = min(E, e0 + per);
        int local = 0;
        for (int e = e0; e < e1; ++e) local += (s_off[e + 1] - s_off[e] + Tl::BM - 1) / Tl::BM;
        int incl = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        int run = incl - local;
        for (int e = e0; e < e1; ++e) {
            s_tile[e] = run;
            run += (s_off[e + 1] - s_off[e] + Tl::BM - 1) / Tl::BM;
        }
        if (lane == 31) s_tile[E] = incl;
    }
    __syncthreads();
}

struct RowTile {
    int e, row0, rows;
};
__device__ __forceinline__ bool find_tile(const int32_t *offsets, int E, int *s_dyn, RowTile *t) {
    int *s_off = s_dyn, *s_tile = s_dyn + E + 1;
    tile_prefix(offsets, E, s_off, s_tile);
    const int g = blockIdx.x;
    if (g >= s_tile[E]) return false;
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_tile[mid] <= g) lo = mid; else hi = mid - 1;
    }
    t->e = lo;
    t->row0 = s_off[lo] + (g - s_tile[lo]) * Tl::BM;
    t->rows = min(Tl::BM, s_off[lo + 1] - t->row0);
    return true;
}

template <typename TA>
__global__ void __launch_bounds__(simt::kThreads)
rows_kernel(const TA *__restrict__ x, const TA *__restrict__ dy, const int32_t *__restrict__ offsets,
            int E, const TA *__restrict__ Wgu, const TA *__restrict__ Wd, int d, int f,
            TA *__restrict__ dgu) {
    pdl_entry();
    extern __shared__ int s_dyn[];
    __shared__ Tl::Smem sm;
    RowTile t;
    if (!find_tile(offsets, E, s_dyn, &t)) return;
    const int n0 = blockIdx.y * Tl::BN;
    const TA *xr = x + (int64_t)t.row0 * d, *yr = dy + (int64_t)t.row0 * d;
    const TA *W = Wgu + (int64_t)t.e * d * 2 * f, *Wt = Wd + (int64_t)t.e * f * d;
    float g[Tl::TM][Tl::TN], u[Tl::TM][Tl::TN], h[Tl::TM][Tl::TN];
    Tl::zero(g);
    Tl::zero(u);
    Tl::zero(h);
    auto la = [&](const TA *a) {
        return [=](int m, int k) { return m < t.rows ? Act<TA>::to_f(a[(int64_t)m * d + k]) : 0.f; };
    };
    Tl::product<true, false>(sm, d, la(xr), [&](int k, int n) {
        return n0 + n < f ? Act<TA>::to_f(W[(int64_t)k * 2 * f + n0 + n]) : 0.f; }, g);
    Tl::product<true, false>(sm, d, la(xr), [&](int k, int n) {
        return n0 + n < f ? Act<TA>::to_f(W[(int64_t)k * 2 * f + f + n0 + n]) : 0.f; }, u);
    Tl::product<true, true>(sm, d, la(yr), [&](int k, int n) {
        return n0 + n < f ? Act<TA>::to_f(Wt[(int64_t)(n0 + n) * d + k]) : 0.f; }, h);
#pragma unroll
    for (int i = 0; i < Tl::TM; ++i) {
        const int m = Tl::row(i);
        if (m >= t.rows) continue;
        TA *o = dgu + (int64_t)(t.row0 + m) * 2 * f;
#pragma unroll
        for (int j = 0; j < Tl::TN; ++j) {
            const int n = n0 + Tl::col(j);
            if (n >= f) continue;
            const float s = 1.f / (1.f + expf(-g[i][j]));
            o[n] = Act<TA>::from_f(h[i][j] * u[i][j] * s * (1.f + g[i][j] * (1.f - s)));
            o[f + n] = Act<TA>::from_f(h[i][j] * g[i][j] * s);
        }
    }
}

template <typename TA>
__global__ void __launch_bounds__(simt::kThreads)
dx_kernel(const TA *__restrict__ dgu, const int32_t *__restrict__ offsets, int E,
          const TA *__restrict__ Wgu, int d, int f, TA *__restrict__ dx) {
    pdl_entry();
    extern __shared__ int s_dyn[];
    __shared__ Tl::Smem sm;
    RowTile t;
    if (!find_tile(offsets, E, s_dyn, &t)) return;
    const int n0 = blockIdx.y * Tl::BN, K = 2 * f;
    const TA *a = dgu + (int64_t)t.row0 * K, *W = Wgu + (int64_t)t.e * d * K;
    float acc[Tl::TM][Tl::TN];
    Tl::zero(acc);
    Tl::product<true, true>(
        sm, K, [&](int m, int k) { return m < t.rows ? Act<TA>::to_f(a[(int64_t)m * K + k]) : 0.f; },
        [&](int k, int n) { return n0 + n < d ? Act<TA>::to_f(W[(int64_t)(n0 + n) * K + k]) : 0.f; },
        acc);
#pragma unroll
    for (int i = 0; i < Tl::TM; ++i)
#pragma unroll
        for (int j = 0; j < Tl::TN; ++j) {
            const int m = Tl::row(i), n = n0 + Tl::col(j);
            if (m < t.rows && n < d) dx[(int64_t)(t.row0 + m) * d + n] = Act<TA>::from_f(acc[i][j]);
        }
}

// dW[e] [M][N] = A^T B over the rows of expert e's segment (A [P][M], B [P][N]).
template <typename TA>
__global__ void __launch_bounds__(simt::kThreads)
weights_kernel(const TA *__restrict__ A, const TA *__restrict__ B,
               const int32_t *__restrict__ offsets, int M, int N, TA *__restrict__ dW) {
    pdl_entry();
    __shared__ Tl::Smem sm;
    const int e = blockIdx.z, m0 = blockIdx.y * Tl::BM, n0 = blockIdx.x * Tl::BN;
    const int r0 = offsets[e], rows = offsets[e + 1] - r0;
    const TA *a = A + (int64_t)r0 * M, *b = B + (int64_t)r0 * N;
    float acc[Tl::TM][Tl::TN];
    Tl::zero(acc);
    Tl::product<false, false>(
        sm, rows, [&](int m, int k) { return m0 + m < M ? Act<TA>::to_f(a[(int64_t)k * M + m0 + m]) : 0.f; },
        [&](int k, int n) { return n0 + n < N ? Act<TA>::to_f(b[(int64_t)k * N + n0 + n]) : 0.f; }, acc);
    TA *o = dW + (int64_t)e * M * N;
#pragma unroll
    for (int i = 0; i < Tl::TM; ++i)
#pragma unroll
        for (int j = 0; j < Tl::TN; ++j) {
            const int m = m0 + Tl::row(i), n = n0 + Tl::col(j);
            if (m < M && n < N) o[(int64_t)m * N + n] = Act<TA>::from_f(acc[i][j]);
        }
}

template <typename TA>
cudaError_t launch_t(const Shape &s, const ExpertsBwd &a, cudaStream_t st) {
    const TA *x = static_cast<const TA *>(a.x_perm), *dy = static_cast<const TA *>(a.dy_perm);
    const TA *Wgu = static_cast<const TA *>(a.Wgu), *Wd = static_cast<const TA *>(a.Wd);
    TA *dgu = static_cast<TA *>(a.ws);
    const unsigned mt = (unsigned)((s.P() + Tl::BM - 1) / Tl::BM + s.E);
    const size_t sh = sizeof(int) * (2 * (size_t)s.E + 2);
    auto tiles = [](int n) { return (unsigned)((n + Tl::BN - 1) / Tl::BN); };
    const dim3 block(simt::kThreads);
    launch_pdl(rows_kernel<TA>, dim3(mt, tiles(s.f)), block, sh, st, x, dy, a.offsets, s.E, Wgu, Wd,
               s.d, s.f, dgu);
    launch_pdl(dx_kernel<TA>, dim3(mt, tiles(s.d)), block, sh, st, (const TA *)dgu, a.offsets, s.E,
               Wgu, s.d, s.f, static_cast<TA *>(a.dx_perm));
    launch_pdl(weights_kernel<TA>, dim3(tiles(s.d), tiles(s.f), s.E), block, 0, st,
               static_cast<const TA *>(a.h_perm), dy, a.offsets, s.f, s.d, static_cast<TA *>(a.dWd));
    launch_pdl(weights_kernel<TA>, dim3(tiles(2 * s.f), tiles(s.d), s.E), block, 0, st, x,
               (const TA *)dgu, a.offsets, s.d, 2 * s.f, static_cast<TA *>(a.dWgu));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_experts_backward_f32(const Shape &s, const ExpertsBwd &a, cudaStream_t st) {
    return launch_t<float>(s, a, st);
}

}  // namespace moe
