// experts_bwd_f32.cu -- gradient of the grouped SwiGLU experts for fp32
// activations, on the CUDA cores.
//
// For expert e and row r of its segment, with g, u = x[r] Wgu[e] recomputed,
// s = sigmoid(g) and dh = dy[r] Wd[e]^T:
//   dg = dh u s (1 + g (1 - s)),   du = dh g s          (rows_kernel -> dgu)
//   dx[r] = [dg du] Wgu[e]^T,
//   dWd[e] = h^T dy,  dWgu[e] = x^T [dg du]             (dx_weights_kernel)
// over the rows of the segment; an expert with no rows gets zero weight
// gradients.  Every sum is fp32 in a fixed order.
//
// Two launches over the tile of simt_gemm.cuh.  T = 64, d = 128, f = 256, E =
// 8: 22.4 us, latency (tiles of 32 x 32; 64 x 64 without the pipeline 45 to 100;
// dx and the weights in launches of their own 24).  T = 1024, k = E = 8, d = f =
// 512 (34 GFLOP): 914 us, 38 TFLOP/s, bound by the multiply-adds and the
// shared-memory loads beside them (128 x 64 tiles 957, 128 x 128 1491).
#include "common.cuh"
#include "kernels.h"
#include "simt_gemm.cuh"

namespace moe {
namespace {

// s_off = offsets; s_tile[e] = sum over e' < e of ceil(count_e' / BM).
template <int BM>
__device__ void tile_prefix(const int32_t *__restrict__ offsets, int E, int *s_off, int *s_tile) {
    for (int e = threadIdx.x; e <= E; e += blockDim.x) s_off[e] = offsets[e];
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int per = (E + 31) / 32;
        const int e0 = min(E, lane * per), e1 = min(E, e0 + per);
        int local = 0;
        for (int e = e0; e < e1; ++e) local += (s_off[e + 1] - s_off[e] + BM - 1) / BM;
        int incl = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        int run = incl - local;
        for (int e = e0; e < e1; ++e) {
            s_tile[e] = run;
            run += (s_off[e + 1] - s_off[e] + BM - 1) / BM;
        }
        if (lane == 31) s_tile[E] = incl;
    }
    __syncthreads();
}

struct RowTile {
    int e, row0, rows;
};
template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t *offsets, int E, int *s_dyn, int g, RowTile *t) {
    int *s_off = s_dyn, *s_tile = s_dyn + E + 1;
    tile_prefix<BM>(offsets, E, s_off, s_tile);
    if (g >= s_tile[E]) return false;
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_tile[mid] <= g) lo = mid; else hi = mid - 1;
    }
    t->e = lo;
    t->row0 = s_off[lo] + (g - s_tile[lo]) * BM;
    t->rows = min(BM, s_off[lo + 1] - t->row0);
    return true;
}

// Dynamic shared memory: the product's stages, then 2 (E + 1) ints.
template <typename Tl>
__global__ void __launch_bounds__(simt::kThreads)
rows_kernel(const float *__restrict__ x, const float *__restrict__ dy,
            const int32_t *__restrict__ offsets, int E, const float *__restrict__ Wgu,
            const float *__restrict__ Wd, int d, int f, float *__restrict__ dgu) {
    pdl_wait();
    extern __shared__ __align__(16) float smem[];
    RowTile t;
    if (!find_tile<Tl::BM>(offsets, E, reinterpret_cast<int *>(smem) + Tl::SMEM_BYTES / 4, blockIdx.x, &t))
        return;
    const int n0 = blockIdx.y * Tl::BN;
    const float *xr = x + (int64_t)t.row0 * d, *yr = dy + (int64_t)t.row0 * d;
    const float *W = Wgu + (int64_t)t.e * d * 2 * f, *Wt = Wd + (int64_t)t.e * f * d;
    float g[Tl::TM][Tl::TN], u[Tl::TM][Tl::TN], h[Tl::TM][Tl::TN];
    Tl::zero(g);
    Tl::zero(u);
    Tl::zero(h);
    auto rows_of = [&](const float *a) {
        return [=](int m, int k) { return m < t.rows ? a + (int64_t)m * d + k : nullptr; };
    };
    auto cols_of = [&](const float *b) {
        return [=](int k, int n) { return n0 + n < f ? b + (int64_t)k * 2 * f + n0 + n : nullptr; };
    };
    Tl::template product<true, false, true>(smem, d, rows_of(xr), cols_of(W), g);
    Tl::template product<true, false, true>(smem, d, rows_of(xr), cols_of(W + f), u);
    Tl::template product<true, true, true>(smem, d, rows_of(yr), [=](int k, int n) {
        return n0 + n < f ? Wt + (int64_t)(n0 + n) * d + k : nullptr; }, h);
#pragma unroll
    for (int i = 0; i < Tl::TM; ++i) {
        const int m = Tl::template row<true>(i);
        if (m >= t.rows) continue;
        float *o = dgu + (int64_t)(t.row0 + m) * 2 * f;
#pragma unroll
        for (int j = 0; j < Tl::TN; ++j) {
            const int n = n0 + Tl::template col<true>(j);
            if (n >= f) continue;
            const float s = 1.f / (1.f + expf(-g[i][j]));
            o[n] = h[i][j] * u[i][j] * s * (1.f + g[i][j] * (1.f - s));
            o[f + n] = h[i][j] * g[i][j] * s;
        }
    }
}

// dW[e] [M][N] = A^T B over the rows of expert e's segment (A [P][M], B [P][N]).
struct WeightProduct {
    const float *A, *B;
    int M, N, tiles;  // tiles of one expert's dW
    float *dW;
};

// dx and both weight gradients, none of which reads another's output, in one
// launch: blocks below dx_blocks are dx's tiles (column tiles fastest), whose
// chain over 2f is the longest, then every expert's tiles of wd and wg.
template <typename Tl>
__global__ void __launch_bounds__(simt::kThreads)
dx_weights_kernel(const float *__restrict__ dgu, const int32_t *__restrict__ offsets, int E,
                  const float *__restrict__ Wgu, int d, int f, float *__restrict__ dx, int dx_blocks,
                  WeightProduct wd, WeightProduct wg) {
    pdl_wait();
    extern __shared__ __align__(16) float smem[];
    float acc[Tl::TM][Tl::TN];
    Tl::zero(acc);
    if ((int)blockIdx.x < dx_blocks) {
        const int nt = (d + Tl::BN - 1) / Tl::BN;
        RowTile t;
        if (!find_tile<Tl::BM>(offsets, E, reinterpret_cast<int *>(smem) + Tl::SMEM_BYTES / 4,
                               (int)blockIdx.x / nt, &t))
            return;
        const int n0 = (int)blockIdx.x % nt * Tl::BN, K = 2 * f;
        const float *a = dgu + (int64_t)t.row0 * K, *W = Wgu + (int64_t)t.e * d * K;
        Tl::template product<true, true, true>(
            smem, K, [=](int m, int k) { return m < t.rows ? a + (int64_t)m * K + k : nullptr; },
            [=](int k, int n) { return n0 + n < d ? W + (int64_t)(n0 + n) * K + k : nullptr; }, acc);
#pragma unroll
        for (int i = 0; i < Tl::TM; ++i)
#pragma unroll
            for (int j = 0; j < Tl::TN; ++j) {
                const int m = Tl::template row<true>(i), n = n0 + Tl::template col<true>(j);
                if (m < t.rows && n < d) dx[(int64_t)(t.row0 + m) * d + n] = acc[i][j];
            }
        return;
    }
    const int per = wd.tiles + wg.tiles, b = (int)blockIdx.x - dx_blocks;
    const int e = b / per, g = b % per;
    const WeightProduct &p = g < wd.tiles ? wd : wg;
    const int tile = g < wd.tiles ? g : g - wd.tiles;
    const int nt = (p.N + Tl::BN - 1) / Tl::BN;
    const int m0 = tile / nt * Tl::BM, n0 = tile % nt * Tl::BN, M = p.M, N = p.N;
    const int r0 = offsets[e], rows = offsets[e + 1] - r0;
    const float *A = p.A + (int64_t)r0 * M, *B = p.B + (int64_t)r0 * N;
    Tl::template product<false, false, false>(
        smem, rows, [=](int m, int k) { return m0 + m < M ? A + (int64_t)k * M + m0 + m : nullptr; },
        [=](int k, int n) { return n0 + n < N ? B + (int64_t)k * N + n0 + n : nullptr; }, acc);
    float *o = p.dW + (int64_t)e * M * N;
#pragma unroll
    for (int i = 0; i < Tl::TM; ++i)
#pragma unroll
        for (int j = 0; j < Tl::TN; ++j) {
            const int m = m0 + Tl::template row<false>(i), n = n0 + Tl::template col<false>(j);
            if (m < M && n < N) o[(int64_t)m * N + n] = acc[i][j];
        }
}

template <typename Tl> cudaError_t launch_t(const Shape &s, const ExpertsBwd &a, cudaStream_t st) {
    const float *x = static_cast<const float *>(a.x_perm), *dy = static_cast<const float *>(a.dy_perm);
    const float *Wgu = static_cast<const float *>(a.Wgu), *Wd = static_cast<const float *>(a.Wd);
    float *dgu = static_cast<float *>(a.ws);
    const int64_t P = s.P();
    const unsigned mt = (unsigned)((P + Tl::BM - 1) / Tl::BM + (P < s.E ? P : s.E));
    const size_t prefix = sizeof(int) * (2 * (size_t)s.E + 2);
    auto tiles = [](int n, int b) { return (unsigned)((n + b - 1) / b); };
    const dim3 block(simt::kThreads);
    cudaError_t err;
    if ((err = simt::opt_in<rows_kernel<Tl>>(Tl::SMEM_BYTES + 16 * 1024)) != cudaSuccess ||
        (err = simt::opt_in<dx_weights_kernel<Tl>>(Tl::SMEM_BYTES + 16 * 1024)) != cudaSuccess)
        return err;
    launch_pdl(rows_kernel<Tl>, dim3(mt, tiles(s.f, Tl::BN)), block, Tl::SMEM_BYTES + prefix, st, x, dy,
               a.offsets, s.E, Wgu, Wd, s.d, s.f, dgu);
    auto product = [&](const float *A, int M, const float *B, int N, void *dW) {
        return WeightProduct{A, B, M, N, (int)(tiles(M, Tl::BM) * tiles(N, Tl::BN)), static_cast<float *>(dW)};
    };
    const WeightProduct wd = product(static_cast<const float *>(a.h_perm), s.f, dy, s.d, a.dWd);
    const WeightProduct wg = product(x, s.d, dgu, 2 * s.f, a.dWgu);
    const int64_t dx_blocks = (int64_t)mt * tiles(s.d, Tl::BN);
    const int64_t blocks = dx_blocks + (int64_t)s.E * (wd.tiles + wg.tiles);
    if (blocks > INT32_MAX) {
        set_error_message("experts' gradient tile count exceeds 2^31");
        return cudaErrorInvalidValue;
    }
    launch_pdl(dx_weights_kernel<Tl>, dim3((unsigned)blocks), block, Tl::SMEM_BYTES + prefix, st,
               (const float *)dgu, a.offsets, s.E, Wgu, s.d, s.f, static_cast<float *>(a.dx_perm),
               (int)dx_blocks, wd, wg);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_experts_backward_f32(const Shape &s, const ExpertsBwd &a, cudaStream_t st) {
    using L = simt::Large;
    const int64_t row_tiles = (s.P() + L::BM - 1) / L::BM;
    // the row products have the fewest tiles
    const bool large = row_tiles * ((s.d + L::BN - 1) / L::BN) >= 2 * 152;
    return large ? launch_t<simt::Large>(s, a, st) : launch_t<simt::Small>(s, a, st);
}

}  // namespace moe
