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
// 8: 14.1 us, latency (one tile shape of 32 x 32 for all products 22.4; dx and
// the weights in launches of their own 24).  T = 1024, k = E = 8, d = f = 512 (34
// GFLOP): 821 us, 42 TFLOP/s, bound by the multiply-adds and the instructions
// beside them (64 x 64 tiles of 4 x 4 micro tiles, g and u apart, unpacked: 914).
// T = 512, d = f = 488, E = 32, k = 4, routed unevenly: 298 us (508).
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

// Dynamic shared memory of a kernel with products of two tile shapes: the larger
// one's stages; then 2 (E + 1) ints of tile_prefix.
template <typename A, typename B>
constexpr int kSmem = A::SMEM_BYTES > B::SMEM_BYTES ? A::SMEM_BYTES : B::SMEM_BYTES;

// g and u are one product over twice the columns, so that x's fragments are read
// once for both: a thread holds g in its first TN accumulators of a row, u of the
// same columns in the others.
template <typename Tl> using Wide = simt::Tile<Tl::BM, 2 * Tl::BN, Tl::TM, 2 * Tl::TN, Tl::VN>;

template <typename Tl>
__global__ void __launch_bounds__(Tl::THREADS)
rows_kernel(const float *__restrict__ x, const float *__restrict__ dy,
            const int32_t *__restrict__ offsets, int E, const float *__restrict__ Wgu,
            const float *__restrict__ Wd, int d, int f, float *__restrict__ dgu) {
    using GU = Wide<Tl>;
    static_assert(Tl::TN == Tl::VN, "a run of g is followed by u's");
    pdl_wait();
    extern __shared__ __align__(16) float smem[];
    RowTile t;
    if (!find_tile<Tl::BM>(offsets, E, reinterpret_cast<int *>(smem) + kSmem<Tl, GU> / 4, blockIdx.x, &t))
        return;
    const int n0 = blockIdx.y * Tl::BN;
    const float *xr = x + (int64_t)t.row0 * d, *yr = dy + (int64_t)t.row0 * d;
    const float *W = Wgu + (int64_t)t.e * d * 2 * f, *Wt = Wd + (int64_t)t.e * f * d;
    float gu[Tl::TM][2 * Tl::TN], h[Tl::TM][Tl::TN];  // g, then u
    GU::zero(gu);
    Tl::zero(h);
    auto rows_of = [&](const float *a) {
        return [=](int m, int k) { return m < t.rows ? a + (int64_t)m * d + k : nullptr; };
    };
    GU::template product<true, false>(smem, d, rows_of(xr), [=](int k, int n) {
        const int half = n < Tl::BN ? 0 : 1, c = n0 + n - half * Tl::BN;
        return c < f ? W + (int64_t)k * 2 * f + half * f + c : nullptr; }, gu);
    Tl::template product<true, true>(smem, d, rows_of(yr), [=](int k, int n) {
        return n0 + n < f ? Wt + (int64_t)(n0 + n) * d + k : nullptr; }, h);
#pragma unroll
    for (int i = 0; i < Tl::TM; ++i) {
        const int m = Tl::row(i);
        if (m >= t.rows) continue;
        float *o = dgu + (int64_t)(t.row0 + m) * 2 * f;
#pragma unroll
        for (int j = 0; j < Tl::TN; j += Tl::VN) {
            const int n = n0 + Tl::col(j);
            if (n >= f) continue;
            float dg[Tl::VN], du[Tl::VN];
#pragma unroll
            for (int l = 0; l < Tl::VN; ++l) {
                const float g = gu[i][j + l], u = gu[i][Tl::TN + j + l], dh = h[i][j + l];
                const float s = 1.f / (1.f + expf(-g));
                dg[l] = dh * u * s * (1.f + g * (1.f - s));
                du[l] = dh * g * s;
            }
            Tl::store(o + n, dg);
            Tl::store(o + f + n, du);
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
template <typename X, typename W>
__global__ void __launch_bounds__(W::THREADS, W::MIN_BLOCKS)
dx_weights_kernel(const float *__restrict__ dgu, const int32_t *__restrict__ offsets, int E,
                  const float *__restrict__ Wgu, int d, int f, float *__restrict__ dx, int dx_blocks,
                  WeightProduct wd, WeightProduct wg) {
    pdl_wait();
    extern __shared__ __align__(16) float smem[];
    static_assert(X::THREADS == W::THREADS, "one block size");
    if ((int)blockIdx.x < dx_blocks) {
        const int nt = (d + X::BN - 1) / X::BN;
        RowTile t;
        if (!find_tile<X::BM>(offsets, E, reinterpret_cast<int *>(smem) + kSmem<X, W> / 4,
                               (int)blockIdx.x / nt, &t))
            return;
        float acc[X::TM][X::TN];
        X::zero(acc);
        const int n0 = (int)blockIdx.x % nt * X::BN, K = 2 * f;
        const float *a = dgu + (int64_t)t.row0 * K, *w = Wgu + (int64_t)t.e * d * K;
        X::template product<true, true>(
            smem, K, [=](int m, int k) { return m < t.rows ? a + (int64_t)m * K + k : nullptr; },
            [=](int k, int n) { return n0 + n < d ? w + (int64_t)(n0 + n) * K + k : nullptr; }, acc);
        X::each_run(acc, [&](int m, int c, const float *v) {
            if (m < t.rows && n0 + c < d) X::store(dx + (int64_t)(t.row0 + m) * d + n0 + c, v);
        });
        return;
    }
    const int per = wd.tiles + wg.tiles, b = (int)blockIdx.x - dx_blocks;
    const int e = b / per, g = b % per;
    const WeightProduct &p = g < wd.tiles ? wd : wg;
    const int tile = g < wd.tiles ? g : g - wd.tiles;
    const int nt = (p.N + W::BN - 1) / W::BN;
    const int m0 = tile / nt * W::BM, n0 = tile % nt * W::BN, M = p.M, N = p.N;
    const int r0 = offsets[e], rows = offsets[e + 1] - r0;
    const float *A = p.A + (int64_t)r0 * M, *B = p.B + (int64_t)r0 * N;
    float acc[W::TM][W::TN];
    W::zero(acc);
    W::template product<false, false>(
        smem, rows, [=](int m, int k) { return m0 + m < M ? A + (int64_t)k * M + m0 + m : nullptr; },
        [=](int k, int n) { return n0 + n < N ? B + (int64_t)k * N + n0 + n : nullptr; }, acc);
    float *o = p.dW + (int64_t)e * M * N;
    W::each_run(acc, [&](int m, int c, const float *v) {
        if (m0 + m < M && n0 + c < N) W::store(o + (int64_t)(m0 + m) * N + n0 + c, v);
    });
}

unsigned tiles(int n, int b) { return (unsigned)((n + b - 1) / b); }
// Row tiles at most: a partial one for each expert with rows.
unsigned row_tiles_most(const Shape &s, int b) {
    return (unsigned)((s.P() + b - 1) / b + (s.P() < s.E ? s.P() : s.E));
}
constexpr int kPrefixMax = 16 * 1024;
size_t prefix_bytes(const Shape &s) { return sizeof(int) * (2 * (size_t)s.E + 2); }

// 128 threads each.  Rows of the segment x columns:
using Tiny = simt::Tile<16, 32, 2, 2>;    // the most blocks, six stages: short chains of latency
using Short = simt::Tile<16, 64, 2, 4>;
using Mid = simt::Tile<32, 64, 4, 4>;
using Tall = simt::Tile<64, 64, 8, 4>;    // the largest whose g, u and dh fit a thread
using Large = simt::Tile<64, 128, 8, 8>;

template <typename R> cudaError_t launch_rows(const Shape &s, const ExpertsBwd &a, cudaStream_t st) {
    constexpr int smem = kSmem<R, Wide<R>>;
    cudaError_t err = simt::opt_in<rows_kernel<R>>(smem + kPrefixMax);
    if (err != cudaSuccess) return err;
    launch_pdl(rows_kernel<R>, dim3(row_tiles_most(s, R::BM), tiles(s.f, R::BN)), dim3(R::THREADS),
               smem + prefix_bytes(s), st, static_cast<const float *>(a.x_perm),
               static_cast<const float *>(a.dy_perm), a.offsets, s.E,
               static_cast<const float *>(a.Wgu), static_cast<const float *>(a.Wd), s.d, s.f,
               static_cast<float *>(a.ws));
    return cudaGetLastError();
}

template <typename X, typename W>
cudaError_t launch_dx_weights(const Shape &s, const ExpertsBwd &a, cudaStream_t st) {
    constexpr int smem = kSmem<X, W>;
    cudaError_t err = simt::opt_in<dx_weights_kernel<X, W>>(smem + kPrefixMax);
    if (err != cudaSuccess) return err;
    const float *dgu = static_cast<const float *>(a.ws);
    auto product = [&](const void *A, int M, const void *B, int N, void *dW) {
        return WeightProduct{static_cast<const float *>(A), static_cast<const float *>(B), M, N,
                             (int)(tiles(M, W::BM) * tiles(N, W::BN)), static_cast<float *>(dW)};
    };
    const WeightProduct wd = product(a.h_perm, s.f, a.dy_perm, s.d, a.dWd);
    const WeightProduct wg = product(a.x_perm, s.d, dgu, 2 * s.f, a.dWgu);
    const int64_t dx_blocks = (int64_t)row_tiles_most(s, X::BM) * tiles(s.d, X::BN);
    const int64_t blocks = dx_blocks + (int64_t)s.E * (wd.tiles + wg.tiles);
    if (blocks > INT32_MAX) {
        set_error_message("experts' gradient tile count exceeds 2^31");
        return cudaErrorInvalidValue;
    }
    launch_pdl(dx_weights_kernel<X, W>, dim3((unsigned)blocks), dim3(W::THREADS), smem + prefix_bytes(s), st,
               dgu, a.offsets, s.E, static_cast<const float *>(a.Wgu), s.d, s.f,
               static_cast<float *>(a.dx_perm), (int)dx_blocks, wd, wg);
    return cudaGetLastError();
}

// Tiles of a product over the rows of all segments: each expert's last one is
// half full on average.
int64_t row_tiles(const Shape &s, int bm, int columns) {
    const int64_t experts = s.P() < s.E ? s.P() : s.E;
    return (s.P() / bm + (experts + 1) / 2) * columns;
}

}  // namespace

// The tiles, by what runs out first.  Few blocks, or segments shorter than a
// tile: smaller tiles; else the larger micro tile, which reads less shared
// memory per multiply-add.  Measured (us), rows an expert r:
//   rows_kernel, Tiny / Short / Mid / Tall
//     T = 64, d = 128, f = 256, E = 8, k = 2               7.0 / 9.5 / 13.4 / 19
//     T = 64, d = f = 512, E = 128, k = 8 (r = 4)          147 / 126 / 193 / 326
//     T = 1024, d = 256, f = 512, E = 8, k = 2 (r = 256)   73 / 64 / 60 / 76
//     T = 1024, d = f = 512, E = 128, k = 8 (r = 64)       606 / 527 / 452 / 466
//     T = 1024, d = f = 512, E = k = 8 (r = 1024)          530 / 458 / 373 / 329
//   dx in Tiny / Mid / Large tiles, the weight gradients' Large, same shapes
//     8.3 / 18 / 48,  189 / 227 / 336,  94 / 85 / 105,  741 / 656 / 666,  686 / 567 / 508
//   weight gradients in Tiny / Mid / Large tiles, dx's Tiny
//     T = 64, d = 128, f = 256, E = 8, k = 2               11.0 / 11.0 / 8.3
//     T = 300, d = f = 128, E = 4, k = 2 (r = 150)         9.6 / 7.9 / 13.9
//     T = 200, d = f = 512, E = 4, k = 2 (r = 100)         59.5 / 45.1 / 41.4
cudaError_t launch_experts_backward_f32(const Shape &s, const ExpertsBwd &a, cudaStream_t st) {
    constexpr int kSms = 152;
    const int64_t r = s.P() / s.E;
    cudaError_t err;
    if (r < 16 || row_tiles(s, Mid::BM, tiles(s.f, Mid::BN)) < kSms)
        err = row_tiles(s, Tiny::BM, tiles(s.f, Tiny::BN)) < 2 * kSms ? launch_rows<Tiny>(s, a, st)
                                                                     : launch_rows<Short>(s, a, st);
    else
        err = r >= 256 && row_tiles(s, Tall::BM, tiles(s.f, Tall::BN)) >= 3 * kSms
                  ? launch_rows<Tall>(s, a, st)
                  : launch_rows<Mid>(s, a, st);
    if (err != cudaSuccess) return err;
    auto weight_tiles = [&](int bm, int bn) {
        return (int64_t)s.E * (tiles(s.f, bm) * tiles(s.d, bn) + tiles(s.d, bm) * tiles(2 * s.f, bn));
    };
    // a weight gradient's chain is as long as its segment
    const bool w_large = r <= 64 || weight_tiles(Large::BM, Large::BN) >= kSms;
    const bool w_mid = weight_tiles(Mid::BM, Mid::BN) >= kSms;
    if (r < 16 || row_tiles(s, Mid::BM, tiles(s.d, Mid::BN)) < kSms)
        return w_large ? launch_dx_weights<Tiny, Large>(s, a, st)
               : w_mid ? launch_dx_weights<Tiny, Mid>(s, a, st)
                       : launch_dx_weights<Tiny, Tiny>(s, a, st);
    if (!w_large)
        return w_mid ? launch_dx_weights<Mid, Mid>(s, a, st) : launch_dx_weights<Mid, Tiny>(s, a, st);
    return r >= 256 && row_tiles(s, Large::BM, tiles(s.d, Large::BN)) >= 2 * kSms
               ? launch_dx_weights<Large, Large>(s, a, st)
               : launch_dx_weights<Mid, Large>(s, a, st);
}

}  // namespace moe
