// simt_gemm.cuh -- one block's tile of a matrix product on the CUDA cores, in
// fp32: acc[i][j] += sum_k A(m, k) B(k, n).  The operands come through
// functors, so the callers say how a tile's element is found (ragged
// segments, transposed weights, another type); elements outside the matrix
// are the functors' zeros.
#pragma once

#include "common.cuh"

namespace moe {
namespace simt {

constexpr int kThreads = 256;

// BM x BN tile of 256 threads; thread (tx, ty) of a CG x RG grid holds the
// elements (ty + i * RG, tx + j * CG), so shared-memory reads are broadcasts
// along a row and consecutive along a column.
template <int BM_, int BN_, int BK_, int TM_, int TN_> struct Tile {
    static constexpr int BM = BM_, BN = BN_, BK = BK_, TM = TM_, TN = TN_;
    static constexpr int RG = BM / TM, CG = BN / TN;
    static_assert(RG * CG == kThreads, "256 threads");
    struct Smem {
        float a[BK][BM + 1];
        float b[BK][BN + 1];
    };
    static __device__ __forceinline__ int row(int i) { return (int)threadIdx.x / CG + i * RG; }
    static __device__ __forceinline__ int col(int j) { return (int)threadIdx.x % CG + j * CG; }
    static __device__ __forceinline__ void zero(float (&acc)[TM][TN]) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = 0.f;
    }
    // A_K / B_K: the operand is contiguous along k (else along m / n), so
    // consecutive threads load consecutive k.
    template <bool A_K, bool B_K, typename LA, typename LB>
    static __device__ __forceinline__ void product(Smem &sm, int K, LA la, LB lb,
                                                   float (&acc)[TM][TN]) {
        constexpr int NA = BM * BK / kThreads, NB = BN * BK / kThreads;
        float ra[NA], rb[NB];  // the next step's elements, loaded during this step's products
        auto load = [&](int k0) {
#pragma unroll
            for (int r = 0; r < NA; ++r) {
                const int i = (int)threadIdx.x + r * kThreads;
                const int m = A_K ? i / BK : i % BM, k = A_K ? i % BK : i / BM;
                ra[r] = k0 + k < K ? la(m, k0 + k) : 0.f;
            }
#pragma unroll
            for (int r = 0; r < NB; ++r) {
                const int i = (int)threadIdx.x + r * kThreads;
                const int n = B_K ? i / BK : i % BN, k = B_K ? i % BK : i / BN;
                rb[r] = k0 + k < K ? lb(k0 + k, n) : 0.f;
            }
        };
        if (K > 0) load(0);
        for (int k0 = 0; k0 < K; k0 += BK) {
            __syncthreads();  // the previous step's reads are done
#pragma unroll
            for (int r = 0; r < NA; ++r) {
                const int i = (int)threadIdx.x + r * kThreads;
                sm.a[A_K ? i % BK : i / BM][A_K ? i / BK : i % BM] = ra[r];
            }
#pragma unroll
            for (int r = 0; r < NB; ++r) {
                const int i = (int)threadIdx.x + r * kThreads;
                sm.b[B_K ? i % BK : i / BN][B_K ? i / BK : i % BN] = rb[r];
            }
            __syncthreads();
            if (k0 + BK < K) load(k0 + BK);
#pragma unroll
            for (int kk = 0; kk < BK; ++kk) {
                float a[TM], b[TN];
#pragma unroll
                for (int i = 0; i < TM; ++i) a[i] = sm.a[kk][row(i)];
#pragma unroll
                for (int j = 0; j < TN; ++j) b[j] = sm.b[kk][col(j)];
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
            }
        }
    }
};

}  // namespace simt
}  // namespace moe
