// simt_gemm.cuh -- one block's tile of an fp32 matrix product on the CUDA
// cores: acc[i][j] += sum_k A(m, k) B(k, n), for operands stored either way
// round.  The callers say through functors where four consecutive elements
// lie (ragged segments, transposed weights) or that they are outside the
// matrix; such elements are zeros.
#pragma once

#include "common.cuh"
#include "once.h"
#include "tc_ptx.cuh"

namespace moe {
namespace simt {

constexpr int BK = 32;  // k per stage

__device__ __forceinline__ void copy16_or_zero(float *dst, const float *src) {
    if (src) tc::cp_async16(tc::smem_u32(dst), src);
    else *reinterpret_cast<float4 *>(dst) = make_float4(0.f, 0.f, 0.f, 0.f);
}
template <int V> __device__ __forceinline__ void lds(float *v, const float *s) {
    if constexpr (V == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(s);
    else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(s);
}

// BM x BN tile, TM x TN elements a thread, in runs of V (four, or two where a
// thread has only two) that lie next to each other: every read of shared memory
// is a vector.  A k-contiguous operand is staged as [rows][BK], 16-byte chunk c of
// row r at c ^ (r / V % 8), so that threads reading the same k of neighbouring
// runs meet different banks; the other kind as [BK][columns].
//
// Stages in flight (cp.async): six for the smallest tiles, and two where micro tiles of
// 8 x 8 leave room for more blocks by that, with the registers of four a block of 128
// threads (router's fp32 products, T = 8192, d = 4096, E = 128: 341 us to 320).
template <int BM_, int BN_, int TM_, int TN_, int VN_ = (TN_ < 4 ? TN_ : 4)> struct Tile {
    static constexpr int BM = BM_, BN = BN_, TM = TM_, TN = TN_;
    static constexpr int RG = BM / TM, CG = BN / TN, THREADS = RG * CG;
    static constexpr int VM = TM < 4 ? TM : 4, VN = VN_;
    static constexpr int STAGES = BM * BN <= 16 * 32 ? 6 : TM * TN == 64 ? 2 : 3;
    static constexpr int MIN_BLOCKS = STAGES == 2 ? 4 : 1;
    static constexpr int A_FLOATS = BM * BK, B_FLOATS = BN * BK;
    static constexpr int SMEM_BYTES = STAGES * (A_FLOATS + B_FLOATS) * (int)sizeof(float);

    static_assert(TM % VM == 0 && TN % VN == 0 && VN % 2 == 0 && VN <= 4 && BM % 4 == 0 && BN % 4 == 0, "");

    // Element (i, j) of this thread.
    static __device__ __forceinline__ int row(int i) {
        return i / VM * (RG * VM) + (int)threadIdx.x / CG * VM + i % VM;
    }
    static __device__ __forceinline__ int col(int j) {
        return j / VN * (CG * VN) + (int)threadIdx.x % CG * VN + j % VN;
    }
    // f(row, col, run) for each run of VN elements.
    template <typename F> static __device__ __forceinline__ void each_run(const float (&acc)[TM][TN], F f) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; j += VN) f(row(i), col(j), &acc[i][j]);
    }
    static __device__ __forceinline__ void store(float *dst, const float *v) {
        if constexpr (VN == 4) *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
        else *reinterpret_cast<float2 *>(dst) = make_float2(v[0], v[1]);
    }
    static __device__ __forceinline__ void zero(float (&acc)[TM][TN]) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = 0.f;
    }

    // Stages rows k0 .. k0 + BK - 1 of k of an operand with N rows or columns.
    template <bool KC, int N, int V, typename L>
    static __device__ __forceinline__ void stage(float *dst, int k0, int K, L at) {
        constexpr int C = (KC ? BK : N) / 4, ALL = N * BK / 4;  // chunks of a row, and in all
#pragma unroll
        for (int r = 0; r < (ALL + THREADS - 1) / THREADS; ++r) {
            const int i = (int)threadIdx.x + r * THREADS;
            if (ALL % THREADS && i >= ALL) break;
            const int o = i / C, c = i % C;
            const int m = KC ? o : 4 * c, k = k0 + (KC ? 4 * c : o);
            copy16_or_zero(dst + (KC ? o * BK + 4 * (c ^ (o / V % 8)) : 4 * i), k < K ? at(m, k) : nullptr);
        }
    }
    // v[i][q]: element at(i) of the operand, k = kk + q, q < 4.
    template <bool KC, int N, int T, int V, typename AT>
    static __device__ __forceinline__ void fragment(const float *src, int kk, float (&v)[T][4], AT at) {
        if constexpr (KC) {
#pragma unroll
            for (int i = 0; i < T; ++i) lds<4>(v[i], src + at(i) * BK + 4 * (kk / 4 ^ (at(i) / V % 8)));
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int i = 0; i < T; i += V) {
                    float w[V];
                    lds<V>(w, src + (kk + q) * N + at(i));
#pragma unroll
                    for (int l = 0; l < V; ++l) v[i + l][q] = w[l];
                }
        }
    }

    // la(m, k) / lb(k, n): address of four consecutive elements (along k for
    // a k-contiguous operand, else along m / n), or nullptr.  K: any; a
    // k-contiguous operand has K a multiple of 4.
    template <bool A_K, bool B_K, typename LA, typename LB>
    static __device__ __forceinline__ void product(float *smem, int K, LA la, LB lb,
                                                   float (&acc)[TM][TN]) {
        float *sa = smem, *sb = smem + STAGES * A_FLOATS;
        const int steps = (K + BK - 1) / BK;
        auto load = [&](int step) {
            if (step < steps) {
                const int k0 = step * BK, s = step % STAGES;
                stage<A_K, BM, VM>(sa + s * A_FLOATS, k0, K, la);
                stage<B_K, BN, VN>(sb + s * B_FLOATS, k0, K, [&](int n, int k) { return lb(k, n); });
            }
            tc::cp_async_commit();  // an empty group past the end keeps the count
        };
        __syncthreads();  // an earlier product's reads are done
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) load(s);
        for (int step = 0; step < steps; ++step) {
            tc::cp_async_wait_group<STAGES - 2>();
            __syncthreads();  // this stage has landed; the one before it has been read
            load(step + STAGES - 1);
            const float *a_s = sa + step % STAGES * A_FLOATS, *b_s = sb + step % STAGES * B_FLOATS;
#pragma unroll(TM <= 2 ? BK / 4 : 2)  // small tiles: all of the step's loads ahead
            for (int kk = 0; kk < (TM <= 2 ? BK : min(BK, K - step * BK)); kk += 4) {
                float a[TM][4], b[TN][4];
                fragment<A_K, BM, TM, VM>(a_s, kk, a, [](int i) { return row(i); });
                fragment<B_K, BN, TN, VN>(b_s, kk, b, [](int j) { return col(j); });
#pragma unroll
                for (int q = 0; q < 4; ++q)  // packed: 5 to 12 % faster than scalar multiply-adds
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int j = 0; j < TN; j += 2) {
                            const float2 r =
                                fma2(make_float2(a[i][q], a[i][q]), make_float2(b[j][q], b[j + 1][q]),
                                     make_float2(acc[i][j], acc[i][j + 1]));
                            acc[i][j] = r.x;
                            acc[i][j + 1] = r.y;
                        }
            }
        }
        tc::cp_async_wait_group<0>();
    }
};

// Raises a kernel's dynamic shared memory limit, once per kernel and device, and asks for
// all of an SM's shared memory: blocks of two kernels share an SM only under one division
// between shared memory and L1 (dWr's blocks beside dx's: T = 16384, d = 128, E = 40 32 us,
// so 28).
template <auto K> inline cudaError_t opt_in(size_t bytes) {
    static OncePerDevice once;
    return once([&](int) {
        cudaError_t err =
            cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (err != cudaSuccess) return err;
        return cudaFuncSetAttribute(K, cudaFuncAttributePreferredSharedMemoryCarveout,
                                    cudaSharedmemCarveoutMaxShared);
    });
}

}  // namespace simt
}  // namespace moe
