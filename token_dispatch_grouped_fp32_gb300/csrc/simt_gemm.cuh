// simt_gemm.cuh -- one block's tile of an fp32 matrix product on the CUDA
// cores: acc[i][j] += sum_k A(m, k) B(k, n), for operands stored either way
// round.  The callers say through functors where four consecutive elements
// lie (ragged segments, transposed weights) or that they are outside the
// matrix; such elements are zeros.
#pragma once

#include <atomic>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace simt {

constexpr int kThreads = 256;
constexpr int BK = 32;      // k per stage
constexpr int kStages = 3;  // stages in flight (cp.async)

__device__ __forceinline__ void copy16_or_zero(float *dst, const float *src) {
    if (src) tc::cp_async16(tc::smem_u32(dst), src);
    else *reinterpret_cast<float4 *>(dst) = make_float4(0.f, 0.f, 0.f, 0.f);
}

// BM x BN tile of 256 threads, TM x TN elements each.  A k-contiguous operand
// is staged as [rows][BK], the other kind as [BK][columns], both in rows of
// 16 bytes more, so that a thread's four elements along the contiguous axis
// are one shared-memory load and a warp's loads fall into different banks.
template <int BM_, int BN_> struct Tile {
    static constexpr int BM = BM_, BN = BN_, TM = BM / 16, TN = BN / 16;
    static constexpr int RG = 16, CG = 16;
    static constexpr int A_FLOATS = BM * BK + 4 * (BM > BK ? BM : BK);
    static constexpr int B_FLOATS = BN * BK + 4 * (BN > BK ? BN : BK);
    static constexpr int SMEM_BYTES = kStages * (A_FLOATS + B_FLOATS) * (int)sizeof(float);

    // Element (i, j) of this thread.  A_K: A is k-contiguous.  Columns are
    // strided where an operand of the tile's products is a k-contiguous B,
    // else consecutive.
    template <bool A_K> static __device__ __forceinline__ int row(int i) {
        const int ty = (int)threadIdx.x / CG;
        return A_K ? ty + i * RG : ty * TM + i;
    }
    template <bool STRIDED> static __device__ __forceinline__ int col(int j) {
        const int tx = (int)threadIdx.x % CG;
        return STRIDED ? tx + j * CG : tx * TN + j;
    }
    static __device__ __forceinline__ void zero(float (&acc)[TM][TN]) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = 0.f;
    }

    // la(m, k) / lb(k, n): address of four consecutive elements (along k for
    // a k-contiguous operand, else along m / n), or nullptr.  K: any; a
    // k-contiguous operand has K a multiple of 4.
    template <bool A_K, bool B_K, bool STRIDED, typename LA, typename LB>
    static __device__ __forceinline__ void product(float *smem, int K, LA la, LB lb,
                                                   float (&acc)[TM][TN]) {
        static_assert(!B_K || STRIDED, "a k-contiguous B needs strided columns");
        constexpr int LDA = (A_K ? BK : BM) + 4, LDB = (B_K ? BK : BN) + 4;
        float *sa = smem, *sb = smem + kStages * A_FLOATS;
        const int steps = (K + BK - 1) / BK;
        auto load = [&](int step) {
            if (step < steps) {
                const int k0 = step * BK, s = step % kStages;
                constexpr int CA = (A_K ? BK : BM) / 4, CB = (B_K ? BK : BN) / 4;  // chunks a row
#pragma unroll
                for (int r = 0; r < (BM * BK / 4 + kThreads - 1) / kThreads; ++r) {
                    const int i = (int)threadIdx.x + r * kThreads;
                    if (BM * BK / 4 % kThreads && i >= BM * BK / 4) break;
                    const int o = i / CA, c = i % CA * 4;
                    const int m = A_K ? o : c, k = k0 + (A_K ? c : o);
                    copy16_or_zero(sa + s * A_FLOATS + o * LDA + c, k < K ? la(m, k) : nullptr);
                }
#pragma unroll
                for (int r = 0; r < (BN * BK / 4 + kThreads - 1) / kThreads; ++r) {
                    const int i = (int)threadIdx.x + r * kThreads;
                    if (BN * BK / 4 % kThreads && i >= BN * BK / 4) break;
                    const int o = i / CB, c = i % CB * 4;
                    const int n = B_K ? o : c, k = k0 + (B_K ? c : o);
                    copy16_or_zero(sb + s * B_FLOATS + o * LDB + c, k < K ? lb(k, n) : nullptr);
                }
            }
            tc::cp_async_commit();  // an empty group past the end keeps the count
        };
        __syncthreads();  // an earlier product's reads are done
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) load(s);
        for (int step = 0; step < steps; ++step) {
            tc::cp_async_wait_group<kStages - 2>();
            __syncthreads();  // this stage has landed; the one before it has been read
            load(step + kStages - 1);
            const float *a_s = sa + step % kStages * A_FLOATS, *b_s = sb + step % kStages * B_FLOATS;
#pragma unroll(TM <= 2 ? BK / 4 : 2)  // small tiles: all of the step's loads ahead
            for (int kk = 0; kk < BK; kk += 4) {
                float a[TM][4], b[TN][4];
                if constexpr (A_K) {
#pragma unroll
                    for (int i = 0; i < TM; ++i)
                        *reinterpret_cast<float4 *>(a[i]) =
                            *reinterpret_cast<const float4 *>(a_s + row<A_K>(i) * LDA + kk);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int i = 0; i < TM; ++i) a[i][q] = a_s[(kk + q) * LDA + row<A_K>(i)];
                }
                if constexpr (B_K) {
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        *reinterpret_cast<float4 *>(b[j]) =
                            *reinterpret_cast<const float4 *>(b_s + col<STRIDED>(j) * LDB + kk);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int j = 0; j < TN; ++j) b[j][q] = b_s[(kk + q) * LDB + col<STRIDED>(j)];
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int j = 0; j < TN; ++j) acc[i][j] = fmaf(a[i][q], b[j][q], acc[i][j]);
            }
        }
        tc::cp_async_wait_group<0>();
    }
};

// Tiles: 64 x 64, or 32 x 32 where the larger would leave SMs without a block.
using Large = Tile<64, 64>;
using Small = Tile<32, 32>;

// Raises a kernel's dynamic shared memory limit, once per kernel and device.
template <auto K> inline cudaError_t opt_in(size_t bytes) {
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    if ((err = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes)) !=
        cudaSuccess)
        return err;
    done[dev].store(true, std::memory_order_relaxed);
    return cudaSuccess;
}

}  // namespace simt
}  // namespace moe
