// gemm_tiles.cuh -- what the tensor-core grouped GEMMs of the forward and the
// backward pass share: which tile shape serves an expert's rows, and the
// coalesced store of a block of accumulator rows.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace tc {

// Lane l holds packed[i] = bf16 pair (columns 2i, 2i+1 of a block of 8*NC
// columns) of row (rbase + l): NC 16-byte chunks of 8 columns, chunk c in
// packed[4c .. 4c+3].  An NC x NC transpose of the chunks within each group
// of NC lanes (butterfly steps over the lane bits below NC) leaves lane
// NC*g + j with chunk j of rows NC*g .. NC*g + NC-1 in the chunk slots, so
// each store instruction writes 16*NC contiguous bytes of each of 32/NC
// rows: for NC = 8, 48 shuffles and 8 16-byte stores per block.  Rows are ld
// elements apart; columns from col_end on are not stored.
template <int NC>
__device__ __forceinline__ void store_rows_transposed(uint32_t (&packed)[4 * NC],
                                                      __nv_bfloat16 *out, int64_t rbase,
                                                      int rows_valid, int col0, int col_end,
                                                      int64_t ld) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int s = NC / 2; s >= 1; s >>= 1) {
        const bool upper = (lane & s) != 0;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (c & s) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t send = upper ? packed[4 * c + q] : packed[4 * (c + s) + q];
                const uint32_t recv = __shfl_xor_sync(0xffffffffu, send, s);
                if (upper) packed[4 * c + q] = recv;
                else packed[4 * (c + s) + q] = recv;
            }
        }
    }
    const int grp = lane / NC;
    const int col = col0 + 8 * (lane % NC);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int r = NC * grp + i;
        if (r < rows_valid && col + 8 <= col_end)
            stg16(out + (rbase + r) * ld + col,
                  make_uint4(packed[4 * i], packed[4 * i + 1], packed[4 * i + 2], packed[4 * i + 3]));
    }
}

// Experts split between the two tile shapes by row count: CTA-pair tiles
// (256 rows) serve an expert when they pad its rows to no more than 1.16x
// what 128-row single-CTA tiles would (the single tile's cost per MMA row,
// measured, from its larger shared-memory fill per SM).  The predicate is
// evaluated on the device from `offsets`, identically by both launches.
constexpr int kAllExperts = 0, kPairExperts = 1, kSingleExperts = 2;
__host__ __device__ __forceinline__ bool pair_tiles_pay(int count) {
    const int pair_rows = (count + 255) / 256 * 256, single_rows = (count + 127) / 128 * 128;
    return pair_rows * 100 <= single_rows * 116;
}
__device__ __forceinline__ int expert_row_tiles(int count, int tile_m, int experts) {
    if (experts != kAllExperts && pair_tiles_pay(count) != (experts == kPairExperts)) return 0;
    return (count + tile_m - 1) / tile_m;
}

constexpr int kPairRowsPerExpert = 512;  // average rows per expert that selects CTA pairs
// Upper bound of the row tiles: sum_e ceil(count_e/TM) <= P/TM + min(E, P).
inline int64_t row_tiles_bound(const Shape &s, int tile_m) {
    const int64_t P = s.P();
    return (P + tile_m - 1) / tile_m + std::min<int64_t>(s.E, P);
}

// Tile shapes of a call.  Pairs when experts average >= 512 rows; 128-row
// single-CTA tiles for small per-expert batches (decode); in between, each
// expert goes to the shape that pads it less (pair_tiles_pay), in two
// launches per product.
enum TileMode { kModePairs, kModeHybrid, kModeSingles };
constexpr int kHybridRowsPerExpert = 64;  // below this average: single-CTA tiles only
inline TileMode tile_mode(const Shape &s) {
    if (s.P() >= (int64_t)kPairRowsPerExpert * s.E) return kModePairs;
    if (s.P() >= (int64_t)kHybridRowsPerExpert * s.E) return kModeHybrid;
    return kModeSingles;
}

}  // namespace tc
}  // namespace moe
