// gemm_bwd_tc.cu -- the matrix products of the layer's gradient for bf16
// activations on the sm_103a tensor cores (tcgen05.mma, accumulators in
// tensor memory, operands staged by TMA): one persistent kernel template.
//
// Experts.  For expert e and row r of its segment, five products in order:
//   DH   dh[r]   = dy[r] Wd[e]^T                      fp32, to the workspace
//   GU   (g, u)  = x[r] Wgu[e], then in the epilogue, with s = sigmoid(g),
//        dgu[r]  = [dh u s (1 + g (1 - s)), dh g s]   bf16, to the workspace
//   DX   dx[r]   = dgu[r] Wgu[e]^T                    bf16
//   DW   dWd[e]  = sum_r h[r]^T dy[r],  dWgu[e] = sum_r x[r]^T dgu[r]   bf16
// 16 P d f floating-point operations in all, 2 of the 8 units (GU) to form
// the gate and up products again.  g, u and dh never leave fp32: the only
// rounding between inputs and outputs is dgu's, which is an operand of the
// last products.
//
// Router (see route_bwd.cu, which splits the fp32 operands into bf16 terms):
//   RX   dx[t]   = add[t] + sum_c A[t][c] B[c]        A [T][K], B [K][d]
//   RW   part[s] = sum over the tokens of split s of A[t]^T x[t]   fp32
//
// Row products (DH, GU, DX, RX) have the forward's tiles: 256 rows x 256 columns
// for a CTA pair (cta_group::2), 128 x 256 for a single CTA, row tiles within
// one expert's segment, the shape chosen by the rows per expert
// (gemm_tiles.cuh).  The weights are read as stored: DH and DX contract over
// their contiguous axis (K-major B), GU and RX over the other (MN-major B; in
// GU a tile's 256 accumulator columns are 128 gate and the 128 matching up
// columns).
//
// Batches whose row products have fewer tiles than SMs take two launches for them
// (SPLIT): GU, which forms dh as well in a third of its accumulator columns, and
// DX, each tile's K axis divided among the CTAs of a cluster, which add up one
// another's accumulators through distributed shared memory in a fixed order.
//
// Weight products (DW, RW) contract over the rows of a segment, so both
// operands are MN-major and the K axis is ragged.  The last K step of a segment may hold
// rows of the next expert (any value, a NaN too): MMAs are issued for whole
// groups of 16 rows only up to the segment's end, and where the end falls
// inside such a group, one warp (the fixer) zeroes the group's remaining rows
// of both operands in shared memory.  For such a stage each CTA's loads
// complete on a barrier of its own; the fixer zeroes, orders its writes before
// the tensor core's reads (proxy fence), and reports the stage on the full
// barrier: an arrival, or in a pair a 16-byte bulk copy of each CTA whose
// bytes complete the leader's barrier.  An expert with no rows has zeros
// written by the epilogue, without an MMA.
//
// What bounds a pair's tile is shared memory: a K step fills 32 KB per CTA and
// the MMAs read 32 KB of it in 512 cycles, all of its 128 bytes a cycle.  Four
// experts of 1024 rows, d = 4096, f = 7168: DX 94 % of the tensor pipe (1654
// TFLOP/s over its last, partial round too), DH and GU 84 to 86 % (1720, 1696),
// DW 75 % (1650): its tiles of 16 K steps pass their 64 KB of output per CTA
// through shared memory as well, 9.2 K cycles at 128 bytes, 10.9 K measured.
// With few rows an expert the bound is memory: the weights read by DH, GU and
// DX, the gradients that DW writes (24 experts of 100 rows, d = f = 2880: dWgu
// 143 us, 5.5 TB/s).  The Mixtral shape (T = 4096) takes 5.2 to 5.5 ms in all,
// 1410 to 1480 TFLOP/s under the power cap, the gpt-oss one (T = 8192) 4.1 to 4.6.
//
// Roles: warp 0 TMA loads, warp 1 tensor memory and MMAs (both one thread),
// warps 2-9 the epilogue (two warps to each 32-lane quarter, half the columns
// each), warp 10 the fixer (weight products).  Two accumulators of 256
// columns: one tile's epilogue overlaps the next tile's products.
//
// Every wait is bounded, as in the forward: one that runs out records a
// timeout, and every role drains its copies and MMAs before the tensor memory
// is released.
#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "gemm_tiles.cuh"
#include "kernels.h"
#include "once.h"
#include "tc_ptx.cuh"

namespace moe {
namespace tc {
namespace {

constexpr int BM = 128, BN = 256, BK = 64, UMMA_K = 16;
constexpr int A_BYTES = BM * BK * 2;
constexpr int ATOM_BYTES = BK * 128;  // MN-major: 64 K-rows x 64 columns
constexpr int TMEM_COLS = 2 * BN;
constexpr int kEpiWarps = 8;
constexpr int MAX_E = 1024;
// K steps of one accumulation in RW.  The tensor cores' fp32 sum drops low
// bits at every step, so long sums lose them in proportion (4096 tokens: dWr
// more than 1e-6 off); sums of kChunk steps are added in fp32 by the epilogue
// (3e-7 to 6e-7 off, and no slower).
constexpr int kChunk = 8;

enum Kind { DH, GU, DX, DW, RX, RW };
// Weight products: both operands MN-major, K the rows of a segment.
template <int KIND> constexpr bool kWeights = KIND == DW || KIND == RW;

template <int KIND> constexpr int threads() { return 32 * (2 + kEpiWarps + (kWeights<KIND> ? 1 : 0)); }

template <int CTAS, int KIND> struct Cfg {
    static constexpr bool PAIR = CTAS == 2;
    static constexpr int TILE_M = BM * CTAS;
    static constexpr int B_COLS = BN / CTAS;  // B columns (or rows of N) held by one CTA
    static constexpr int B_ATOMS = B_COLS / 64;
    static constexpr int B_BYTES = B_COLS * BK * 2;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    // One stage goes to the epilogue's output blocks (OUT_BYTES a warp) where
    // the output leaves by TMA stores: tiles with few K steps, whose time is
    // their epilogue (24 experts of 100 rows: dWgu 163 -> 143 us against
    // transposing shuffles; 32 bytes a lane from registers 231).
    static constexpr bool STAGED = KIND == DW || KIND == RX;
    static constexpr int STAGES = (PAIR ? 6 : 4) - (STAGED ? 1 : 0);
    static constexpr int OUT_BYTES = STAGED ? 32 * 128 : 0;
    static constexpr int OFF_A = 0;
    static constexpr int OFF_B = STAGES * A_BYTES;
    static constexpr int OFF_OUT = OFF_B + STAGES * B_BYTES;
    static constexpr int OFF_BAR = OFF_OUT + kEpiWarps * OUT_BYTES;
    static constexpr int NUM_BARS = 3 * STAGES + 5;  // full, empty, tail; tmem full, empty; drain
    static constexpr int OFF_SIGNAL = (OFF_BAR + NUM_BARS * 8 + 15) / 16 * 16;
    static constexpr int OFF_TMEM = OFF_SIGNAL + 16 * CTAS;
    static constexpr int OFF_ABORT = OFF_TMEM + 4;
    static constexpr int OFF_OFFS = OFF_ABORT + 4;
    static constexpr int OFF_TILE = OFF_OFFS + 4 * (MAX_E + 1);
    static constexpr int SMEM_BYTES = OFF_TILE + 4 * (MAX_E + 1) + 1024;
};

struct Params {
    const int32_t *offsets;
    int E;
    int K;        // reduction length of a row product
    int M;        // weight products: rows of an output
    int N;        // columns of the output (GU: f, gate and up alike)
    int n_tiles;  // column tiles
    int m_tiles;  // weight products: row tiles
    int m_fast;   // weight products: row tiles vary fastest
    int f;        // GU: column offset of the up half
    int a_blocks, b_blocks;  // MN-major A / B through maps of 64-column blocks
    float *dh;               // DH writes, GU reads (see dh_quad)
    __nv_bfloat16 *out;
    const __nv_bfloat16 *add;  // RX: added to the product (may be out), or nullptr
    float *part;               // RW: [segments][N][M]
    int experts;  // which experts a row product's launch serves
    // Ordering against the neighbouring launches (programmatic dependent launch).
    //  release_late: let the next launch start once this one need not wait any
    //    more, so that by then every kernel it depends on has completed.
    //  overlap_prev: this launch does not read the previous one's output, so
    //    it starts without waiting and waits for it only before it exits; its
    //    completion still implies the previous launch's.
    // Else a launch waits at its start and the next one starts at its end: the
    // blocks of a launch resident before their time took slots from this one.
    // Neither order can leave launches waiting for one another, on one stream or
    // several.  A launch starts only when every block of the one before it has
    // started (each has released it or ended), and waits for nothing but that
    // launch; started blocks keep their SMs, and wait inside only for their own
    // cluster, which starts as a whole.  So, from the first launch on, each one
    // that others wait for runs to its end, whatever waits on the other SMs.
    int release_late, overlap_prev;
    DevStatus ds;
};

struct Work {
    int e, row0, rows;  // the rows of segment e that the tile covers (weight products: all)
    int m0, n_blk;      // weight products: first row of the output; column tile
};

// A unit's walk over the tile list: tile, tile + nunits, ...  Weight products
// step (expert, slow tile index, fast tile index) as a mixed-radix number, so
// a tile costs no division: their tiles can be one or two K steps long, and
// the MMA issuer's time between two tiles is then the tensor cores' too.
template <int KIND> struct Walk {
    int tile, total, step;
    int e, slow, fast, de, dslow, dfast, nslow, nfast;
    __device__ __forceinline__ Walk(const Params &p, int unit, int nunits, int total_)
        : tile(unit), total(total_), step(nunits) {
        if constexpr (kWeights<KIND>) {
            nfast = p.m_fast ? p.m_tiles : p.n_tiles;
            nslow = p.m_fast ? p.n_tiles : p.m_tiles;
            e = unit / (nfast * nslow);
            slow = unit / nfast - e * nslow;
            fast = unit % nfast;
            de = nunits / (nfast * nslow);
            dslow = nunits / nfast - de * nslow;
            dfast = nunits % nfast;
        }
    }
    __device__ __forceinline__ bool more() const { return tile < total; }
    __device__ __forceinline__ void next() {
        tile += step;
        if constexpr (kWeights<KIND>) {
            fast += dfast;
            slow += dslow;
            e += de;
            if (fast >= nfast) {
                fast -= nfast;
                ++slow;
            }
            if (slow >= nslow) {
                slow -= nslow;
                ++e;
            }
        }
    }
    __device__ __forceinline__ Work at(const int *s_off, const int *s_tile, const Params &p,
                                       int tile_m) const {
        Work w;
        if constexpr (kWeights<KIND>) {
            w.e = e;
            w.n_blk = p.m_fast ? slow : fast;
            w.m0 = (p.m_fast ? fast : slow) * tile_m;
            w.row0 = s_off[e];
            w.rows = s_off[e + 1] - w.row0;
        } else {
            const int g = tile / p.n_tiles;
            int lo = 0, hi = p.E - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_tile[mid] <= g) lo = mid; else hi = mid - 1;
            }
            const int mt = s_tile[lo + 1] - s_tile[lo];
            const int r = tile - s_tile[lo] * p.n_tiles;
            w.e = lo;
            w.n_blk = r / mt;
            w.row0 = s_off[lo] + (r % mt) * tile_m;
            w.rows = min(tile_m, s_off[lo + 1] - w.row0);
            w.m0 = 0;
        }
        return w;
    }
};

// dh in the workspace: groups of up to 32 rows counted from a segment's
// start (both tile shapes are whole groups), each group's f x rows floats
// ordered by 16-byte column quad, then row, so that a warp whose lanes hold
// the rows writes and reads 512 contiguous bytes per instruction.  Group g of
// `rows` rows from row r0 starts at r0 * f.
__device__ __forceinline__ float4 *dh_quad(float *dh, int64_t r0, int f, int rows, int col, int lane) {
    return reinterpret_cast<float4 *>(dh + r0 * f + (int64_t)col * rows) + lane;
}

// 32 columns of lane's row, zeros outside the rows and columns there are.
__device__ __forceinline__ void load_dh(const Params &p, int64_t r0, int rows, int col, int lane,
                                        float (&dh)[32]) {
#pragma unroll
    for (int v = 0; v < 8; ++v) {
        float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
        const int n = col + 4 * v;
        if (lane < rows && n < p.N) q = __ldcg(dh_quad(p.dh, r0, p.N, rows, n, lane));
        dh[4 * v] = q.x;
        dh[4 * v + 1] = q.y;
        dh[4 * v + 2] = q.z;
        dh[4 * v + 3] = q.w;
    }
}

__device__ __forceinline__ void gate_gradient(float g, float u, float dh, float &dg, float &du) {
    const float s = __fdividef(1.f, 1.f + __expf(-g));
    const float t = dh * s;
    du = t * g;
    dg = t * u * fmaf(g, 1.f - s, 1.f);
}

__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&v);
}

// Sum over the CTAs of a cluster of 32 columns, from column col0, of this lane's
// row of their accumulators (each at `dump`, [BN columns][BM rows]), in the order
// of the CTAs.
__device__ __forceinline__ void sum_cluster(uint32_t dump, int ctas, int col0, int row, float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0.f;
    for (int c = 0; c < ctas; ++c) {
        const uint32_t at = map_to_rank(dump, c) + 4 * (col0 * BM + row);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] += ld_cluster(at + 4 * BM * i);
    }
}

// SPLIT (GU, DX): a cluster of single CTAs serves one tile, each CTA a part of K;
// the launch has a cluster for every tile there can be.
template <int CTAS, int KIND, bool SPLIT>
__global__ void __launch_bounds__(threads<KIND>(), 1)
gemm_bwd_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmB2,
                   Params p) {
    using C = Cfg<CTAS, KIND>;
    constexpr bool PAIR = C::PAIR;
    constexpr int STAGES = C::STAGES;
    constexpr bool A_MN = kWeights<KIND>, B_MN = KIND != DH && KIND != DX;
    constexpr uint32_t IDESC = idesc_bf16_ab(C::TILE_M, BN, A_MN, B_MN);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    const uint32_t base_s = (raw_s + 1023u) & ~1023u;
    uint8_t *base = smem_raw + (base_s - raw_s);
    const uint32_t bar_full = base_s + C::OFF_BAR;      // [STAGES] (a pair uses the leader's)
    const uint32_t bar_empty = bar_full + 8 * STAGES;   // [STAGES]
    const uint32_t bar_tail = bar_empty + 8 * STAGES;   // [STAGES] this CTA's loads of a cut stage
    const uint32_t bar_tfull = bar_tail + 8 * STAGES;   // [2]
    const uint32_t bar_tempty = bar_tfull + 16;         // [2] (a pair uses the leader's)
    const uint32_t bar_drain = bar_tempty + 16;
    volatile uint32_t *s_tmem = reinterpret_cast<volatile uint32_t *>(base + C::OFF_TMEM);
    volatile int *s_abort = reinterpret_cast<volatile int *>(base + C::OFF_ABORT);
    int *s_off = reinterpret_cast<int *>(base + C::OFF_OFFS);
    int *s_tile = reinterpret_cast<int *>(base + C::OFF_TILE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = p.E;
    const uint32_t rank = PAIR ? cluster_rank() : 0u;  // of the tile's rows
    const bool leader = rank == 0;
    // GU forms dh too: 128 columns of dy Wd^T beside the gate and up ones,
    // from K steps of their own after the others (A through tmOut, B tmB2).
    constexpr bool WITH_DH = SPLIT && KIND == GU;
    constexpr int DUMP_COLS = BN + (WITH_DH ? BN / 2 : 0);
    static_assert(!SPLIT || (!PAIR && (KIND == GU || KIND == DX) && C::OFF_BAR >= 4 * BM * DUMP_COLS &&
                             DUMP_COLS <= TMEM_COLS),
                  "the accumulators of a split product take the stages' place");
    const int parts = SPLIT ? (int)cluster_size() : 1, part = SPLIT ? (int)cluster_rank() : 0;
    const int unit = (int)blockIdx.x / (SPLIT ? parts : CTAS);
    const int nunits = (int)gridDim.x / (SPLIT ? parts : CTAS);
    const uint32_t sig_full = PAIR ? map_to_rank(bar_full, 0) : bar_full;
    const uint32_t sig_tempty = PAIR ? map_to_rank(bar_tempty, 0) : bar_tempty;

    if (threadIdx.x == 0) {
        *s_abort = 0;
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(bar_full + 8 * i, 1);
            mbar_init(bar_empty + 8 * i, 1);
            mbar_init(bar_tail + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_tfull + 8 * i, 1);
            mbar_init(bar_tempty + 8 * i, kEpiWarps * CTAS);
        }
        mbar_init(bar_drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<CTAS>(base_s + C::OFF_TMEM, TMEM_COLS);
    if (!p.overlap_prev) pdl_wait();
    if (p.release_late) pdl_release();
    for (int e = threadIdx.x; e <= E; e += (int)blockDim.x) s_off[e] = __ldcg(p.offsets + e);
    __syncthreads();
    if (!kWeights<KIND> && warp == 2) {  // row tiles of the experts before each expert
        const int per = (E + 31) / 32;
        const int e0 = min(E, lane * per), e1 = min(E, e0 + per);
        int local = 0;
        for (int e = e0; e < e1; ++e)
            local += expert_row_tiles(s_off[e + 1] - s_off[e], C::TILE_M, p.experts);
        int incl = local;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        int run = incl - local;
        for (int e = e0; e < e1; ++e) {
            s_tile[e] = run;
            run += expert_row_tiles(s_off[e + 1] - s_off[e], C::TILE_M, p.experts);
        }
        if (lane == 31) s_tile[E] = incl;
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();
    tc_fence_after();

    const uint32_t tmem_base = *s_tmem;
    const int total = kWeights<KIND> ? E * p.m_tiles * p.n_tiles : s_tile[E] * p.n_tiles;
    // K steps of a row product's tile that are this CTA's
    const int nk_all = (p.K + BK - 1) / BK;
    const int ks_row = nk_all * part / parts, nk_row = nk_all * (part + 1) / parts;
    const int nk_dh = WITH_DH ? nk_row - ks_row : 0;  // ... and as many again of dh
    // Past-the-end K step of a tile, and whether its last one needs the fixer
    auto ksteps = [&](const Work &w) { return kWeights<KIND> ? (w.rows + BK - 1) / BK : nk_row; };
    auto cut = [&](const Work &w) { return kWeights<KIND> && (w.rows & 15) != 0; };

    if (warp == 0) {
        // ------------------------- TMA producer -------------------------
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            uint32_t issued = 0, last_par = 0;   // full barriers armed here: ever / last parity
            uint32_t tissued = 0, tail_par = 0;  // tail barriers: ever / parity of the next phase
            bool ok = true;
            for (Walk<KIND> wk(p, unit, nunits, total); wk.more() && ok; wk.next()) {
                const Work w = wk.at(s_off, s_tile, p, C::TILE_M);
                const int nk = ksteps(w) + nk_dh;
                for (int ks = ks_row; ks < nk; ++ks) {
                    if (!wait_bounded(bar_empty + 8 * s, ph ^ 1u, p.ds, s_abort)) {
                        ok = false;
                        break;
                    }
                    const bool tail = cut(w) && ks == nk - 1;
                    if (leader) {
                        if (PAIR || !tail)  // (a single CTA's fixer arrives itself)
                            mbar_arrive_expect_tx(bar_full + 8 * s,
                                                  (tail ? 16
                                                   : WITH_DH && ks >= nk_row ? A_BYTES + C::B_BYTES / 2
                                                                             : C::STAGE_BYTES) * CTAS);
                        issued |= 1u << s;
                        last_par = (last_par & ~(1u << s)) | (ph << s);
                    }
                    uint32_t fb = sig_full + 8 * s;
                    if (kWeights<KIND> && tail) {
                        mbar_arrive_expect_tx(bar_tail + 8 * s, C::STAGE_BYTES);
                        tissued |= 1u << s;
                        tail_par ^= 1u << s;
                        fb = PAIR ? map_to_rank(bar_tail + 8 * s, rank) : bar_tail + 8 * s;
                    }
                    const int k0 = ks * BK;
                    const uint32_t adst = base_s + C::OFF_A + s * A_BYTES;
                    const uint32_t bdst = base_s + C::OFF_B + s * C::B_BYTES;
                    if constexpr (kWeights<KIND>) {
                        const int kr = w.row0 + k0, mc = w.m0 + (int)rank * BM;
                        if (p.a_blocks) {
                            tma_load_4d<CTAS>(adst, &tmA, 0, kr, mc >> 6, 0, fb);
                        } else {
                            tma_load_3d<CTAS>(adst, &tmA, mc, kr, 0, fb);
                            tma_load_3d<CTAS>(adst + ATOM_BYTES, &tmA, mc + 64, kr, 0, fb);
                        }
                        const int nc = w.n_blk * BN + (int)rank * C::B_COLS;
                        if (p.b_blocks) {
#pragma unroll
                            for (int a = 0; a < C::B_ATOMS; a += 2)
                                tma_load_4d<CTAS>(bdst + a * ATOM_BYTES, &tmB, 0, kr, (nc >> 6) + a, 0, fb);
                        } else {
#pragma unroll
                            for (int a = 0; a < C::B_ATOMS; ++a)
                                tma_load_3d<CTAS>(bdst + a * ATOM_BYTES, &tmB, nc + 64 * a, kr, 0, fb);
                        }
                    } else if (WITH_DH && ks >= nk_row) {
                        const int kd = (ks - nk_dh) * BK;
                        tma_load_2d<CTAS>(adst, &tmOut, kd, w.row0, fb);
                        tma_load_3d<CTAS>(bdst, &tmB2, kd, w.n_blk * (BN / 2), w.e, fb);
                    } else {
                        tma_load_2d<CTAS>(adst, &tmA, k0, w.row0 + (int)rank * BM, fb);
                        if constexpr (KIND == GU) {
                            // gate columns, then the matching up columns (offset f)
                            const int g0 = w.n_blk * (BN / 2);
#pragma unroll
                            for (int a = 0; a < C::B_ATOMS; a += 2) {
                                const int nc = g0 + ((PAIR ? (int)rank : a / 2) ? p.f : 0);
                                if (p.b_blocks) {
                                    tma_load_4d<CTAS>(bdst + a * ATOM_BYTES, &tmB, 0, k0, nc >> 6, w.e, fb);
                                } else {
                                    tma_load_3d<CTAS>(bdst + a * ATOM_BYTES, &tmB, nc, k0, w.e, fb);
                                    tma_load_3d<CTAS>(bdst + (a + 1) * ATOM_BYTES, &tmB, nc + 64, k0, w.e, fb);
                                }
                            }
                        } else if constexpr (KIND == RX) {
                            const int nc = w.n_blk * BN + (int)rank * C::B_COLS;
#pragma unroll
                            for (int a = 0; a < C::B_ATOMS; a += 2) {
                                if (p.b_blocks) {
                                    tma_load_4d<CTAS>(bdst + a * ATOM_BYTES, &tmB, 0, k0, (nc >> 6) + a, 0, fb);
                                } else {
                                    tma_load_3d<CTAS>(bdst + a * ATOM_BYTES, &tmB, nc + 64 * a, k0, 0, fb);
                                    tma_load_3d<CTAS>(bdst + (a + 1) * ATOM_BYTES, &tmB, nc + 64 * a + 64, k0, 0, fb);
                                }
                            }
                        } else {
                            tma_load_3d<CTAS>(bdst, &tmB, k0, w.n_blk * BN + (int)rank * C::B_COLS, w.e, fb);
                        }
                    }
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            // drain: every phase armed here must have received all of its bytes
            for (int i = 0; i < STAGES; ++i) {
                volatile int never = 0;
                if (kWeights<KIND> && ((tissued >> i) & 1u) &&
                    !wait_bounded(bar_tail + 8 * i, ((tail_par >> i) & 1u) ^ 1u, p.ds, &never,
                                  drain_limit(p.ds)))
                    break;
                if (((issued >> i) & 1u) &&
                    !wait_bounded(bar_full + 8 * i, (last_par >> i) & 1u, p.ds, &never,
                                  drain_limit(p.ds)))
                    break;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------- MMA issuer ---------------------------
        if (leader && lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            int it = 0;
            bool ok = true;
            // K-major operands: rows of 128 bytes, 8-row groups 1024 B apart, a
            // K step of 16 elements 32 bytes along the row.  MN-major: 64-column
            // atoms 8 KB apart, 8-row K groups 1024 B apart, a K step of 16 rows
            // 2 KB.  Stages and K steps only move the start address.
            const uint64_t adesc0 = smem_desc_sw128(base_s + C::OFF_A, A_MN ? ATOM_BYTES : 16, 1024);
            const uint64_t bdesc0 = smem_desc_sw128(base_s + C::OFF_B, B_MN ? ATOM_BYTES : 16, 1024);
            const uint64_t bdesc_dh = smem_desc_sw128(base_s + C::OFF_B, 16, 1024);
            constexpr uint32_t IDESC_DH = idesc_bf16_ab(C::TILE_M, BN / 2, false, false);
            constexpr uint32_t ASTEP = A_MN ? 2048 : 32, BSTEP = B_MN ? 2048 : 32;
            if (p.ds.inject_wait_timeout) ok = wait_bounded(bar_drain, 0, p.ds, s_abort);
            for (Walk<KIND> wk(p, unit, nunits, total); wk.more() && ok; wk.next()) {
                int nk = nk_row, last = BK / UMMA_K;  // MMAs of the last K step
                if constexpr (kWeights<KIND>) {
                    const Work w = wk.at(s_off, s_tile, p, C::TILE_M);
                    nk = ksteps(w);
                    last = (w.rows - (nk - 1) * BK + UMMA_K - 1) / UMMA_K;
                }
                int ks = ks_row;
                do {  // accumulations: one, or in RW one per kChunk steps
                    const int acc = it & 1;
                    const uint32_t aph = (uint32_t)(it >> 1) & 1u;
                    ++it;
                    if (!wait_bounded(bar_tempty + 8 * acc, aph ^ 1u, p.ds, s_abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
                    const int ks0 = ks, ks1 = KIND == RW ? min(nk, ks + kChunk) : nk + nk_dh;
                    for (; ks < ks1; ++ks) {
                        // a cut stage of a pair is reported from the peer CTA too
                        if (!wait_bounded<PAIR && kWeights<KIND>>(bar_full + 8 * s, ph, p.ds, s_abort)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t a_st = adesc0 + (uint64_t)((s * A_BYTES) >> 4);
                        const uint64_t b_st = bdesc0 + (uint64_t)((s * C::B_BYTES) >> 4);
                        const int n = kWeights<KIND> && ks == nk - 1 ? last : BK / UMMA_K;
                        if (WITH_DH && ks >= nk_row) {
                            const uint64_t b_dh = bdesc_dh + (uint64_t)((s * C::B_BYTES) >> 4);
#pragma unroll
                            for (int kk = 0; kk < BK / UMMA_K; ++kk)
                                mma_bf16<CTAS>(d_tmem + BN, a_st + (uint64_t)((kk * ASTEP) >> 4),
                                               b_dh + (uint64_t)((kk * 32) >> 4), IDESC_DH,
                                               ((ks - nk_row) | kk) != 0 ? 1u : 0u);
                        } else
#pragma unroll
                        for (int kk = 0; kk < BK / UMMA_K; ++kk)
                            if (!kWeights<KIND> || kk < n)
                                mma_bf16<CTAS>(d_tmem, a_st + (uint64_t)((kk * ASTEP) >> 4),
                                               b_st + (uint64_t)((kk * BSTEP) >> 4), IDESC,
                                               ((ks - ks0) | kk) != 0 ? 1u : 0u);
                        mma_commit_all<CTAS>(bar_empty + 8 * s);
                        if (++s == STAGES) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                    if (!ok) break;
                    mma_commit_all<CTAS>(bar_tfull + 8 * acc);
                } while (ks < nk);
            }
            mma_commit_local<CTAS>(bar_drain);
            volatile int never = 0;
            wait_bounded(bar_drain, 0, p.ds, &never, drain_limit(p.ds));
        }
        __syncwarp();
    } else if (warp < 2 + kEpiWarps) {
        // --------------------------- epilogue ----------------------------
        const int quarter = warp & 3;          // tensor-memory lanes of this warp
        const int half = (warp - 2) >> 2;      // its half of the columns
        const int wrow0 = (int)rank * BM + quarter * 32;
        int it = 0;
        bool ok = true;
        for (Walk<KIND> wk(p, unit, nunits, total); wk.more(); wk.next()) {
            const Work w = wk.at(s_off, s_tile, p, C::TILE_M);
            uint32_t t_row = 0;
            int acc = 0;
            // the next accumulator, complete
            auto ready = [&]() {
                acc = it & 1;
                const uint32_t aph = (uint32_t)(it >> 1) & 1u;
                ++it;
                ok = __all_sync(0xffffffffu, wait_bounded(bar_tfull + 8 * acc, aph, p.ds, s_abort));
                tc_fence_after();
                t_row = tmem_base + (uint32_t)(acc * BN) + ((uint32_t)(quarter * 32) << 16);
            };
            const int have = kWeights<KIND> ? p.M - w.m0 : w.rows;
            const int rv = max(0, min(32, have - wrow0));  // rows of this warp
            // The accumulator is handed back as soon as it is in registers.  The
            // arrival passes on no memory contents, only that the loads from
            // tensor memory are complete, so in a pair it is a relaxed one: a
            // release at cluster scope would wait for the warp's global stores
            // (Qwen3 shape, T = 2048, Zipf: 803 us, relaxed 671).
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR) mbar_arrive_cluster_relaxed(sig_tempty + 8 * acc);
                    else mbar_arrive(bar_tempty + 8 * acc);
                }
            };
            // Outputs that end with their matrix leave 32 rows x 64 columns at a
            // time, through shared memory (128-byte swizzle) and a TMA store.
            const uint32_t out_buf = base_s + C::OFF_OUT + (warp - 2) * C::OUT_BYTES;
            auto store_block = [&](int col, int row, int e) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&tmOut, out_buf, col, row, e);
                    bulk_commit();
                }
            };
            if constexpr (KIND != RW) {
                ready();
                if (!ok) break;
            }
            if constexpr (SPLIT) {  // the accumulator to shared memory, for the cluster
                if (rv > 0)
#pragma unroll
                    for (int c = half * (DUMP_COLS / 2); c < (half + 1) * (DUMP_COLS / 2); c += 32) {
                        uint32_t y[32];
                        tmem_ld32(t_row + c, y);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            reinterpret_cast<uint32_t *>(base)[(c + i) * BM + wrow0 + lane] = y[i];
                    }
            } else if constexpr (KIND == DH) {
                const int64_t r0 = w.row0 + wrow0;
                const int n0 = w.n_blk * BN + half * (BN / 2);
                uint32_t y[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(t_row + half * (BN / 2) + 32 * c, y[c]);
                tmem_ld_wait();
                release();
                if (lane < rv)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int v = 0; v < 8; ++v) {
                            const int n = n0 + 32 * c + 4 * v;
                            if (n < p.N)
                                *dh_quad(p.dh, r0, p.N, rv, n, lane) = make_float4(
                                    __uint_as_float(y[c][4 * v]), __uint_as_float(y[c][4 * v + 1]),
                                    __uint_as_float(y[c][4 * v + 2]), __uint_as_float(y[c][4 * v + 3]));
                        }
            } else if constexpr (KIND == GU) {
                const int64_t r0 = w.row0 + wrow0;
                const int n0 = w.n_blk * (BN / 2) + half * (BN / 4);
                uint32_t pg[32], pu[32];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float dh[32];
                    load_dh(p, r0, rv, n0 + 32 * c, lane, dh);
                    uint32_t g[32], u[32];
                    tmem_ld32(t_row + half * (BN / 4) + 32 * c, g);
                    tmem_ld32(t_row + BN / 2 + half * (BN / 4) + 32 * c, u);
                    tmem_ld_wait();
                    if (c == 1) release();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float dg[2], du[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            gate_gradient(__uint_as_float(g[2 * i + j]), __uint_as_float(u[2 * i + j]),
                                          dh[2 * i + j], dg[j], du[j]);
                        pg[16 * c + i] = pack2(dg[0], dg[1]);
                        pu[16 * c + i] = pack2(du[0], du[1]);
                    }
                }
                const int64_t ld = 2 * (int64_t)p.f;
                store_rows_transposed<8>(pg, p.out, r0, rv, n0, p.N, ld);
                store_rows_transposed<8>(pu, p.out + p.f, r0, rv, n0, p.N, ld);
            } else if constexpr (KIND == RW) {
                // accumulations of kChunk steps, added here in fp32
                const int n0 = w.n_blk * BN + half * (BN / 2);
                float sum[128];
#pragma unroll
                for (int c = 0; c < 128; ++c) sum[c] = 0.f;
                const int nk = ksteps(w);
                for (int ks = 0; ks == 0 || ks < nk; ks += kChunk) {
                    ready();
                    if (!ok) break;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t y[32];
                        tmem_ld32(t_row + half * (BN / 2) + 32 * c, y);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) sum[32 * c + i] += __uint_as_float(y[i]);
                    }
                    release();
                }
                if (!ok) break;
                // a column of the product is 32 consecutive floats of the warp's lanes
                float *o = p.part + ((int64_t)w.e * p.N + n0) * p.M + w.m0 + wrow0 + lane;
                if (lane < rv)
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (n0 + c < p.N) o[(int64_t)c * p.M] = sum[c];
            } else if constexpr (KIND == RX) {
                const int n0 = w.n_blk * BN + half * (BN / 2);
                uint32_t y[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(t_row + half * (BN / 2) + 32 * c, y[c]);
                tmem_ld_wait();
                release();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int n = n0 + 64 * c;
                    if (rv == 0 || n >= p.N) break;  // warp-uniform
                    if (lane == 0) bulk_wait_read();  // the buffer's last store has read it
                    __syncwarp();
                    if (p.add) {  // the block of the other gradient, to where its lanes read it
#pragma unroll
                        for (int v = 0; v < 8; ++v) {
                            const int r = 4 * v + (lane >> 3), q = lane & 7;
                            if (r < rv && n + 8 * q < p.N)
                                cp_async16(out_buf + r * 128 + ((q ^ (r & 7)) << 4),
                                           p.add + ((int64_t)w.row0 + wrow0 + r) * p.N + n + 8 * q);
                        }
                        cp_async_wait_all();
                        __syncwarp();
                    }
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        const uint32_t at = out_buf + lane * 128 + ((v ^ (lane & 7)) << 4);
                        float f[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            f[i] = __uint_as_float(y[2 * c + v / 4][8 * (v % 4) + i]);
                        if (p.add) {
                            float t[8];
                            unpack16(lds16(at), t, static_cast<const __nv_bfloat16 *>(nullptr));
#pragma unroll
                            for (int i = 0; i < 8; ++i) f[i] += t[i];
                        }
                        sts16(at, pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]),
                              pack2(f[6], f[7]));
                    }
                    store_block(n, w.row0 + wrow0, 0);
                }
            } else {
                const bool none = KIND == DW && w.rows == 0;
                const int n0 = w.n_blk * BN + half * (BN / 2);
                uint32_t packed[2][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t y[32];
                    tmem_ld32(t_row + half * (BN / 2) + 32 * c, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        packed[c / 2][16 * (c & 1) + i] =
                            none ? 0u : pack2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]));
                }
                release();
                if constexpr (KIND == DX) {  // a segment's rows end inside a tile: predicated stores
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        store_rows_transposed<8>(packed[c], p.out, w.row0 + wrow0, rv, n0 + 64 * c,
                                                 p.N, p.N);
                } else {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if (rv == 0 || n0 + 64 * c >= p.N) break;  // warp-uniform
                        if (lane == 0) bulk_wait_read();  // the buffer's last store has read it
                        __syncwarp();
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            sts16(out_buf + lane * 128 + ((v ^ (lane & 7)) << 4), packed[c][4 * v],
                                  packed[c][4 * v + 1], packed[c][4 * v + 2], packed[c][4 * v + 3]);
                        store_block(n0 + 64 * c, w.m0 + wrow0, w.e);
                    }
                }
            }
        }
        if (C::STAGED && lane == 0) bulk_wait_all();  // before the shared memory is released
        __syncwarp();
    } else if constexpr (kWeights<KIND>) {
        // ---------------------------- fixer ------------------------------
        // Zeroes rows [rem, rem rounded up to 16) of both operands in the last
        // K step of a segment whose end cuts a group of 16 rows.  A K row is
        // 128 bytes in each 64-column atom; the swizzle moves bytes within it.
        int s = 0;
        uint32_t tail_par = 0;
        const uint32_t slot = PAIR ? map_to_rank(base_s + C::OFF_SIGNAL + 16 * rank, 0) : 0u;
        for (Walk<KIND> wk(p, unit, nunits, total); wk.more(); wk.next()) {
            const Work w = wk.at(s_off, s_tile, p, C::TILE_M);
            const int nk = ksteps(w);
            s = (s + nk) % STAGES;
            if (!cut(w)) continue;
            const int st = (s + STAGES - 1) % STAGES;  // the tile's last stage
            // (this warp may reach the wait long before the stage is loaded)
            if (!__all_sync(0xffffffffu, wait_bounded(bar_tail + 8 * st, (tail_par >> st) & 1u, p.ds,
                                                      s_abort, drain_limit(p.ds))))
                break;
            tail_par ^= 1u << st;
            const int rem = w.rows - (nk - 1) * BK;
            const int pieces = 8 * (((rem + 15) & ~15) - rem);  // 16-byte pieces per atom
            uint8_t *a = base + C::OFF_A + st * A_BYTES + rem * 128;
            uint8_t *b = base + C::OFF_B + st * C::B_BYTES + rem * 128;
            for (int i = lane; i < pieces * (2 + C::B_ATOMS); i += 32) {
                const int atom = i / pieces, o = (i - atom * pieces) * 16;
                uint8_t *q = atom < 2 ? a + atom * ATOM_BYTES + o : b + (atom - 2) * ATOM_BYTES + o;
                *reinterpret_cast<uint4 *>(q) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (PAIR)
                    bulk_copy_to_cluster(slot, base_s + C::OFF_A + st * A_BYTES, 16, sig_full + 8 * st);
                else
                    mbar_arrive(bar_full + 8 * st);
            }
        }
        __syncwarp();
    }

    if constexpr (SPLIT) {
        // Every CTA's accumulators lie in its shared memory now, in the stages' place
        // (a cluster has one tile at most, so no more loads come).  Each adds up and
        // stores 32-column blocks of the tile: block b (GU: b of the gate columns, of
        // the up and of the dh ones) is CTA b mod parts' task.
        cluster_sync();
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const Walk<KIND> wk(p, unit, nunits, total);
        if (warp >= 2 && wk.more() && *s_abort == 0) {
            const Work w = wk.at(s_off, s_tile, p, C::TILE_M);
            const int rv = max(0, min(32, w.rows - quarter * 32)), row = quarter * 32 + lane;
            const int64_t r0 = w.row0 + quarter * 32;
            constexpr int BLOCKS = BN / 32 / (KIND == GU ? 2 : 1);
            for (int b = half * (BLOCKS / 2); b < (half + 1) * (BLOCKS / 2); ++b) {
                const int n = (w.n_blk * BLOCKS + b) * 32;
                if (b % parts != part || rv == 0 || n >= p.N) continue;  // warp-uniform
                float y[32];
                sum_cluster(base_s, parts, 32 * b, row, y);
                if constexpr (KIND == GU) {
                    float u[32], dh[32];
                    sum_cluster(base_s, parts, BN / 2 + 32 * b, row, u);
                    sum_cluster(base_s, parts, BN + 32 * b, row, dh);
                    uint32_t pg[16], pu[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float dg[2], du[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            gate_gradient(y[2 * i + j], u[2 * i + j], dh[2 * i + j], dg[j], du[j]);
                        pg[i] = pack2(dg[0], dg[1]);
                        pu[i] = pack2(du[0], du[1]);
                    }
                    const int64_t ld = 2 * (int64_t)p.f;
                    store_rows_transposed<4>(pg, p.out, r0, rv, n, p.N, ld);
                    store_rows_transposed<4>(pu, p.out + p.f, r0, rv, n, p.N, ld);
                } else {
                    uint32_t packed[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) packed[i] = pack2(y[2 * i], y[2 * i + 1]);
                    store_rows_transposed<4>(packed, p.out, r0, rv, n, p.N, p.N);
                }
            }
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR || SPLIT) cluster_sync();  // (SPLIT: the others have read this CTA's memory)
    tc_fence_after();
    if (warp == 1) tmem_dealloc<CTAS>(tmem_base, TMEM_COLS);
    if (p.overlap_prev) pdl_wait();
}

// ------------------------------ host side ----------------------------------
template <int CTAS, int KIND>
cudaLaunchConfig_t launch_config(unsigned grid, int cluster, cudaStream_t st, cudaLaunchAttribute *attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads<KIND>(), 1, 1);
    cfg.dynamicSmemBytes = (Cfg<CTAS, KIND>::SMEM_BYTES);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

template <int CTAS, int KIND> cudaError_t prepare(int *resident) {
    cudaError_t err = cudaFuncSetAttribute(gemm_bwd_tc_kernel<CTAS, KIND, false>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (Cfg<CTAS, KIND>::SMEM_BYTES));
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = launch_config<CTAS, KIND>(CTAS, CTAS, nullptr, attr);
    int n = 0;
    if ((err = cudaOccupancyMaxActiveClusters(&n, gemm_bwd_tc_kernel<CTAS, KIND, false>, &cfg)) !=
        cudaSuccess)
        return err;
    *resident = std::min(*resident, n);
    return cudaSuccess;
}

template <int CTAS> cudaError_t prepare_all(int *resident) {
    *resident = INT32_MAX;
    cudaError_t err;
    if ((err = prepare<CTAS, DH>(resident)) != cudaSuccess ||
        (err = prepare<CTAS, GU>(resident)) != cudaSuccess ||
        (err = prepare<CTAS, DX>(resident)) != cudaSuccess ||
        (err = prepare<CTAS, DW>(resident)) != cudaSuccess ||
        (err = prepare<CTAS, RX>(resident)) != cudaSuccess ||
        (err = prepare<CTAS, RW>(resident)) != cudaSuccess)
        return err;
    return *resident >= 1 ? cudaSuccess : cudaErrorInvalidConfiguration;
}

struct DeviceInfo {
    std::atomic<int> units[3];  // resident single CTAs [1] and pairs [2]
};

template <int CTAS, int KIND>
cudaError_t launch_one(int units, int64_t tiles, const CUtensorMap &a, const CUtensorMap &b,
                       const CUtensorMap &out, const Params &p, cudaStream_t st) {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg =
        launch_config<CTAS, KIND>(CTAS * (unsigned)std::min<int64_t>(units, tiles), CTAS, st, attr);
    return cudaLaunchKernelEx(&cfg, gemm_bwd_tc_kernel<CTAS, KIND, false>, a, b, out, b, p);
}

// Row products with so few tiles that SMs would idle: each tile on a cluster of up
// to eight CTAs, with at least eight K steps each (shorter parts cost more in the
// sum than they save: T = 1024, E = 1, d = f = 256 45 us to 48), and dh in GU's launch.
// Five launches took (d = 2048, f = 768, E = 8, k = 2) at T = 1 67 us, now 45 with the
// weight products beside them; T = 64 77 and 62; T = 24, d = 2880, f = 168, E = 3 63 and 31;
// T = 178, d = 256, f = 2712 74 and 36.
template <int KIND> cudaError_t prepare_split() {
    return cudaFuncSetAttribute(gemm_bwd_tc_kernel<1, KIND, true>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (Cfg<1, KIND>::SMEM_BYTES));
}
// CTAs a tile, or 0 (fewer than `least`, or the tiles more than one round).
int split_parts(const Shape &s, const DeviceInfo &d, int n_tiles, int K, int least) {
    const int64_t steps = (K + BK - 1) / BK, tiles = row_tiles_bound(s, BM) * n_tiles;
    const int64_t parts = std::min<int64_t>({8, d.units[1] / tiles, std::max<int64_t>(1, steps / 8)});
    return parts >= least ? (int)parts : 0;
}
template <int KIND>
cudaError_t launch_split(const Shape &s, int parts, const CUtensorMap &a, const CUtensorMap &b,
                         const CUtensorMap &a2, const CUtensorMap &b2, Params p, cudaStream_t st) {
    p.experts = kAllExperts;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = launch_config<1, KIND>(
        (unsigned)(parts * row_tiles_bound(s, BM) * p.n_tiles), parts, st, attr);
    return cudaLaunchKernelEx(&cfg, gemm_bwd_tc_kernel<1, KIND, true>, a, b, a2, b2, p);
}

// A row product over all experts: one launch, or one per tile shape.  The
// maps' boxes differ between the shapes (KBox: B is K-major).
template <int KIND, typename MapB>
cudaError_t launch_rows(const Shape &s, const DeviceInfo &d, const CUtensorMap &a, MapB map_b,
                        Params p, cudaStream_t st) {
    const TileMode mode = tile_mode(s);
    CUtensorMap b;
    cudaError_t err = cudaSuccess;
    p.experts = kAllExperts;
    const int late = p.release_late;
    if (mode != kModeSingles) {
        if (!map_b(&b, 2)) return cudaErrorInvalidValue;
        if (mode == kModeHybrid) {
            p.experts = kPairExperts;
            p.release_late = 1;
        }
        err = launch_one<2, KIND>(d.units[2], row_tiles_bound(s, 2 * BM) * p.n_tiles, a, b, a, p, st);
        if (err != cudaSuccess || mode == kModePairs) return err;
        p.experts = kSingleExperts;
        p.release_late = late;
        p.overlap_prev = 1;
    }
    if (!map_b(&b, 1)) return cudaErrorInvalidValue;
    return launch_one<1, KIND>(d.units[1], row_tiles_bound(s, BM) * p.n_tiles, a, b, a, p, st);
}

// MN-major view of a row-major [rows][cols] matrix (weights: one per expert).
bool mn_map(CUtensorMap *m, const void *p, int64_t E, int64_t rows, int64_t cols, int *blocks) {
    *blocks = cols % 64 == 0;
    return *blocks ? tensor_map_weight_blocks(m, p, E, rows, cols, 2)
                   : tensor_map_weights(m, p, E, rows, cols);
}

// Tiles of a weight product's [M][N] output, and whether CTA pairs serve it.
struct WeightTiles {
    bool pair;
    int m, n;
};
WeightTiles weight_tiles(int M, int N) {
    const bool pair = pair_tiles_pay(M);
    return {pair, (M + (pair ? 2 : 1) * BM - 1) / ((pair ? 2 : 1) * BM), (N + BN - 1) / BN};
}

// dW[e] [M][N] = sum over the segment's rows of A[r]^T B[r].
cudaError_t launch_weights(const Shape &s, const DeviceInfo &d, const void *A, int M, const void *B,
                           int N, void *dW, bool overlap, Params p, cudaStream_t st) {
    CUtensorMap a, b, o;
    if (!mn_map(&a, A, 1, s.P(), M, &p.a_blocks) || !mn_map(&b, B, 1, s.P(), N, &p.b_blocks) ||
        !tensor_map_out(&o, dW, s.E, M, N))
        return cudaErrorInvalidValue;
    p.M = M;
    p.N = N;
    p.experts = kAllExperts;
    p.release_late = 0;
    p.overlap_prev = overlap;
    const WeightTiles t = weight_tiles(M, N);
    p.m_tiles = t.m;
    p.n_tiles = t.n;
    p.m_fast = p.m_tiles <= p.n_tiles;
    const int64_t tiles = (int64_t)s.E * p.m_tiles * p.n_tiles;
    if (tiles >= INT32_MAX) {
        set_error_message("weight gradient tile count exceeds 2^31");
        return cudaErrorInvalidValue;
    }
    return t.pair ? launch_one<2, DW>(d.units[2], tiles, a, b, o, p, st)
                  : launch_one<1, DW>(d.units[1], tiles, a, b, o, p, st);
}

}  // namespace
}  // namespace tc

namespace tc {
namespace {

// The current device's resident units; also checks the tensor-map encoder.
cudaError_t device_info(const DeviceInfo **out) {
    static DeviceInfo info[OncePerDevice::kDevices];
    static OncePerDevice once;
    int dev = 0;
    cudaError_t err = once([&](int device) {
        int singles = 0, pairs = 0;
        cudaError_t e;
        if ((e = prepare_all<1>(&singles)) != cudaSuccess ||
            (e = prepare_all<2>(&pairs)) != cudaSuccess ||
            (e = prepare_split<GU>()) != cudaSuccess || (e = prepare_split<DX>()) != cudaSuccess) {
            set_error_message("the gradient's matrix products do not fit on device %d", device);
            return e;
        }
        info[device].units[1] = singles;
        info[device].units[2] = pairs;
        return cudaSuccess;
    });
    if (err != cudaSuccess || (err = cudaGetDevice(&dev)) != cudaSuccess) return err;
    if (!tensor_map_encoder()) {
        set_error_message("cuTensorMapEncodeTiled is not available from the driver");
        return cudaErrorNotSupported;
    }
    *out = &info[dev];
    return cudaSuccess;
}

}  // namespace
}  // namespace tc

size_t experts_backward_tc_scratch_bytes(const Shape &s) {
    const size_t pf = (size_t)s.P() * s.f;
    return (4 * pf + 255) / 256 * 256 + 4 * pf;  // dh (fp32), dgu (bf16, 2f columns)
}

cudaError_t launch_experts_backward_tc(const Shape &s, const ExpertsBwd &x, const DevStatus &ds,
                                       cudaStream_t st) {
    using namespace tc;
    const DeviceInfo *info;
    cudaError_t err = device_info(&info);
    if (err != cudaSuccess) return err;
    const DeviceInfo &d = *info;
    const int64_t P = s.P();
    if (row_tiles_bound(s, BM) * (std::max(s.d, s.f) / (BN / 2) + 1) >= (int64_t)INT32_MAX) {
        set_error_message("experts' gradient tile count exceeds 2^31");
        return cudaErrorInvalidValue;
    }
    float *dh = static_cast<float *>(x.ws);
    void *dgu = static_cast<uint8_t *>(x.ws) + (4 * (size_t)P * s.f + 255) / 256 * 256;
    CUtensorMap tx, tdy, tdgu;
    if (!tensor_map_rows(&tx, x.x_perm, P, s.d, BM) || !tensor_map_rows(&tdy, x.dy_perm, P, s.d, BM) ||
        !tensor_map_rows(&tdgu, dgu, P, 2 * (int64_t)s.f, BM)) {
        set_error_message("cuTensorMapEncodeTiled rejected an operand (alignment or size)");
        return cudaErrorInvalidValue;
    }
    Params p = {};
    p.offsets = x.offsets;
    p.E = s.E;
    p.f = s.f;
    p.dh = dh;
    p.ds = ds;
    Params q = p;
    q.K = s.d;
    q.N = s.f;
    auto map_wd = [&](CUtensorMap *m, int rows) {
        return tensor_map_weights_k(m, x.Wd, s.E, s.f, s.d, rows); };
    auto map_gu = [&](CUtensorMap *m, int) {
        // two-atom boxes need the up half to start on a block too
        return s.f % 64 == 0 ? tensor_map_weight_blocks(m, x.Wgu, s.E, s.d, 2 * (int64_t)s.f, 2)
                             : tensor_map_weights(m, x.Wgu, s.E, s.d, 2 * (int64_t)s.f); };
    Params g = q;
    g.n_tiles = (s.f + BN / 2 - 1) / (BN / 2);
    g.out = static_cast<__nv_bfloat16 *>(dgu);
    g.b_blocks = s.f % 64 == 0;
    const int parts = split_parts(s, d, g.n_tiles, g.K, 1);
    // dWd's product reads neither dh nor dgu, dWgu's no dx: while the weights fit in
    // L2 each starts beside the product before it, where SMs are free (T = 64, d = 128,
    // f = 256, E = 8: 29 us to 19; T = 4096, k = 2, d = 2048, f = 768, E = 8: 184 to 174).
    // With more weights their writes meet the other's reads in HBM: T = 20, k = 2, d = f =
    // 4096, E = 4 222 to 241, the gpt-oss shape +2 %.
    const bool overlap = (int64_t)s.E * s.d * s.f * 6 <= (int64_t)128 << 20;
    auto weights_d = [&] {
        return launch_weights(s, d, x.h_perm, s.f, x.dy_perm, s.d, x.dWd, overlap, p, st); };
    g.release_late = overlap;
    if (parts) {
        CUtensorMap b, b2;
        if (!map_gu(&b, 1) || !map_wd(&b2, BN / 2)) return cudaErrorInvalidValue;
        err = launch_split<GU>(s, parts, tx, b, tdy, b2, g, st);
    } else {
        q.n_tiles = (s.f + BN - 1) / BN;
        err = launch_rows<DH>(
            s, d, tdy, [&](CUtensorMap *m, int ctas) { return map_wd(m, BN / ctas); }, q, st);
        if (err != cudaSuccess) return err;
        err = launch_rows<GU>(s, d, tx, map_gu, g, st);
    }
    if (err != cudaSuccess) return err;
    if (overlap && (err = weights_d()) != cudaSuccess) return err;
    q = p;
    q.K = 2 * s.f;
    q.N = s.d;
    q.n_tiles = (s.d + BN - 1) / BN;
    q.out = static_cast<__nv_bfloat16 *>(x.dx_perm);
    auto map_dx = [&](CUtensorMap *m, int ctas) {
        return tensor_map_weights_k(m, x.Wgu, s.E, s.d, 2 * (int64_t)s.f, BN / ctas); };
    q.release_late = overlap;
    if (const int parts = split_parts(s, d, q.n_tiles, q.K, 2)) {
        CUtensorMap b;
        if (!map_dx(&b, 1)) return cudaErrorInvalidValue;
        err = launch_split<DX>(s, parts, tdgu, b, tdgu, b, q, st);
    } else {
        err = launch_rows<DX>(s, d, tdgu, map_dx, q, st);
    }
    if (err != cudaSuccess) return err;
    if (!overlap && (err = weights_d()) != cudaSuccess) return err;
    return launch_weights(s, d, x.x_perm, s.d, dgu, 2 * s.f, x.dWgu, overlap, p, st);
}

cudaError_t launch_route_backward_tc(const Shape &s, const RouteProducts &r, const DevStatus &ds,
                                     cudaStream_t st) {
    using namespace tc;
    const DeviceInfo *info;
    cudaError_t err = device_info(&info);
    if (err != cudaSuccess) return err;
    Params p = {};
    p.ds = ds;
    p.experts = kAllExperts;
    CUtensorMap a, b, o;
    // RX: the tokens are one segment
    p.release_late = 1;  // RW does not read its output
    p.offsets = r.all;
    p.E = 1;
    p.K = r.K;
    p.N = s.d;
    p.n_tiles = (s.d + BN - 1) / BN;
    p.add = static_cast<const __nv_bfloat16 *>(r.dx_in);
    const bool pair = s.T > BM;
    if (!tensor_map_rows(&a, r.dl_x, s.T, r.K, BM, r.ld) || !mn_map(&b, r.W, 1, r.K, s.d, &p.b_blocks) ||
        !tensor_map_out(&o, r.dx, 1, s.T, s.d)) {
        set_error_message("cuTensorMapEncodeTiled rejected an operand (alignment or size)");
        return cudaErrorInvalidValue;
    }
    const int64_t row_tiles = (s.T + (pair ? 2 : 1) * BM - 1) / ((pair ? 2 : 1) * BM);
    if (row_tiles * p.n_tiles >= INT32_MAX) {
        set_error_message("router gradient tile count exceeds 2^31");
        return cudaErrorInvalidValue;
    }
    err = pair ? launch_one<2, RX>(info->units[2], row_tiles * p.n_tiles, a, b, o, p, st)
               : launch_one<1, RX>(info->units[1], row_tiles * p.n_tiles, a, b, o, p, st);
    if (err != cudaSuccess) return err;
    // RW: the splits of the token axis are the segments
    p.release_late = 0;
    p.overlap_prev = 1;
    p.offsets = r.splits;
    p.E = r.n_splits;
    p.M = s.d;
    p.N = r.K;
    p.part = r.part;
    const WeightTiles t = weight_tiles(p.M, p.N);
    p.m_tiles = t.m;
    p.n_tiles = t.n;
    p.m_fast = t.m <= t.n;
    if (!mn_map(&a, r.x, 1, s.T, s.d, &p.a_blocks)) return cudaErrorInvalidValue;
    p.b_blocks = 0;  // the terms' rows are wider than the columns used
    if (!tensor_map_weights(&b, r.dl_w, 1, s.T, r.K, r.ld)) return cudaErrorInvalidValue;
    const int64_t tiles = (int64_t)p.E * t.m * t.n;
    return t.pair ? launch_one<2, RW>(info->units[2], tiles, a, b, a, p, st)
                  : launch_one<1, RW>(info->units[1], tiles, a, b, a, p, st);
}

int route_backward_splits(int64_t T, int d, int cols) {
    const tc::WeightTiles t = tc::weight_tiles(d, cols);
    const int64_t units = t.pair ? device_sm_count() / 2 : device_sm_count();
    int64_t best = 1, best_cost = INT64_MAX;
    for (int64_t n = 1; n <= 32 && (n == 1 || T / n >= 128); ++n) {
        const int64_t waves = ((int64_t)t.m * t.n * n + units - 1) / units;
        const int64_t steps = ((T + n - 1) / n + tc::BK - 1) / tc::BK;
        const int64_t cost = waves * (steps + 6);  // a tile's epilogue is worth about 6 steps
        if (cost < best_cost) {
            best = n;
            best_cost = cost;
        }
    }
    return (int)best;
}

}  // namespace moe
