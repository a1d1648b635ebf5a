// route_bwd.cu -- gradient of the router.
//
// With dw the gradient of the chosen experts' weights, S = sum_i w_i dw_i (other
// scores than moe_route's by ScoreGrad; "renormalised" below is every case in
// which only the chosen logits have a gradient):
//   renormalised weights are a softmax over the chosen logits alone, so
//     dl[idx_j] = w_j (dw_j - S), every other logit's gradient is zero;
//   plain softmax weights: dl[e] = p_e (g_e - S), g_e = dw_j where e = idx_j
//     and 0 elsewhere, p = softmax over all E logits.
//   dWr = dl^T x,   dbias = sum_t dl,   dx = dx_in + dl Wr.
//
// bf16 x: the products run on the tensor cores (gemm_bwd_tc.cu).  dl and Wr
// are fp32, so they are written as sums of bf16 terms: v = hi + mid + lo to
// 2^-25 of v.  dWr takes all three terms of dl against x, which is exact in
// bf16, each term in its own accumulator columns; dx, which is rounded to
// bf16, takes hi Whi + mid Whi + hi Wlo, within 2^-17.  A token's terms lie as
// [lo | hi | mid | hi], E8 (E rounded up to 8) columns each: the first three
// blocks are dWr's operand, the last three, against [Whi; Whi; Wlo], dx's.
// Launches: terms (with the split of Wr), dx, dWr over splits of the token
// axis, their sum.  T = 16384, d = 2048, E = 128, k = 8: 70 us, of them about 20 in
// dx's and 33 in dWr's products (bound by shared memory, see gemm_bwd_tc.cu),
// where fp32 products on the CUDA cores took 860.
// fp32 x: the same steps on the CUDA cores, bound by the multiply-adds (T = 8192,
// d = 4096, k = 8, E = 64 without renormalisation: 172 us, dx 88 and dWr 82);
// renormalised with many experts, dx is the sum of the chosen experts' rows of
// Wr (143 us; E = 128 220, with the product over all E 320).
// At most 8 experts: one pass on the CUDA cores for both types (below).  Short
// batches: all sums in one launch after the terms (small_batch).
#include "common.cuh"
#include "kernels.h"
#include "simt_gemm.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTokenBlocks = 152 * 8;
constexpr int kSplitCols = 4 * kThreads;  // elements of Wr per block
constexpr int kCopyCols = 8 * kThreads;   // elements of x per block

template <bool MAX> __device__ __forceinline__ float warp_all(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    return v;
}

struct Terms {
    __nv_bfloat16 hi, mid, lo;
};
__device__ __forceinline__ Terms split3(float v) {
    Terms t;
    t.hi = __float2bfloat16_rn(v);
    const float r = v - __bfloat162float(t.hi);
    t.mid = __float2bfloat16_rn(r);
    t.lo = __float2bfloat16_rn(r - __bfloat162float(t.mid));
    if (!isfinite(v)) t.mid = t.lo = __float2bfloat16_rn(0.f);  // hi alone is the value
    return t;
}

__device__ __forceinline__ uint32_t pack(__nv_bfloat16 a, __nv_bfloat16 b) {
    return (uint32_t)__bfloat16_as_ushort(a) | (uint32_t)__bfloat16_as_ushort(b) << 16;
}

struct TermsArgs {
    const float *logits;
    const int32_t *idx;
    const float *w, *dw;
    int64_t T;
    int E, k, renorm;
    ScoreGrad f;
    float *dl, *bias_part;  // [T][E]; [token blocks][E8]
    float *dl8;  // fp32 x only: dl in rows of E8 columns
    // fp32 x, dx from the chosen rows of Wr: their dl [T][k], and the ids with
    // -1 for one outside [0, E)
    float *dlk;
    int32_t *rows;
    // bf16 x only (dl4 != nullptr): the terms [T][4*E8], Wr [E][d] and its
    // terms [3*E8][d], and the segment boundaries of the two products
    __nv_bfloat16 *dl4, *W3;
    const float *Wr;
    int E8, d, token_blocks, n_splits, split;
    int32_t *all, *splits;
    // small batches, bf16 x: its copy in fp32, T * d elements
    const __nv_bfloat16 *x;
    float *x32;
};

// Blocks below token_blocks: a warp per token at a time, its row of dl in
// shared memory (then written whole, as floats and as terms) and the warp's
// running sum of the rows for the bias.  The blocks after: kSplitCols elements
// of Wr, or kCopyCols of x, each.
__global__ void __launch_bounds__(kThreads) terms_kernel(TermsArgs a, DevStatus ds) {
    pdl_wait();
    extern __shared__ float sh[];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, E8 = a.E8;
    if ((int)blockIdx.x >= a.token_blocks && a.x32) {
        const int64_t i = (int64_t)((int)blockIdx.x - a.token_blocks) * kCopyCols + 8 * threadIdx.x;
        if (i >= a.T * a.d) return;
        float v[8];
        unpack16(ldg16(a.x + i), v, static_cast<const __nv_bfloat16 *>(nullptr));
        *reinterpret_cast<float4 *>(a.x32 + i) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(a.x32 + i + 4) = make_float4(v[4], v[5], v[6], v[7]);
        return;
    }
    if ((int)blockIdx.x >= a.token_blocks) {
        const int64_t n = (int64_t)E8 * a.d, real = (int64_t)a.E * a.d;
        const int64_t i0 = (int64_t)((int)blockIdx.x - a.token_blocks) * kSplitCols + threadIdx.x;
#pragma unroll
        for (int j = 0; j < kSplitCols / kThreads; ++j) {
            const int64_t i = i0 + j * kThreads;
            if (i >= n) break;
            const Terms t = split3(i < real ? a.Wr[i] : 0.f);
            a.W3[i] = t.hi;
            a.W3[n + i] = t.hi;
            a.W3[2 * n + i] = t.mid;
        }
        return;
    }
    if (blockIdx.x == 0 && a.dl4) {
        for (int i = threadIdx.x; i <= a.n_splits; i += kThreads)
            a.splits[i] = (int32_t)min(a.T, (int64_t)i * a.split);
        if (threadIdx.x == 0) {
            a.all[0] = 0;
            a.all[1] = (int32_t)a.T;
        }
    }
    float *row = sh + wid * E8, *sum = sh + (kWarps + wid) * E8;
    for (int e = lane; e < E8; e += 32) row[e] = sum[e] = 0.f;
    __syncwarp();
    const int64_t step = (int64_t)a.token_blocks * kWarps;
    for (int64_t t = (int64_t)blockIdx.x * kWarps + wid; t < a.T; t += step) {
        int e = -1;
        float wj = 0.f, dj = 0.f;
        if (lane < a.k) {
            e = a.idx[t * a.k + lane];
            wj = a.w[t * a.k + lane];
            dj = a.dw[t * a.k + lane];
            if ((unsigned)e >= (unsigned)a.E) {
                raise_error(ds, kErrBadRouting);
                e = -1;
                wj = dj = 0.f;
            }
        }
        const float S = warp_all<false>(wj * dj);
        const float *L = a.logits + t * a.E;
        if (!a.renorm) {
            float m = -INFINITY;
            for (int i = lane; i < a.E; i += 32) m = fmaxf(m, L[i]);
            m = warp_all<true>(m);
            if (m == -INFINITY) m = 0.f;  // a row of -inf: scores of 0
            float z = 0.f;
            for (int i = lane; i < a.E; i += 32) {
                row[i] = expf(L[i] - m);
                z += row[i];
            }
            z = warp_all<false>(z);
            const float inv = z != 0.f ? 1.f / z : 0.f;
            for (int i = lane; i < a.E; i += 32) row[i] *= inv * (0.f - S);
            __syncwarp();
            if (e >= 0) row[e] = expf(L[e] - m) * inv * (a.f.scale * dj - S);
        } else {
            const float v = a.f.chosen(wj, dj, S, a.f.sigmoid && e >= 0 ? L[e] : 0.f);
            if (e >= 0) row[e] = v;
            if (a.dlk && lane < a.k) {
                a.dlk[t * a.k + lane] = v;
                a.rows[t * a.k + lane] = e;
            }
        }
        __syncwarp();
        // the row as floats and as terms, four columns a lane
        const bool whole = (a.E & 3) == 0;
        float *o = a.dl + t * a.E;
        for (int v = lane; v < E8 / 4; v += 32) {
            const float4 r = *reinterpret_cast<const float4 *>(row + 4 * v);
            if (whole) {
                if (4 * v < a.E) *reinterpret_cast<float4 *>(o + 4 * v) = r;
            } else {
                if (4 * v < a.E) o[4 * v] = r.x;
                if (4 * v + 1 < a.E) o[4 * v + 1] = r.y;
                if (4 * v + 2 < a.E) o[4 * v + 2] = r.z;
                if (4 * v + 3 < a.E) o[4 * v + 3] = r.w;
            }
            if (a.dl8) *reinterpret_cast<float4 *>(a.dl8 + t * E8 + 4 * v) = r;
            uint2 hi = make_uint2(0, 0), mid = hi, lo = hi;
            if (r.x != 0.f || r.y != 0.f || r.z != 0.f || r.w != 0.f) {  // mostly zeros when renormalised
                float4 *acc = reinterpret_cast<float4 *>(sum + 4 * v);
                float4 q = *acc;
                q.x += r.x;
                q.y += r.y;
                q.z += r.z;
                q.w += r.w;
                *acc = q;
                if (a.dl4) {
                    const Terms x = split3(r.x), y = split3(r.y), z = split3(r.z), w = split3(r.w);
                    hi = make_uint2(pack(x.hi, y.hi), pack(z.hi, w.hi));
                    mid = make_uint2(pack(x.mid, y.mid), pack(z.mid, w.mid));
                    lo = make_uint2(pack(x.lo, y.lo), pack(z.lo, w.lo));
                }
            }
            if (a.dl4) {
                uint2 *d4 = reinterpret_cast<uint2 *>(a.dl4 + t * 4 * E8) + v;
                d4[0] = lo;
                d4[E8 / 4] = hi;
                d4[2 * (E8 / 4)] = mid;
                d4[3 * (E8 / 4)] = hi;
            }
        }
        __syncwarp();
        if (a.renorm && e >= 0) row[e] = 0.f;  // all zero again for the next token
        __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E8; e += kThreads) {
        float s = 0.f;
        for (int i = 0; i < kWarps; ++i) s += sh[(kWarps + i) * E8 + e];
        a.bias_part[(int64_t)blockIdx.x * E8 + e] = s;
    }
}

// dWr[e][c] = the sum over splits and terms of part[s][b*stride + e][c]: SHARE
// warps take 128 elements, a range of the partial sums each.  1 or 8: 12
// partial sums (the Qwen3 router) take 5.5 us with 1 and 7.4 with 8, while one
// warp alone would wait for 114 (the Mixtral router, 5.6 us with 8) in 29 rounds.
// The blocks after those sum the bias.
template <int SHARE>
__global__ void __launch_bounds__(kThreads)
sum_kernel(const float *__restrict__ part, int splits, int terms, int stride, int E, int E8, int d,
           float *__restrict__ dWr, const float *__restrict__ bias_part, int token_blocks,
           int weight_blocks, float *__restrict__ dbias) {
    pdl_wait();
    __shared__ float4 s_part[kThreads];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    if ((int)blockIdx.x < weight_blocks) {
        const int64_t group = (int64_t)blockIdx.x * (kWarps / SHARE) + wid / SHARE;
        const int64_t i = 4 * (group * 32 + lane);
        const bool have = i < (int64_t)E * d;
        const int n = splits * terms, per = (n + SHARE - 1) / SHARE, mine = wid % SHARE;
        const int z1 = min(n, (mine + 1) * per);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (have) {
            const int64_t e = i / d, c = i % d;
            for (int z0 = mine * per; z0 < z1; z0 += 4) {  // four loads in flight
                float4 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int z = z0 + j;  // (split, term)
                    v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (z < z1)
                        v[j] = *reinterpret_cast<const float4 *>(part + ((int64_t)z * stride + e) * d + c);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc.x += v[j].x;
                    acc.y += v[j].y;
                    acc.z += v[j].z;
                    acc.w += v[j].w;
                }
            }
        }
        s_part[threadIdx.x] = acc;
        __syncthreads();
        if (mine > 0 || !have) return;
        for (int w = 1; w < SHARE; ++w) {
            const float4 v = s_part[32 * (wid + w) + lane];
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
        }
        *reinterpret_cast<float4 *>(dWr + i) = acc;
        return;
    }
    // four experts a block, all threads over the token blocks
    const int e = 4 * ((int)blockIdx.x - weight_blocks);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 5
    for (int b = threadIdx.x; b < token_blocks; b += kThreads) {
        const float4 v = *reinterpret_cast<const float4 *>(bias_part + (int64_t)b * E8 + e);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    s_part[threadIdx.x] = s;
    __syncthreads();
    if (wid >= 4 || e + wid >= E) return;
    float t = 0.f;
    for (int i = lane; i < kThreads; i += 32) t += reinterpret_cast<const float *>(s_part)[4 * i + wid];
    t = warp_all<false>(t);
    if (lane == 0) dbias[e + wid] = t;
}

// ------------------------------ few experts ---------------------------------
// E <= 8: both products in one pass over the tokens on the CUDA cores, 4 T E d
// operations beside 2 T d elements moved.  A thread owns CPT columns: their Wr
// and their running dWr, 8 experts each, stay in registers, which leaves few
// warps, so its columns of the next tokens come through a ring in shared
// memory (cp.async).  A block's tokens' rows of dl are formed by its threads, a
// token each, while the first copies are under way.  Measured against the
// tensor-core products: E = 8, T = d = 4096 without renormalisation 24.1 us to
// 34.3; twice the columns' registers at E = 16, T = 8192, d = 4096 62 us to 50.
constexpr int kFewThreads = 128;
constexpr int kFewMaxE = 8;
constexpr int kFewMaxTokens = 256;  // per block
constexpr int kFewRing = 16, kFewStep = 4;  // tokens in the ring, and of one group of copies

struct FewArgs {
    const void *x, *dx_in;
    const float *Wr, *logits;
    const int32_t *idx;
    const float *w, *dw;
    int64_t T;
    int E, E8, k, d, renorm, tokens;
    ScoreGrad f;
    float *dl, *part, *bias_part;
    void *dx;
};

template <typename TA>
__global__ void __launch_bounds__(kFewThreads, 3)
few_experts_kernel(FewArgs a, DevStatus ds) {
    pdl_wait();
    constexpr int EM = kFewMaxE, CPT = 16 / sizeof(TA);
    __shared__ __align__(16) float s_dl[kFewMaxTokens][EM];
    extern __shared__ __align__(16) unsigned char ring_raw[];
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int n = (int)min((int64_t)a.tokens, a.T - t0);
    const int E = a.E, k = a.k;
    const int c = ((int)blockIdx.y * kFewThreads + (int)threadIdx.x) * CPT;
    const TA *x = static_cast<const TA *>(a.x) + t0 * a.d + c;
    const TA *in = static_cast<const TA *>(a.dx_in);
    TA *out = static_cast<TA *>(a.dx) + t0 * a.d + c;
    if (in) in += t0 * a.d + c;
    // this thread's slots of the ring: x, then dx_in
    uint4 *ring = reinterpret_cast<uint4 *>(ring_raw) + threadIdx.x;
    uint4 *ring_in = ring + kFewRing * kFewThreads;
    auto fetch = [&](int i0) {  // tokens i0 .. i0 + kFewStep - 1, one group of copies
#pragma unroll
        for (int u = 0; u < kFewStep; ++u)
            if (i0 + u < n && c < a.d) {
                const int slot = (i0 + u) % kFewRing * kFewThreads;
                tc::cp_async16(tc::smem_u32(ring + slot), x + (int64_t)(i0 + u) * a.d);
                if (in) tc::cp_async16(tc::smem_u32(ring_in + slot), in + (int64_t)(i0 + u) * a.d);
            }
        tc::cp_async_commit();
    };
#pragma unroll
    for (int g = 0; g < kFewRing / kFewStep - 1; ++g) fetch(g * kFewStep);
    for (int i = threadIdx.x; i < n; i += kFewThreads) {  // token t0 + i's row of dl
        const int64_t t = t0 + i;
        float S = 0.f;
        for (int j = 0; j < k; ++j) {
            const bool ok = (unsigned)a.idx[t * k + j] < (unsigned)E;
            if (!ok) raise_error(ds, kErrBadRouting);
            S += ok ? a.w[t * k + j] * a.dw[t * k + j] : 0.f;
        }
        float m = -INFINITY, z = 0.f, p[EM];
        if (!a.renorm) {
#pragma unroll
            for (int e = 0; e < EM; ++e) {
                p[e] = e < E ? a.logits[t * E + e] : -INFINITY;
                m = fmaxf(m, p[e]);
            }
            if (m == -INFINITY) m = 0.f;  // a row of -inf: scores of 0
#pragma unroll
            for (int e = 0; e < EM; ++e) {
                p[e] = e < E ? expf(p[e] - m) : 0.f;
                z += p[e];
            }
        }
        const float inv = z != 0.f ? 1.f / z : 0.f;
#pragma unroll
        for (int e = 0; e < EM; ++e) s_dl[i][e] = a.renorm ? 0.f : p[e] * inv * (0.f - S);
        for (int j = 0; j < k; ++j) {
            const int e = a.idx[t * k + j];
            if ((unsigned)e >= (unsigned)E) continue;
            const float d = a.dw[t * k + j];
            s_dl[i][e] = a.renorm ? a.f.chosen(a.w[t * k + j], d, S,
                                               a.f.sigmoid ? a.logits[t * E + e] : 0.f)
                                  : expf(a.logits[t * E + e] - m) * inv * (a.f.scale * d - S);
        }
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    if (blockIdx.y == 0) {
        for (int i = threadIdx.x; i < n * E; i += kFewThreads)
            a.dl[t0 * E + i] = s_dl[i / E][i % E];
        for (int e = wid; e < a.E8; e += kFewThreads / 32) {
            float s = 0.f;
            if (e < E)
                for (int i = lane; i < n; i += 32) s += s_dl[i][e];
            s = warp_all<false>(s);
            if (lane == 0) a.bias_part[(int64_t)blockIdx.x * a.E8 + e] = s;
        }
    }
    if (c >= a.d) return;
    constexpr int H = CPT / 2;  // pairs of columns
    float2 W[EM][H], acc[EM][H];
#pragma unroll
    for (int e = 0; e < EM; ++e)
#pragma unroll
        for (int i = 0; i < H; ++i) {
            W[e][i] = e < E ? __ldg(reinterpret_cast<const float2 *>(a.Wr + (int64_t)e * a.d + c) + i)
                            : make_float2(0.f, 0.f);
            acc[e][i] = make_float2(0.f, 0.f);
        }
    for (int i0 = 0; i0 < n; i0 += kFewStep) {
        fetch(i0 + kFewRing - kFewStep);
        tc::cp_async_wait_group<kFewRing / kFewStep - 1>();  // this step's copies have landed
#pragma unroll
        for (int u = 0; u < kFewStep; ++u) {
            if (i0 + u >= n) continue;
            const int slot = (i0 + u) % kFewRing * kFewThreads;
            float xv[CPT], sum[CPT];
            float2 dx2[H];
            unpack16(ring[slot], xv, static_cast<const TA *>(nullptr));
#pragma unroll
            for (int i = 0; i < H; ++i) dx2[i] = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < EM; ++e) {
                const float g = s_dl[i0 + u][e];
                const float2 gg = make_float2(g, g);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    dx2[i] = fma2(gg, W[e][i], dx2[i]);
                    acc[e][i] = fma2(gg, make_float2(xv[2 * i], xv[2 * i + 1]), acc[e][i]);
                }
            }
#pragma unroll
            for (int i = 0; i < H; ++i) {
                sum[2 * i] = dx2[i].x;
                sum[2 * i + 1] = dx2[i].y;
            }
            if (in) {
                float o[CPT];
                unpack16(ring_in[slot], o, static_cast<const TA *>(nullptr));
#pragma unroll
                for (int i = 0; i < CPT; ++i) sum[i] += o[i];
            }
            stg16(out + (int64_t)(i0 + u) * a.d, pack16(sum, static_cast<const TA *>(nullptr)));
        }
    }
#pragma unroll
    for (int e = 0; e < EM; ++e)
        if (e < E) {
            float *q = a.part + ((int64_t)blockIdx.x * E + e) * a.d + c;
#pragma unroll
            for (int i = 0; i < CPT; i += 4)
                *reinterpret_cast<float4 *>(q + i) =
                    make_float4(acc[e][i / 2].x, acc[e][i / 2].y, acc[e][i / 2 + 1].x, acc[e][i / 2 + 1].y);
        }
}

// ------------------------- fp32 x, on the CUDA cores ------------------------
// Tiles of the two products over dl8, the rows of dl padded to E8 columns.
// out[e][n] = the sum over the K tokens from dl8 and x on: experts e0 .., columns n0 ..
template <typename Tl>
__device__ __forceinline__ void dwr_block(float *smem, const float *dl8, const float *x, int K, int E,
                                          int E8, int d, float *out, int e0, int n0) {
    float acc[Tl::TM][Tl::TN];
    Tl::zero(acc);
    Tl::template product<false, false>(
        smem, K,
        [=](int m, int k) { return e0 + m < E8 ? dl8 + (int64_t)k * E8 + e0 + m : nullptr; },
        [=](int k, int n) { return n0 + n < d ? x + (int64_t)k * d + n0 + n : nullptr; }, acc);
    Tl::each_run(acc, [&](int m, int c, const float *v) {
        if (e0 + m < E && n0 + c < d) Tl::store(out + (int64_t)(e0 + m) * d + n0 + c, v);
    });
}

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v) {
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(pack(__float2bfloat16_rn(v.x), __float2bfloat16_rn(v.y)),
                   pack(__float2bfloat16_rn(v.z), __float2bfloat16_rn(v.w)));
}

// dx of tokens t0 .., columns n0 ..
template <typename Tl, typename TA>
__device__ __forceinline__ void dx_block(float *smem, const float *dl8, const float *Wr,
                                         const TA *dx_in, int64_t T, int E, int E8, int d, TA *dx,
                                         int64_t t0, int n0) {
    float acc[Tl::TM][Tl::TN];
    Tl::zero(acc);
    Tl::template product<true, false>(
        smem, E8, [=](int m, int k) { return t0 + m < T ? dl8 + (t0 + m) * E8 + k : nullptr; },
        [=](int k, int n) { return k < E && n0 + n < d ? Wr + (int64_t)k * d + n0 + n : nullptr; }, acc);
    Tl::each_run(acc, [&](int m, int c, const float *v) {
        const int64_t t = t0 + m;
        const int n = n0 + c;
        if (t >= T || n >= d) return;
        float4 o = make_float4(v[0], v[1], v[2], v[3]);
        if (dx_in) {
            const float4 in = load4(dx_in + t * d + n);
            o = make_float4(o.x + in.x, o.y + in.y, o.z + in.z, o.w + in.w);
        }
        store4(dx + t * d + n, o);
    });
}

// part[split][e][c]: the sum over the tokens of one split.  beside_dx: started
// once route_dx_kernel's blocks run, whose output it does not read; it waits for that
// launch at its end, so that the next one follows both.
template <typename Tl>
__global__ void __launch_bounds__(Tl::THREADS)
dwr_kernel(const float *__restrict__ dl8, const float *__restrict__ x, int64_t T, int E, int E8,
           int d, int tokens, int beside_dx, float *__restrict__ part) {
    if (!beside_dx) pdl_wait();
    extern __shared__ __align__(16) float smem[];
    const int64_t t0 = (int64_t)blockIdx.z * tokens;
    dwr_block<Tl>(smem, dl8 + t0 * E8, x + t0 * d, (int)min((int64_t)tokens, T - t0), E, E8, d,
                  part + (int64_t)blockIdx.z * E * d, blockIdx.y * Tl::BM, blockIdx.x * Tl::BN);
    if (beside_dx) pdl_wait();
}

template <typename Tl>
__global__ void __launch_bounds__(Tl::THREADS, Tl::MIN_BLOCKS)
route_dx_kernel(const float *__restrict__ dl8, const float *__restrict__ Wr, const float *dx_in,
                int64_t T, int E, int E8, int d, float *dx) {
    pdl_wait();
    pdl_release();
    extern __shared__ __align__(16) float smem[];
    dx_block<Tl>(smem, dl8, Wr, dx_in, T, E, E8, d, dx, (int64_t)blockIdx.x * Tl::BM, blockIdx.y * Tl::BN);
}

// Small batches of both types: all three sums in one launch, dWr over all
// tokens in one go.
using SmallTile = simt::Tile<32, 64, 4, 4>;
struct SmallArgs {
    const float *dl8, *x, *Wr, *bias_part;
    const void *dx_in;
    int64_t T;
    int E, E8, d, token_blocks, dx_blocks, dwr_blocks;
    void *dx;
    float *dWr, *dbias;
};
template <typename TA>
__global__ void __launch_bounds__(SmallTile::THREADS) small_products_kernel(SmallArgs a) {
    pdl_wait();
    using Tl = SmallTile;
    extern __shared__ __align__(16) float smem[];
    const int nt = (a.d + Tl::BN - 1) / Tl::BN;
    int b = blockIdx.x;
    if (b < a.dx_blocks) {
        dx_block<Tl>(smem, a.dl8, a.Wr, static_cast<const TA *>(a.dx_in), a.T, a.E, a.E8, a.d,
                     static_cast<TA *>(a.dx), (int64_t)(b / nt) * Tl::BM, b % nt * Tl::BN);
        return;
    }
    b -= a.dx_blocks;
    if (b < a.dwr_blocks) {
        dwr_block<Tl>(smem, a.dl8, a.x, (int)a.T, a.E, a.E8, a.d, a.dWr, b / nt * Tl::BM, b % nt * Tl::BN);
        return;
    }
    const int e = (b - a.dwr_blocks) * Tl::THREADS + threadIdx.x;
    if (e >= a.E) return;
    float s = 0.f;
#pragma unroll 8
    for (int i = 0; i < a.token_blocks; ++i) s += a.bias_part[(int64_t)i * a.E8 + e];
    a.dbias[e] = s;
}

// ------------------------------- host side ---------------------------------
// fp32 x, renormalised: dx takes k rows of Wr a token instead of all E where
// that is the lesser (T = 8192, d = 4096, whole gradient, product over all E
// against gathered: k = 8, E = 64 172 us to 143, E = 48 157 to 143, E = 32 108 to 115;
// k = 4, E = 24 104 to 99, E = 16 73 to 77).
bool gathers_rows(const Shape &s) { return !s.bf16 && s.renorm && s.E >= 5 * s.k; }

// Short batches: two launches, terms and small_products_kernel, instead of four, on
// the CUDA cores for both types (bf16, us: T = 16, d = 7168, E = 26 15.5 to 5.8; T = 1,
// d = 7168, E = 256 28 to 14; T = 256, d = 4096, E = 128 24 to 21.5, but T = 512, d = 1024,
// E = 64 17.7 to 20.6, where one block adds over all tokens; fp32, four launches on the
// CUDA cores: T = 64, d = 2048, E = 128 11.3 to 9.1, T = 256, d = 4096, E = 32 11.1 to 12.3).
bool small_batch(const Shape &s) {
    return s.E > kFewMaxE && s.T <= (s.bf16 ? 256 : 128) && s.T * s.E * s.d <= (int64_t)1 << 27;
}

// dx's tiles: tokens x columns (T = 8192, d = 4096, E = 64: large 88 us, small 107;
// T = 512, d = 1024: 6.8 and 4.7, too few blocks).
using DxLarge = simt::Tile<64, 128, 8, 8>;
using DxSmall = simt::Tile<64, 64, 4, 4>;
template <typename Tl> int64_t dx_tiles(const Shape &s) {
    return (s.T + Tl::BM - 1) / Tl::BM * ((s.d + Tl::BN - 1) / Tl::BN);
}

// dWr's tiles: experts x columns, by the experts there are (T = 8192, d = 4096:
// E = 16 35 us, 32 53, 64 82, 128 157; tiles of 64 experts take 82 at any E <= 64).
using Dwr16 = simt::Tile<16, 256, 4, 4>;
using Dwr32 = simt::Tile<32, 128, 8, 4>;
using Dwr64 = simt::Tile<64, 128, 8, 4>;
enum DwrTile { kDwr16, kDwr32, kDwr64 };
DwrTile dwr_tile(const Shape &s) { return s.E <= 16 ? kDwr16 : s.E <= 32 ? kDwr32 : kDwr64; }
// Splits of the token axis that fill the SMs' slots for blocks: one block more
// than the slots costs a second round (T = 8192, d = 4096, E = 64 in 64 x 64 tiles:
// 7 splits, 448 blocks, 106 us; 5 splits, three blocks on some SMs and two on the
// others, 149).  With more tiles than slots, the number whose rounds are fullest.
template <typename Tl> int64_t dwr_splits(const Shape &s) {
    const int64_t slots = 152 * (227 * 1024 / (Tl::SMEM_BYTES + 1024));
    const int64_t t = (int64_t)((s.E + Tl::BM - 1) / Tl::BM) * ((s.d + Tl::BN - 1) / Tl::BN);
    int64_t best = slots / t < 1 ? 1 : slots / t;
    const int64_t least = best;
    for (int64_t n = least + 1; n <= least + 4; ++n)  // 5 % for the larger sum of parts
        if ((t * n + slots - 1) / slots * best * 105 < (t * best + slots - 1) / slots * n * 100)
            best = n;
    return best;
}

struct Plan {
    bool few;    // few_experts_kernel
    bool small;  // small_products_kernel
    int few_cols;  // columns of one of its blocks
    int E8, terms, token_blocks;
    int splits, tokens;  // splits of the token axis in dWr's sum, tokens each
    size_t dl, x32, dlk, rows, W3, all, split_at, bias, part, total;  // workspace offsets
};

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

Plan plan(const Shape &s) {
    Plan p;
    p.E8 = (s.E + 7) / 8 * 8;
    p.few = s.E <= kFewMaxE;
    p.few_cols = kFewThreads * (s.bf16 ? 8 : 4);
    p.small = small_batch(s);
    const bool tensor = s.bf16 && !p.few && !p.small, cores = !s.bf16 && !p.few && !p.small;
    p.terms = tensor ? 3 : 1;
    const int64_t blocks = (s.T + kWarps - 1) / kWarps;
    p.token_blocks = (int)(blocks < kMaxTokenBlocks ? blocks : kMaxTokenBlocks);
    int64_t want;
    if (p.few) {  // one wave: three blocks an SM
        const int64_t cols = (s.d + p.few_cols - 1) / p.few_cols, least = (s.T + kFewMaxTokens - 1) / kFewMaxTokens;
        want = 3 * 152 / cols;
        const int64_t most = (s.T + 7) / 8;
        want = want < 1 ? 1 : want > most ? most : want;
        want = want < least ? least : want;
    } else if (p.small) {
        want = 1;
    } else if (s.bf16) {
        want = route_backward_splits(s.T, s.d, 3 * p.E8);
    } else {
        const DwrTile tile = dwr_tile(s);
        want = tile == kDwr64 ? dwr_splits<Dwr64>(s)
               : tile == kDwr32 ? dwr_splits<Dwr32>(s)
                                : dwr_splits<Dwr16>(s);
        const int64_t most = (s.T + 63) / 64;
        want = want < 1 ? 1 : want > most ? most : want;
    }
    p.tokens = (int)((s.T + want - 1) / want);
    if (tensor) p.tokens = (p.tokens + 63) / 64 * 64;  // whole K steps but for the last split's
    p.splits = (int)((s.T + p.tokens - 1) / p.tokens);
    if (p.few) p.token_blocks = p.splits;
    size_t o = 0;
    p.dl = o;  // four terms of 2 bytes, or padded rows
    if (!p.few) o = up256(o + (tensor ? 8 : 4) * (size_t)s.T * p.E8);
    p.x32 = o;
    if (p.small && s.bf16) o = up256(o + 4 * (size_t)s.T * s.d);
    p.dlk = o;
    if (cores && gathers_rows(s)) o = up256(o + 4 * (size_t)s.P());
    p.rows = o;
    if (cores && gathers_rows(s)) o = up256(o + 4 * (size_t)s.P());
    p.W3 = o;
    if (tensor) o = up256(o + 2 * (size_t)3 * p.E8 * s.d);
    p.all = o;
    o = up256(o + 2 * sizeof(int32_t));
    p.split_at = o;
    o = up256(o + sizeof(int32_t) * ((size_t)p.splits + 1));
    p.bias = o;
    o = up256(o + sizeof(float) * (size_t)p.token_blocks * p.E8);
    p.part = o;
    if (!p.small)
        o = up256(o + sizeof(float) * (size_t)p.splits * p.terms * (p.terms > 1 ? p.E8 : s.E) * s.d);
    p.total = o;
    return p;
}

cudaError_t launch_few(const Shape &s, const RouteBwd &a, const Plan &p, float *part,
                       float *bias_part, const DevStatus &ds, cudaStream_t st) {
    FewArgs f = {a.x,  a.dx_in,       a.Wr,       a.logits, a.idx, a.w,       a.dw,
                 s.T,  s.E,           p.E8,       s.k,      s.d,   s.renorm ? 1 : 0,
                 p.tokens, a.f, a.dlogits, part, bias_part, a.dx};
    const dim3 grid(p.splits, (s.d + p.few_cols - 1) / p.few_cols), block(kFewThreads);
    const size_t ring = (size_t)kFewRing * kFewThreads * 16 * (a.dx_in ? 2 : 1);
    cudaError_t err = s.bf16 ? simt::opt_in<few_experts_kernel<__nv_bfloat16>>(64 * 1024)
                             : simt::opt_in<few_experts_kernel<float>>(64 * 1024);
    if (err != cudaSuccess) return err;
    return s.bf16 ? launch_pdl(few_experts_kernel<__nv_bfloat16>, grid, block, ring, st, f, ds)
                  : launch_pdl(few_experts_kernel<float>, grid, block, ring, st, f, ds);
}

template <typename Tl>
cudaError_t launch_dx(const Shape &s, const RouteBwd &a, const Plan &p, const float *dl8, cudaStream_t st) {
    cudaError_t err = simt::opt_in<route_dx_kernel<Tl>>(Tl::SMEM_BYTES);
    if (err != cudaSuccess) return err;
    launch_pdl(route_dx_kernel<Tl>,
               dim3((unsigned)((s.T + Tl::BM - 1) / Tl::BM), (s.d + Tl::BN - 1) / Tl::BN),
               dim3(Tl::THREADS), Tl::SMEM_BYTES, st, dl8, a.Wr,
               static_cast<const float *>(a.dx_in), s.T, s.E, p.E8, s.d, static_cast<float *>(a.dx));
    return cudaGetLastError();
}

template <typename Tl>
cudaError_t launch_dwr(const Shape &s, const RouteBwd &a, const Plan &p, const float *dl8, float *part,
                       cudaStream_t st) {
    cudaError_t err = simt::opt_in<dwr_kernel<Tl>>(Tl::SMEM_BYTES);
    if (err != cudaSuccess) return err;
    launch_pdl(dwr_kernel<Tl>, dim3((s.d + Tl::BN - 1) / Tl::BN, (s.E + Tl::BM - 1) / Tl::BM, p.splits),
               dim3(Tl::THREADS), Tl::SMEM_BYTES, st, dl8,
               static_cast<const float *>(a.x), s.T, s.E, p.E8, s.d, p.tokens, gathers_rows(s) ? 0 : 1,
               part);
    return cudaGetLastError();
}

cudaError_t launch_products(const Shape &s, const RouteBwd &a, const Plan &p, float *part,
                            float *bias_part, const DevStatus &ds, cudaStream_t st) {
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    TermsArgs t = {};
    t.logits = a.logits;
    t.idx = a.idx;
    t.w = a.w;
    t.dw = a.dw;
    t.T = s.T;
    t.E = s.E;
    t.k = s.k;
    t.renorm = s.renorm ? 1 : 0;
    t.f = a.f;
    t.dl = a.dlogits;
    t.bias_part = bias_part;
    t.E8 = p.E8;
    t.d = s.d;
    t.token_blocks = p.token_blocks;
    t.n_splits = p.splits;
    t.split = p.tokens;
    if (p.small) {
        t.dl8 = reinterpret_cast<float *>(ws + p.dl);
        if (s.bf16) {
            t.x = static_cast<const __nv_bfloat16 *>(a.x);
            t.x32 = reinterpret_cast<float *>(ws + p.x32);
        }
    } else if (s.bf16) {
        t.dl4 = reinterpret_cast<__nv_bfloat16 *>(ws + p.dl);
        t.W3 = reinterpret_cast<__nv_bfloat16 *>(ws + p.W3);
        t.Wr = a.Wr;
        t.all = reinterpret_cast<int32_t *>(ws + p.all);
        t.splits = reinterpret_cast<int32_t *>(ws + p.split_at);
    } else {
        t.dl8 = reinterpret_cast<float *>(ws + p.dl);
        if (gathers_rows(s)) {
            t.dlk = reinterpret_cast<float *>(ws + p.dlk);
            t.rows = reinterpret_cast<int32_t *>(ws + p.rows);
        }
    }
    const int more_blocks = !s.bf16  ? 0
                            : p.small ? (int)((s.T * s.d + kCopyCols - 1) / kCopyCols)
                                      : (int)(((int64_t)p.E8 * s.d + kSplitCols - 1) / kSplitCols);
    const size_t sh = sizeof(float) * 2 * kWarps * (size_t)p.E8;  // at most 64 KB
    cudaError_t err;
    if (sh > 48 * 1024 && (err = simt::opt_in<terms_kernel>(64 * 1024)) != cudaSuccess) return err;
    launch_pdl(terms_kernel, dim3(p.token_blocks + more_blocks), dim3(kThreads), sh, st, t, ds);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
    if (p.small) {
        using Tl = SmallTile;
        const int nt = (s.d + Tl::BN - 1) / Tl::BN;
        SmallArgs q = {t.dl8, s.bf16 ? t.x32 : static_cast<const float *>(a.x), a.Wr, bias_part, a.dx_in,
                       s.T, s.E, p.E8, s.d, p.token_blocks, (int)((s.T + Tl::BM - 1) / Tl::BM) * nt,
                       (s.E + Tl::BM - 1) / Tl::BM * nt, a.dx, a.dWr, a.dbias};
        const int bias_blocks = a.dbias ? (s.E + Tl::THREADS - 1) / Tl::THREADS : 0;
        const dim3 grid(q.dx_blocks + q.dwr_blocks + bias_blocks);
        static_assert(Tl::SMEM_BYTES <= 48 * 1024, "no opt-in");
        launch_pdl(s.bf16 ? small_products_kernel<__nv_bfloat16> : small_products_kernel<float>, grid,
                   dim3(Tl::THREADS), Tl::SMEM_BYTES, st, q);
        return cudaGetLastError();
    }
    if (s.bf16) {
        RouteProducts r;
        r.x = a.x;
        r.dl_w = t.dl4;
        r.dl_x = t.dl4 + p.E8;
        r.W = t.W3;
        r.dx_in = a.dx_in;
        r.K = 3 * p.E8;
        r.n_splits = p.splits;
        r.ld = 4 * (int64_t)p.E8;
        r.all = t.all;
        r.splits = t.splits;
        r.dx = a.dx;
        r.part = part;
        if ((err = launch_route_backward_tc(s, r, ds, st)) != cudaSuccess) return err;
    } else {
        if (gathers_rows(s)) {
            if ((err = launch_gather_sum_f32(s, a.Wr, t.rows, t.dlk, static_cast<const float *>(a.dx_in),
                                             static_cast<float *>(a.dx), st)) != cudaSuccess)
                return err;
        } else {
            err = dx_tiles<DxLarge>(s) >= 152 ? launch_dx<DxLarge>(s, a, p, t.dl8, st)
                                              : launch_dx<DxSmall>(s, a, p, t.dl8, st);
            if (err != cudaSuccess) return err;
        }
        const DwrTile tile = dwr_tile(s);
        err = tile == kDwr64 ? launch_dwr<Dwr64>(s, a, p, t.dl8, part, st)
              : tile == kDwr32 ? launch_dwr<Dwr32>(s, a, p, t.dl8, part, st)
                               : launch_dwr<Dwr16>(s, a, p, t.dl8, part, st);
        if (err != cudaSuccess) return err;
    }
    return cudaGetLastError();
}

}  // namespace

size_t route_backward_scratch_bytes(const Shape &s) { return plan(s).total; }

cudaError_t launch_route_backward(const Shape &s, const RouteBwd &a, const DevStatus &ds,
                                  cudaStream_t st) {
    const Plan p = plan(s);
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    float *part = reinterpret_cast<float *>(ws + p.part);
    float *bias_part = reinterpret_cast<float *>(ws + p.bias);
    cudaError_t err = p.few ? launch_few(s, a, p, part, bias_part, ds, st)
                            : launch_products(s, a, p, part, bias_part, ds, st);
    if (err != cudaSuccess || p.small) return err;
    const int share = p.splits * p.terms > 32 ? kWarps : 1;
    const int columns = 32 * kWarps / share;  // float4 columns of a block
    const int weight_blocks = (int)(((int64_t)s.E * s.d / 4 + columns - 1) / columns);
    auto sum = share == 1 ? sum_kernel<1> : sum_kernel<kWarps>;
    launch_pdl(sum, dim3(weight_blocks + (a.dbias ? (s.E + 3) / 4 : 0)), dim3(kThreads), 0, st,
               (const float *)part, p.splits, p.terms, p.terms > 1 ? p.E8 : s.E, s.E, p.E8, s.d, a.dWr,
               (const float *)bias_part, p.token_blocks, weight_blocks, a.dbias);
    return cudaGetLastError();
}

}  // namespace moe
