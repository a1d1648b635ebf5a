// route_scored.cu -- the router with scores of its own: softmax or sigmoid of
// the logits, a balance bias that acts on the choice and not on the weights,
// groups of experts, top-k, renormalised and scaled weights; and the gradient
// of those weights with respect to the logits.
//
//   s_e = exp(L_e) / sum_i exp(L_i)   or   1 / (1 + exp(-L_e))
//   q_e = s_e + b_e           the choice is made on q (without b: on L, the same order)
//   u_g = max of q in group g, or the sum of its two largest; the best Gk stay
//   w_j = c s_j / (sum of s over the chosen k, or 1)
//
// The choice is that of 64-bit values of q: fp32 values are ranked first, and a
// token whose ranking they cannot settle (two of its values closer than their
// errors, about one token in 1,000 at E = 256) is decided again in fp64.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "once.h"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr uint32_t kNaNKey = 1u;  // below every number's key; 0: no expert, or one already taken

// Order-preserving unsigned image of a value: a larger number has a larger key,
// +0.0 and -0.0 the same, a NaN the lowest.
__device__ __forceinline__ uint32_t key_of(float v) {
    if (isnan(v)) return kNaNKey;
    const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {  // (a NaN for kNaNKey)
    return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

struct SelectArgs {
    float *logits;  // [T][E]; written when nparts > 0, from the partial sums
    const float *partial;
    int nparts;
    const float *logit_bias, *bias;
    int64_t T;
    int E, k, renorm, sigmoid;
    // groups: lanes_per_group lanes share a group of `size` consecutive experts,
    // `per` consecutive ones a lane, so that ids ascend with the lane
    int G, Gk, top2, size, lanes_per_group, per;
    float scale;
    int32_t *idx;
    float *w;
    unsigned *zero_word;
};

// What the decision in fp64 works on, a warp's share: q of the candidates, then their ids.
struct Undecided {
    double *q;
    uint16_t *id;
};

__device__ __forceinline__ bool before(double a, double b) {  // by value alone; a NaN last
    if (isnan(a) || isnan(b)) return !isnan(a) && isnan(b);
    return a > b;
}

struct Softmax {
    float m;      // the largest logit
    double z;     // sum of exp(L - m)
};

__device__ __noinline__ double score64(float L, bool sigmoid, Softmax sm) {
    if (sigmoid) return 1.0 / (1.0 + exp(-(double)L));
    return sm.m == -INFINITY ? 0.0 : exp((double)L - (double)sm.m) / sm.z;
}

// The selection in fp64, for a token that fp32 left open.  floor32: no expert
// whose fp32 value is below it can be chosen; kept: the groups to choose from,
// or, if `groups` is set, those are open as well.  Returns lane j's expert.
__device__ __noinline__ int select64(const SelectArgs &a, const float *L, float m, float floor32,
                                     const float *q32, unsigned kept, bool groups, Undecided u) {
    const int lane = threadIdx.x & 31;
    Softmax sm = {m, 1.0};
    if (!a.sigmoid && m != -INFINITY) {
        double z = 0.0;
        for (int e = lane; e < a.E; e += 32) z += exp((double)L[e] - (double)m);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
        sm.z = z;
    }
    // candidates, in ascending id
    int n = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
        const int e = e0 + lane;
        bool in = e < a.E;
        if (in && !groups) in = ((kept >> (e / a.size)) & 1u) && !(q32[e] < floor32);
        const unsigned b = __ballot_sync(kAll, in);
        if (in) u.id[n + __popc(b & ((1u << lane) - 1u))] = (uint16_t)e;
        n += __popc(b);
    }
    __syncwarp();
    // one logit for all of them (a padded row's): one score
    bool same = a.sigmoid;
    const float first = L[u.id[0]];
    for (int p = lane; p < n; p += 32)
        same = same && __float_as_uint(L[u.id[p]]) == __float_as_uint(first);
    same = __all_sync(kAll, same);
    const double s0 = same ? score64(first, true, sm) : 0.0;
    for (int p = lane; p < n; p += 32) {
        const int e = u.id[p];
        const double s = same ? s0 : score64(L[e], a.sigmoid, sm);
        u.q[p] = a.bias ? s + (double)a.bias[e] : s;
    }
    __syncwarp();
    if (groups) {  // every expert is a candidate: p == e
        double score = 0.0;
        if (lane < a.G) {
            double b1 = NAN, b2 = NAN;
            for (int i = 0; i < a.size; ++i) {
                const double v = u.q[lane * a.size + i];
                if (i == 0) {
                    b1 = v;
                } else if (before(v, b1)) {
                    b2 = b1;
                    b1 = v;
                } else if (i == 1 || before(v, b2)) {
                    b2 = v;
                }
            }
            score = a.top2 && a.size > 1 ? b1 + b2 : b1;
        }
        int ahead = 0;
        for (int h = 0; h < a.G; ++h) {
            const double o = __shfl_sync(kAll, score, h);
            if (before(o, score) || (h < lane && !before(score, o))) ++ahead;
        }
        kept = __ballot_sync(kAll, lane < a.G && ahead < a.Gk);
        for (int p = lane; p < n; p += 32) {
            if (!((kept >> (u.id[p] / a.size)) & 1u)) u.id[p] = 0xFFFFu;
            else if (!a.bias) u.q[p] = (double)L[u.id[p]];
        }
        __syncwarp();
    }
    int mine = 0;
    for (int j = 0; j < a.k; ++j) {
        double v = NAN;
        int at = 0x7fffffff;
        for (int p = lane; p < n; p += 32) {
            if (u.id[p] == 0xFFFFu) continue;
            if (at == 0x7fffffff || before(u.q[p], v)) {
                v = u.q[p];
                at = p;
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            const double ov = __shfl_xor_sync(kAll, v, o);
            const int oat = __shfl_xor_sync(kAll, at, o);
            if (oat != 0x7fffffff &&
                (at == 0x7fffffff || before(ov, v) || (oat < at && !before(v, ov)))) {
                v = ov;
                at = oat;
            }
        }
        if (lane == j) mine = u.id[at];
        __syncwarp();
        if (lane == 0) u.id[at] = 0xFFFFu;
        __syncwarp();
    }
    return mine;
}

// One warp per token.  VPL: values a lane has room for (>= a.per).  EXACT: the
// ranking is that of the logits themselves (no bias, and no group sums), which
// fp32 settles; otherwise shared memory holds the fp64 decision's candidates.
template <int VPL, bool EXACT>
__global__ void __launch_bounds__(256)
select_kernel(const __grid_constant__ SelectArgs a) {
    pdl_entry();
    if (a.zero_word != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.zero_word = 0u;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5, wid = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * warps + wid;
    if (t >= a.T) return;  // warp-uniform
    const int E = a.E;
    float *L = a.logits + t * E;
    const int group = lane / a.lanes_per_group, r = lane % a.lanes_per_group;
    const int e0 = group * a.size + r * a.per;
    const int count = group < a.G ? max(0, min(a.per, a.size - r * a.per)) : 0;

    float v[VPL];
    if (a.nparts > 0) {
        const float *p = a.partial + t * E;
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] = i < count ? p[e0 + i] : 0.f;
#pragma unroll 4
        for (int z = 1; z < a.nparts; ++z) {
            p += a.T * E;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (i < count) v[i] += p[e0 + i];
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            if (i >= count) continue;
            if (a.logit_bias) v[i] += a.logit_bias[e0 + i];
            L[e0 + i] = v[i];
        }
        __syncwarp();
    } else if (VPL % 4 == 0 && a.per == VPL && (E & 3) == 0 && (a.size & 3) == 0) {
#pragma unroll
        for (int i = 0; i + 3 < VPL; i += 4) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < count) x = *reinterpret_cast<const float4 *>(L + e0 + i);
            v[i] = x.x;
            v[i + 1] = x.y;
            v[i + 2] = x.z;
            v[i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] = i < count ? L[e0 + i] : 0.f;
    }

    // softmax: the largest logit and the sum of the exponentials
    float m = -INFINITY, z = 1.f;
    if (!a.sigmoid) {
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (i < count) top = max(top, key_of(v[i]));
        top = __reduce_max_sync(kAll, top);
        if (top > kNaNKey) m = value_of(top);
        z = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (i < count) z += expf(v[i] - m);
        z = warp_sum(z);
    }
    uint32_t key[VPL];
    float *q32 = nullptr;
    Undecided und = {nullptr, nullptr};
    if constexpr (EXACT) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = i < count ? key_of(v[i]) : 0u;
    } else {
        // this warp's share of the shared memory: q in fp64, in fp32, ids
        unsigned char *mine = smem + (size_t)wid * ((14 * E + 15) & ~15);
        und.q = reinterpret_cast<double *>(mine);
        q32 = reinterpret_cast<float *>(mine + 8 * E);
        und.id = reinterpret_cast<uint16_t *>(mine + 12 * E);
        const float inv = 1.f / z;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            key[i] = 0u;
            if (i >= count) continue;
            const float s = a.sigmoid ? 1.f / (1.f + expf(-v[i]))
                                      : m == -INFINITY ? 0.f : expf(v[i] - m) * inv;
            const float q = a.bias ? s + a.bias[e0 + i] : s;
            q32[e0 + i] = q;
            key[i] = key_of(q);
        }
    }
    // How far two values of q have to be apart for fp32 to rank them.  Sigmoid:
    // expf 2 ulp, the sum and the division half a one each: 3 * 2^-23 of s <= 1.
    // Softmax: the difference L - m gives the exponential 2^-24 |L - m| of itself
    // and x e^-x < 0.4, expf 2 ulp, the sum of VPL + 5 terms in series half an ulp
    // each, the reciprocal and the product: below (VPL + 12) 2^-23 of the largest
    // score 1/z.  q itself is rounded to 2^-24 of its size.  Twice that for two
    // values, and some room.
    const float unit = a.sigmoid ? 8.f * 0x1p-23f : 2.f * (VPL + 12) * 0x1p-23f / z;
    auto open = [&](float hi, float lo) {  // also where either is a NaN or both are infinite
        return !(hi - lo > unit + 0x1p-22f * fmaxf(fabsf(hi), fabsf(lo)));
    };

    bool groups_open = false;
    unsigned kept = kAll;
    if (a.Gk < a.G) {
        uint32_t b1 = 0u, b2 = 0u;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            b2 = max(b2, min(b1, key[i]));
            b1 = max(b1, key[i]);
        }
        for (int o = 1; o < a.lanes_per_group; o <<= 1) {
            const uint32_t o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
            b2 = max(max(b2, o2), min(b1, o1));
            b1 = max(b1, o1);
        }
        uint32_t u = b1;
        if constexpr (!EXACT)
            if (a.top2 && b2 != 0u) u = key_of(value_of(b1) + value_of(b2));
        int ahead = 0;
        for (int h = 0; h < a.G; ++h) {
            const uint32_t o = __shfl_sync(kAll, u, h * a.lanes_per_group);
            if (o > u || (o == u && h < group)) ++ahead;
        }
        const bool stays = group < a.G && ahead < a.Gk;
        if constexpr (!EXACT) {
            const float lo = value_of(__reduce_min_sync(kAll, stays ? u : 0xffffffffu));
            const float hi = value_of(__reduce_max_sync(kAll, stays || group >= a.G ? 0u : u));
            // a sum has the errors of its two values and its own rounding
            groups_open = a.top2 ? !(lo - hi > 2.f * unit + 0x1p-21f * fmaxf(fabsf(lo), fabsf(hi)))
                                 : open(lo, hi);
            kept = 0u;
            for (int g = 0; g < a.G; ++g)
                if (__shfl_sync(kAll, (int)stays, g * a.lanes_per_group)) kept |= 1u << g;
        }
        if (!stays)
#pragma unroll
            for (int i = 0; i < VPL; ++i) key[i] = 0u;
        // without a bias the order inside the groups is that of the logits
        if constexpr (!EXACT)
            if (!a.bias && stays)
#pragma unroll
                for (int i = 0; i < VPL; ++i) key[i] = i < count ? key_of(v[i]) : 0u;
    }

    // k rounds: the largest key of the warp, in the lowest lane that has it, at
    // the lowest place there
    uint32_t best = 0u;
#pragma unroll
    for (int i = 0; i < VPL; ++i) best = max(best, key[i]);
    int my_e = 0;
    uint32_t my_key = 0u;
    for (int j = 0; j < a.k; ++j) {
        const uint32_t top = __reduce_max_sync(kAll, best);
        const int owner = __ffs(__ballot_sync(kAll, best == top)) - 1;
        int e = 0;
        if (lane == owner) {
            int at = VPL - 1;
#pragma unroll
            for (int i = VPL - 2; i >= 0; --i)
                if (key[i] == top) at = i;
            e = e0 + at;
            best = 0u;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                if (i == at) key[i] = 0u;
                best = max(best, key[i]);
            }
        }
        e = __shfl_sync(kAll, e, owner);
        if (lane == j) {
            my_e = e;
            my_key = top;
        }
    }
    if constexpr (!EXACT) {
        const uint32_t next = __reduce_max_sync(kAll, best);  // the best that was left
        bool undecided = groups_open;
        float last = 0.f;
        if (a.bias) {
            const float mine = value_of(my_key), above = __shfl_up_sync(kAll, mine, 1);
            last = __shfl_sync(kAll, mine, a.k - 1);
            bool o = lane > 0 && lane < a.k && open(above, mine);
            if (lane == 0 && next != 0u) o = open(last, value_of(next));
            undecided |= __any_sync(kAll, o) != 0;
        }
        if (undecided) {
            __syncwarp();
            // no candidate: those that fp32 puts below the last chosen by more than
            // the errors (a NaN there excludes none)
            const float floor32 = last - (2.f * unit + 0x1p-21f * fabsf(last));
            my_e = select64(a, L, m, floor32, q32, kept, groups_open, und);
        }
    }

    // the weights, a slot a lane
    if (a.sigmoid || a.renorm) {
        const bool slot = lane < a.k;
        const float mine = slot ? L[my_e] : 0.f;
        float s = 0.f;
        if (a.sigmoid) s = slot ? 1.f / (1.f + expf(-mine)) : 0.f;
        float sum = a.sigmoid && a.renorm ? warp_sum(s) : 1.f;
        if (a.renorm && (!a.sigmoid || sum < 0x1p-100f)) {
            // shares of exponentials, shifted by the largest chosen logit; so too
            // sigmoids that underflow together, where 1 + exp(L) is 1
            float top = slot ? mine : -INFINITY;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
            s = !slot || top == -INFINITY ? 0.f : expf(mine - top);
            sum = top == -INFINITY ? 1.f : warp_sum(s);
        }
        if (slot) {
            a.idx[t * a.k + lane] = my_e;
            a.w[t * a.k + lane] = a.scale * (s / sum);
        }
    } else if (lane < a.k) {
        a.idx[t * a.k + lane] = my_e;
        a.w[t * a.k + lane] = m == -INFINITY ? 0.f : a.scale * (expf(L[my_e] - m) / z);
    }
}

template <int VPL>
cudaError_t launch_select_v(const SelectArgs &a, bool exact, cudaStream_t st) {
    const int threads = 256, warps = threads / 32;
    const dim3 grid((unsigned)((a.T + warps - 1) / warps));
    if (exact) return launch_pdl(select_kernel<VPL, true>, grid, dim3(threads), 0, st, a);
    // the candidates' shared memory: 14 bytes an expert and warp
    const size_t smem = (size_t)warps * ((14 * (size_t)a.E + 15) & ~(size_t)15);
    if (smem > 48 * 1024) {
        static OncePerDevice once;
        const cudaError_t e = once([](int) {
            return cudaFuncSetAttribute(select_kernel<VPL, false>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        8 * 14 * 1024);
        });
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(select_kernel<VPL, false>, grid, dim3(threads), smem, st, a);
}

// ------------------------- gradient to the logits --------------------------
//   softmax, renormalised:  dl[idx_j] = w_j (d_j - S/c)
//   softmax:                dl[e]     = s_e (c g_e - S),  g_e = d_j where e = idx_j
//   sigmoid, renormalised:  dl[idx_j] = w_j (d_j - S/c) (1 - s_j)
//   sigmoid:                dl[idx_j] = w_j d_j (1 - s_j)
// with S = sum_j w_j d_j.  A warp per token: its row's chosen entries in shared
// memory, zero elsewhere, then written whole.  VEC: four columns a lane.
constexpr int kGradThreads = 256;
constexpr int kGradWarps = kGradThreads / 32;

struct GradArgs {
    const float *logits;
    const int32_t *idx;
    const float *w, *dw;
    int64_t T;
    int E, k;
    ScoreGrad f;
    float *dl;
};

// DENSE: softmax that is not renormalised; NV: its columns a lane, as float4s or floats
template <bool DENSE, bool VEC, int NV>
__global__ void __launch_bounds__(kGradThreads)
logits_grad_kernel(const GradArgs a, DevStatus ds) {
    pdl_wait();
    extern __shared__ __align__(16) float rows[];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, E = a.E;
    const int stride = (E + 3) & ~3;
    float *row = rows + wid * stride;
    for (int e = lane; e < stride; e += 32) row[e] = 0.f;
    __syncwarp();
    const int64_t t = (int64_t)blockIdx.x * kGradWarps + wid;
    if (t >= a.T) return;
    const float *L = a.logits + t * E;
    float *o = a.dl + t * E;
    int e = -1;
    float wj = 0.f, dj = 0.f;
    if (lane < a.k) {
        e = a.idx[t * a.k + lane];
        wj = a.w[t * a.k + lane];
        dj = a.dw[t * a.k + lane];
        if ((unsigned)e >= (unsigned)E) {
            raise_error(ds, kErrBadRouting);
            e = -1;
            wj = dj = 0.f;
        }
    }
    const float S = warp_sum(wj * dj);
    if constexpr (!DENSE) {
        if (e >= 0) row[e] = a.f.chosen(wj, dj, S, a.f.sigmoid ? L[e] : 0.f);
        __syncwarp();
        if constexpr (VEC) {
            for (int i = lane; i < E / 4; i += 32)
                reinterpret_cast<float4 *>(o)[i] = reinterpret_cast<const float4 *>(row)[i];
        } else {
            for (int i = lane; i < E; i += 32) o[i] = row[i];
        }
    } else {
        constexpr int W = VEC ? 4 : 1;
        if (e >= 0) row[e] = a.f.scale * dj;
        float v[NV][W];
        float m = -INFINITY, z = 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = (lane + 32 * n) * W;
            if constexpr (VEC) {
                float4 x = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                if (c < E) x = *reinterpret_cast<const float4 *>(L + c);
                v[n][0] = x.x;
                v[n][1] = x.y;
                v[n][2] = x.z;
                v[n][3] = x.w;
            } else {
                v[n][0] = c < E ? L[c] : -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < W; ++i) m = fmaxf(m, v[n][i]);
        }
#pragma unroll
        for (int q = 16; q >= 1; q >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, q));
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int i = 0; i < W; ++i) {
                v[n][i] = m == -INFINITY ? 0.f : expf(v[n][i] - m);  // all masked: no scores
                z += v[n][i];
            }
        z = warp_sum(z);
        const float inv = m == -INFINITY ? 0.f : 1.f / z;
        __syncwarp();
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = (lane + 32 * n) * W;
            if (c >= E) continue;
            if constexpr (VEC) {
                const float4 g = *reinterpret_cast<const float4 *>(row + c);
                *reinterpret_cast<float4 *>(o + c) =
                    make_float4(v[n][0] * inv * (g.x - S), v[n][1] * inv * (g.y - S),
                                v[n][2] * inv * (g.z - S), v[n][3] * inv * (g.w - S));
            } else {
                o[c] = v[n][0] * inv * (row[c] - S);
            }
        }
    }
}

template <bool DENSE, bool VEC, int NV>
cudaError_t launch_grad(const GradArgs &a, const DevStatus &ds, cudaStream_t st) {
    const dim3 grid((unsigned)((a.T + kGradWarps - 1) / kGradWarps));
    const size_t smem = sizeof(float) * kGradWarps * (size_t)((a.E + 3) & ~3);
    return launch_pdl(logits_grad_kernel<DENSE, VEC, NV>, grid, dim3(kGradThreads), smem, st, a, ds);
}

template <bool VEC>
cudaError_t launch_grad_any(const GradArgs &a, bool dense, const DevStatus &ds, cudaStream_t st) {
    if (!dense) return launch_grad<false, VEC, 1>(a, ds, st);
    const int n = (a.E + (VEC ? 127 : 31)) / (VEC ? 128 : 32);
    if (n <= 1) return launch_grad<true, VEC, 1>(a, ds, st);
    if (n <= 2) return launch_grad<true, VEC, 2>(a, ds, st);
    if (n <= 4) return launch_grad<true, VEC, 4>(a, ds, st);
    if (VEC || n <= 8) return launch_grad<true, VEC, 8>(a, ds, st);
    if constexpr (!VEC) {
        if (n <= 16) return launch_grad<true, VEC, 16>(a, ds, st);
        return launch_grad<true, VEC, 32>(a, ds, st);
    }
    return cudaErrorInvalidValue;
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

cudaError_t launch_select(const Shape &s, const Router &r, float *logits, const float *partial,
                          int nparts, const float *logit_bias, const float *bias, int32_t *idx,
                          float *w, cudaStream_t st, unsigned *zero_word) {
    SelectArgs a = {};
    a.logits = logits;
    a.partial = partial;
    a.nparts = nparts;
    a.logit_bias = logit_bias;
    a.bias = bias;
    a.T = s.T;
    a.E = s.E;
    a.k = s.k;
    a.renorm = s.renorm;
    a.sigmoid = r.sigmoid;
    a.G = r.Gk < r.G ? r.G : 1;  // all groups kept: none
    a.Gk = r.Gk < r.G ? r.Gk : 1;
    a.top2 = r.top2;
    a.size = s.E / a.G;
    a.lanes_per_group = 32;
    for (int g = 1; g < a.G; g <<= 1) a.lanes_per_group /= 2;
    a.per = (a.size + a.lanes_per_group - 1) / a.lanes_per_group;
    a.scale = r.scale;
    a.idx = idx;
    a.w = w;
    a.zero_word = zero_word;
    const bool exact = !bias && (a.Gk == a.G || !a.top2);
    cudaError_t e;
    if (a.per <= 1) e = launch_select_v<1>(a, exact, st);
    else if (a.per <= 2) e = launch_select_v<2>(a, exact, st);
    else if (a.per <= 4) e = launch_select_v<4>(a, exact, st);
    else if (a.per <= 8) e = launch_select_v<8>(a, exact, st);
    else if (a.per <= 16) e = launch_select_v<16>(a, exact, st);
    else if (a.per <= 32) e = launch_select_v<32>(a, exact, st);
    else e = launch_select_v<64>(a, exact, st);  // E > 512, a number of groups between powers of two
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_logits_grad(const Shape &s, const ScoreGrad &f, const float *logits,
                               const int32_t *idx, const float *w, const float *dw, float *dlogits,
                               const DevStatus &ds, cudaStream_t st) {
    const GradArgs a = {logits, idx, w, dw, s.T, s.E, s.k, f, dlogits};
    const cudaError_t e = (s.E & 3) == 0 ? launch_grad_any<true>(a, f.dense, ds, st)
                                         : launch_grad_any<false>(a, f.dense, ds, st);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_balance(const int32_t *counts, int64_t layers, int E, float rate, float *bias,
                           float *imbalance, cudaStream_t st) {
    const cudaError_t e = launch_pdl(balance_kernel, dim3((unsigned)layers), dim3(kBalanceThreads), 0,
                                     st, counts, E, rate, bias, imbalance);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
