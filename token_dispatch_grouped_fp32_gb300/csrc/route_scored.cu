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

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "once.h"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
// The warp's largest number; NaN where no lane has one.
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
// 2^x and 1/x to 2 ulp and 1 ulp.
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

struct SelectArgs {
    float *logits;  // [T][E]; written when nparts > 0, from the partial sums
    const float *partial;
    int nparts;
    const float *logit_bias, *bias;
    int64_t T;
    int E, k, renorm, sigmoid;
    // groups: 1 << shift lanes share a group of `size` consecutive experts, `per`
    // consecutive ones a lane, so that ids ascend with the lane
    int G, Gk, top2, size, shift, per;
    float scale;
    int half;  // half the power of two that holds k slots
    int32_t *idx;
    float *w;
    unsigned *zero_word;
};

// Sum and largest over the slots (lanes below 2 * half), in all lanes.
__device__ __forceinline__ float slots_sum(float v, int half) {
    for (int o = half; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return __shfl_sync(kAll, v, 0);
}
__device__ __forceinline__ float slots_max(float v, int half) {
    for (int o = half; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return __shfl_sync(kAll, v, 0);
}

// A candidate, or a slot of the selection.
struct __align__(8) Ranked {
    float q;
    int id;
};
constexpr Ranked kNobody = {NAN, 0};

// A warp's shared memory: candidates and slots, and for the tokens that they do
// not settle the row of q, with a list of experts and their 64-bit values.
struct Scratch {
    Ranked *few, *slot;   // [32] each
    long long *key;       // [E]
    float *row;           // [E]
    uint16_t *id;         // [E]
};
__host__ __device__ inline int scratch_bytes(int E) { return 512 + ((14 * E + 15) & ~15); }
__device__ __forceinline__ Scratch scratch_of(unsigned char *smem, int wid, int E) {
    unsigned char *p = smem + (size_t)wid * scratch_bytes(E);
    return {reinterpret_cast<Ranked *>(p), reinterpret_cast<Ranked *>(p + 256),
            reinterpret_cast<long long *>(p + 512), reinterpret_cast<float *>(p + 512 + 8 * E),
            reinterpret_cast<uint16_t *>(p + 512 + 12 * E)};
}

// Order-preserving whole-number image of a 64-bit value (compared without the
// slow fp64 pipe): -0.0 and 0.0 alike, a NaN below every number.
constexpr long long kNaNKey = -0x7fffffffffffffffll;
__device__ __forceinline__ long long key_of(double v) {
    if (isnan(v)) return kNaNKey;
    const long long b = __double_as_longlong(v + 0.0);
    return b >= 0 ? b : (long long)(0x8000000000000000ull - (unsigned long long)b);
}
__device__ __forceinline__ double value_of(long long key) {
    if (key == kNaNKey) return NAN;
    return __longlong_as_double(
        key >= 0 ? key : (long long)(0x8000000000000000ull - (unsigned long long)key));
}

// sum of exp(L - m) over a row
__device__ __noinline__ double softmax_sum64(const float *L, int E, float m) {
    double z = 0.0;
    for (int e = threadIdx.x & 31; e < E; e += 32) z += exp((double)L[e] - (double)m);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
    return z;
}
// q of one expert in fp64 (a lane's own); on_logits: the logit itself
__device__ __noinline__ double value64(const SelectArgs &a, const float *L, int e, bool on_logits,
                                       float m, double z) {
    const double x = (double)L[e];
    double s = x;
    if (!on_logits)
        s = a.sigmoid ? 1.0 / (1.0 + exp(-x)) : m == -INFINITY ? 0.0 : exp(x - (double)m) / z;
    return a.bias ? s + (double)a.bias[e] : s;
}

// The 64-bit values of the n experts in u.id, to u.key.  One logit for all of them
// (a padded row's): one score.
__device__ __noinline__ void values64(const SelectArgs &a, const float *L, float m, bool on_logits,
                                      int n, const Scratch &u) {
    const int lane = threadIdx.x & 31;
    const double z = a.sigmoid || on_logits || m == -INFINITY ? 1.0 : softmax_sum64(L, a.E, m);
    const float first = L[u.id[0]];
    bool same = true;
    for (int p = lane; p < n; p += 32)
        same = same && __float_as_uint(L[u.id[p]]) == __float_as_uint(first);
    same = __all_sync(kAll, same);
    double s0 = 0.0;
    if (same) {
        const double x = (double)first;
        s0 = on_logits ? x
             : a.sigmoid ? 1.0 / (1.0 + exp(-x))
             : m == -INFINITY ? 0.0 : exp(x - (double)m) / z;
    }
    for (int p = lane; p < n; p += 32) {
        const int e = u.id[p];
        u.key[p] = key_of(!same ? value64(a, L, e, on_logits, m, z)
                          : a.bias ? s0 + (double)a.bias[e] : s0);
    }
    __syncwarp();
}

// The experts for which in(e) holds, in ascending order, to u.id.
template <typename F> __device__ __forceinline__ int list_experts(int E, const Scratch &u, F in) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const bool is = in(e0 + lane);
        const unsigned b = __ballot_sync(kAll, is);
        if (is) u.id[n + __popc(b & ((1u << lane) - 1u))] = (uint16_t)(e0 + lane);
        n += __popc(b);
    }
    __syncwarp();
    return n;
}

// Which groups stay, decided in fp64 where fp32 left it open: `sure` do, and of the
// groups in `near` the best `need`.  Masks: bit g << shift.  u.row: every
// q; floor32 (a group's lanes): only its values from there up can be of its score.
__device__ __noinline__ unsigned groups64(const SelectArgs &a, const float *L, float m,
                                          bool on_logits, unsigned sure, unsigned near, int need,
                                          float floor32, const Scratch &u) {
    const int lane = threadIdx.x & 31, shift = a.shift;
    const int n = list_experts(a.E, u, [&](int e) {
        const int g = min(e, a.E - 1) / a.size;
        const float f = __shfl_sync(kAll, floor32, g << shift);
        return e < a.E && ((near >> (g << shift)) & 1u) && !(u.row[e] < f);
    });
    values64(a, L, m, on_logits, n, u);
    // lane g << shift: its group's score
    const int mine = lane >> shift;
    const bool is = ((near >> lane) & 1u) != 0;
    long long key = kNaNKey;
    if (is) {
        int have = 0;
        long long b1 = kNaNKey, b2 = kNaNKey;
        for (int p = 0; p < n; ++p) {
            if (u.id[p] / a.size != mine) continue;
            const long long v = u.key[p];
            ++have;
            if (v > b1) {
                b2 = b1;
                b1 = v;
            } else if (v > b2) {
                b2 = v;
            }
        }
        key = a.top2 && a.size > 1 ? key_of(value_of(b1) + value_of(b2)) : b1;
    }
    int ahead = 0;
    for (int h = 0; h < a.G; ++h) {
        const long long o = __shfl_sync(kAll, key, h << shift);
        if (((near >> (h << shift)) & 1u) && (o > key || (o == key && h < mine))) ++ahead;
    }
    return sure | __ballot_sync(kAll, is && ahead < need);
}

// The k best of the n experts in u.id, by their 64-bit values: lane j's expert.
__device__ __noinline__ int best64(const SelectArgs &a, const float *L, float m, bool on_logits,
                                   int n, const Scratch &u) {
    const int lane = threadIdx.x & 31;
    values64(a, L, m, on_logits, n, u);
    for (int p = lane; p < n; p += 32) {
        const long long v = u.key[p];
        int ahead = 0;
        for (int o = 0; o < n; ++o) {
            const long long w = u.key[o];
            if (w > v || (w == v && o < p)) ++ahead;
        }
        if (ahead < a.k) u.slot[ahead].id = u.id[p];
    }
    __syncwarp();
    return u.slot[lane].id;
}

// k rounds over the row in shared memory (NaN: not to be chosen, or taken), where
// the candidates are more than a warp has lanes: lane j's expert and q, and the
// largest that was left (NaN: none).  False where fewer than k are numbers.
__device__ __noinline__ bool select_rounds(int E, int k, float *row, Ranked *mine, float *next) {
    const int lane = threadIdx.x & 31;
    for (int j = 0; j <= k; ++j) {
        float v = NAN;
        int at = 0;
        for (int e = lane; e < E; e += 32) {
            const float x = row[e];
            if (x > v || (isnan(v) && !isnan(x))) {
                v = x;
                at = e;
            }
        }
        const float top = warp_max(v);
        if (j == k) {
            *next = top;
            break;
        }
        if (isnan(top)) return false;
        const int e = (int)__reduce_min_sync(kAll, v == top ? (unsigned)at : 0xffffffffu);
        if (lane == j) *mine = {top, e};
        __syncwarp();
        if (lane == 0) row[e] = NAN;
        __syncwarp();
    }
    return true;
}

// A warp per token, several tokens one after the other where there are many.
// VPL: values a lane has room for (>= a.per).  EXACT: the ranking is that of the
// logits themselves (no bias, and no group sums).
//
// The k-th largest of the lanes' maxima is a bound that k values reach, and few
// more (with k = 8 and 8 values a lane about 10, with k = 16 about 21): these
// candidates are gathered in shared memory, one a lane, and each counts those ahead
// of it, instead of k rounds of a warp maximum with its removal.
template <int VPL, bool EXACT>
__global__ void __launch_bounds__(256, VPL <= 8 ? 4 : VPL <= 16 ? 3 : VPL <= 32 ? 2 : 1)
select_kernel(const __grid_constant__ SelectArgs a) {
    pdl_entry();
    if (a.zero_word != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.zero_word = 0u;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5, wid = threadIdx.x >> 5;
    const int E = a.E;
    const int group = lane >> a.shift, r = lane & ((1 << a.shift) - 1);
    const int e0 = group * a.size + r * a.per;
    const int count = group < a.G ? max(0, min(a.per, a.size - r * a.per)) : 0;
    const bool whole = VPL % 4 == 0 && a.per == VPL && (E & 3) == 0 && (a.size & 3) == 0;
    const unsigned below = (1u << lane) - 1u;
    const Scratch u = scratch_of(smem, wid, E);
    u.few[lane] = kNobody;
    u.slot[lane] = kNobody;

    for (int64_t t = (int64_t)blockIdx.x * warps + wid; t < a.T; t += (int64_t)gridDim.x * warps) {
        float *L = a.logits + t * E;
        float v[VPL];  // NaN: no expert
        if (a.nparts > 0) {
            const float *p = a.partial + t * E;
#pragma unroll
            for (int i = 0; i < VPL; ++i) v[i] = i < count ? p[e0 + i] : NAN;
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
        } else if (whole) {
#pragma unroll
            for (int i = 0; i + 3 < VPL; i += 4) {
                float4 x = make_float4(NAN, NAN, NAN, NAN);
                if (i < count) x = *reinterpret_cast<const float4 *>(L + e0 + i);
                v[i] = x.x;
                v[i + 1] = x.y;
                v[i + 2] = x.z;
                v[i + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) v[i] = i < count ? L[e0 + i] : NAN;
        }
        __syncwarp();  // (the row as written, and the last token's slots as read)

        // softmax, where scores or their sum are needed: the largest logit m, and z
        float m = -INFINITY, z = 1.f;
        if (!a.sigmoid && (!EXACT || !a.renorm)) {
            float top = v[0];
#pragma unroll
            for (int i = 1; i < VPL; ++i) top = fmaxf(top, v[i]);
            top = warp_max(top);
            if (!isnan(top)) m = top;
            z = 0.f;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (i < count) z += exp2_fast((v[i] - m) * kLog2e);
            z = warp_sum(z);
        }
        if constexpr (!EXACT) {
            const float inv = m == -INFINITY ? 0.f : 1.f / z;
            if (a.sigmoid) {
#pragma unroll
                for (int i = 0; i < VPL; ++i) v[i] = rcp_fast(1.f + exp2_fast(v[i] * -kLog2e));
            } else {
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    v[i] = m == -INFINITY && i < count ? 0.f : exp2_fast((v[i] - m) * kLog2e) * inv;
            }
            if (a.bias) {
                if (whole && count == VPL) {
#pragma unroll
                    for (int i = 0; i + 3 < VPL; i += 4) {
                        const float4 b = *reinterpret_cast<const float4 *>(a.bias + e0 + i);
                        v[i] += b.x;
                        v[i + 1] += b.y;
                        v[i + 2] += b.z;
                        v[i + 3] += b.w;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < VPL; ++i)
                        if (i < count) v[i] += a.bias[e0 + i];
                }
            }
        }
        // How far two values of q have to be apart for fp32 to rank them.  Sigmoid:
        // the exponential 2 ulp and its argument's rounding, 2^-24 |L|, times s (1 - s)
        // and |L| s (1 - s) < 0.3; the sum half an ulp, the reciprocal one: below
        // 2^-22.  Softmax: the argument's two roundings give the exponential
        // 2^-23 |L - m| of itself, and x e^-x < 0.4; the exponential 2 ulp, the sum of
        // VPL + 5 terms in series half an ulp each, reciprocal and product: below
        // (VPL + 12) 2^-23 of the largest score 1/z.  q itself is rounded to 2^-24 of
        // its size.  Twice that for two values, and some room.
        float unit = 0.f;
        if constexpr (!EXACT)
            unit = a.sigmoid ? 8.f * 0x1p-23f : 2.f * (VPL + 12) * 0x1p-23f * rcp_fast(z);
        auto open = [&](float hi, float lo) {  // also where either is a NaN or both are infinite
            return !(hi - lo > unit + 0x1p-22f * fmaxf(fabsf(hi), fabsf(lo)));
        };
        const bool exact = EXACT || !a.bias;  // v are logits, from the choice among the experts on

        float best = NAN;
        unsigned kept = kAll;
        if (a.Gk < a.G) {
            float score, floor32;
            if (EXACT || !a.top2 || a.size == 1) {
                best = v[0];
#pragma unroll
                for (int i = 1; i < VPL; ++i) best = fmaxf(best, v[i]);
                score = best;
                for (int o = 1; o < (1 << a.shift); o <<= 1)
                    score = fmaxf(score, __shfl_xor_sync(kAll, score, o));
                floor32 = score;
            } else {
                float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    b2 = fmaxf(b2, v[i] > b1 ? b1 : v[i]);
                    b1 = fmaxf(b1, v[i]);
                }
                best = b1;
                for (int o = 1; o < (1 << a.shift); o <<= 1) {
                    const float o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
                    b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
                    b1 = fmaxf(b1, o1);
                }
                // (no second number, or an excluded expert: left to groups64)
                score = group < a.G && b2 > -INFINITY ? b1 + b2 : NAN;
                floor32 = isnan(score) ? NAN : b2;
            }
            // the Gk-th largest score, and the groups that reach it or come near
            const bool head = r == 0 && group < a.G;
            float cur = head ? score : NAN, bound = NAN;
            for (int j = 0; j < a.Gk;) {
                const float top = warp_max(cur);
                if (isnan(top)) break;
                bound = top;
                j += __popc(__ballot_sync(kAll, cur == top));
                if (cur == top) cur = NAN;
            }
            // (a sum has the errors of its two values and its own rounding)
            const float off = EXACT ? 0.f : 2.f * unit + 0x1p-21f * fabsf(bound);
            const unsigned reach = __ballot_sync(kAll, head && !(score < bound - off));
            if (__popc(reach) == a.Gk) {
                kept = reach;
            } else {
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if (i < count) u.row[e0 + i] = v[i];
                __syncwarp();
                const unsigned sure = __ballot_sync(kAll, head && score > bound + off);
                if (!EXACT) floor32 -= unit + 0x1p-22f * fabsf(floor32);
                kept = groups64(a, L, m, EXACT, sure, reach & ~sure, a.Gk - __popc(sure), floor32, u);
            }
            // without a bias the order inside the groups is that of the logits
            if (!EXACT && !a.bias) {
                best = NAN;
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    v[i] = i < count ? L[e0 + i] : NAN;
                    best = fmaxf(best, v[i]);
                }
            }
            if (((kept >> (group << a.shift)) & 1u) == 0u) {
                best = NAN;
#pragma unroll
                for (int i = 0; i < VPL; ++i) v[i] = NAN;
            }
        } else {
            best = v[0];
#pragma unroll
            for (int i = 1; i < VPL; ++i) best = fmaxf(best, v[i]);
        }

        // a bound that k values reach: the k-th largest distinct maximum of a lane
        float bound = -INFINITY;
        for (int j = 0; j < a.k; ++j) {
            const float top = warp_max(best);
            if (isnan(top)) {  // fewer lanes than that: every value
                bound = -INFINITY;
                break;
            }
            bound = top;
            if (best == top) best = NAN;
        }
        // the values that the chosen ones are among, and those too near to rank
        const float floor32 = exact ? bound : bound - (unit + 0x1p-21f * fabsf(bound));
        int n = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool in = v[i] >= floor32;
            const unsigned b = __ballot_sync(kAll, in);
            if (b == 0u) continue;
            const int at = n + __popc(b & below);
            if (in && at < 32) u.few[at] = {v[i], e0 + i};
            n += __popc(b);
        }
        __syncwarp();
        Ranked mine = u.few[lane];
        bool undecided;
        if (n >= a.k && n <= 32) {
            int ahead = 0;
            for (int p = 0; p < n; p += 4) {  // (nobody: NaN, ahead of none)
                const float4 x = *reinterpret_cast<const float4 *>(u.few + p);
                const float4 y = *reinterpret_cast<const float4 *>(u.few + p + 2);
                ahead += (x.x > mine.q) + (x.z > mine.q) + (y.x > mine.q) + (y.z > mine.q);
            }
            if (lane < n) u.slot[ahead] = mine;
            __syncwarp();
            u.few[lane] = kNobody;
            const int id = mine.id;
            mine = u.slot[lane];  // (equal values leave a slot after them empty)
            const float above = __shfl_up_sync(kAll, mine.q, 1);
            undecided = __any_sync(kAll, lane > 0 && lane <= a.k && lane < n &&
                                             (exact ? isnan(mine.q) : open(above, mine.q)));
            if (undecided) {
                if (lane < n) u.id[lane] = (uint16_t)id;
                __syncwarp();
                // (in ascending order: equal values go to the lower place)
                if (lane < n) {
                    int place = 0;
                    for (int p = 0; p < n; ++p) place += u.id[p] < id;
                    u.row[place] = __int_as_float(id);
                }
                __syncwarp();
                if (lane < n) u.id[lane] = (uint16_t)__float_as_int(u.row[lane]);
                __syncwarp();
                mine.id = best64(a, L, m, exact, n, u);
                __syncwarp();
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (i < count) u.row[e0 + i] = v[i];
            u.few[lane] = kNobody;
            __syncwarp();
            float next = NAN;
            undecided = !select_rounds(E, a.k, u.row, &mine, &next);
            if (!exact) {
                const float above = __shfl_up_sync(kAll, mine.q, 1);
                bool o = lane > 0 && lane < a.k && open(above, mine.q);
                if (lane == a.k - 1 && !isnan(next)) o |= open(mine.q, next);
                undecided |= __any_sync(kAll, o) != 0;
            }
            if (undecided) {  // (the rounds took values out of the row)
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if (i < count) u.row[e0 + i] = v[i];
                __syncwarp();
                const int c = list_experts(E, u, [&](int e) {
                    return e < E && ((kept >> (min(e, E - 1) / a.size << a.shift)) & 1u) &&
                           !(u.row[e] < floor32);
                });
                mine.id = best64(a, L, m, exact, c, u);
                __syncwarp();
            }
        }
        u.slot[lane] = kNobody;
        const int my_e = mine.id;

        // the weights, a slot a lane
        const bool slot = lane < a.k;
        const float logit = slot ? L[my_e] : -INFINITY;
        float w;
        if (a.sigmoid || a.renorm) {
            float s = a.sigmoid ? rcp_fast(1.f + expf(-logit)) : 0.f;
            float sum = 1.f;
            if (a.sigmoid && a.renorm) sum = slots_sum(slot ? s : 0.f, a.half);
            if (a.renorm && (!a.sigmoid || sum < 0x1p-100f)) {
                // shares of exponentials, shifted by the largest chosen logit; so too
                // sigmoids that underflow together, where 1 + exp(L) is 1
                const float top = slots_max(logit, a.half);
                s = !slot || top == -INFINITY ? 0.f : expf(logit - top);
                sum = slots_sum(s, a.half);
                if (top == -INFINITY) sum = 1.f;
            }
            w = a.scale * __fdividef(s, sum);
        } else {
            w = m == -INFINITY ? 0.f : a.scale * __fdividef(expf(logit - m), z);
        }
        if (slot) {
            a.idx[t * a.k + lane] = my_e;
            a.w[t * a.k + lane] = w;
        }
    }
}

template <int VPL>
cudaError_t launch_select_v(const SelectArgs &a, bool exact, cudaStream_t st) {
    const int threads = 256, warps = threads / 32;
    const size_t smem = (size_t)warps * scratch_bytes(a.E);
    // as many blocks as stay resident (8 of 32 registers a thread), then more tokens a warp
    const int64_t blocks = (a.T + warps - 1) / warps;
    const dim3 grid((unsigned)std::min<int64_t>(blocks, (int64_t)device_sm_count() * 8));
    if (smem > 48 * 1024) {
        static OncePerDevice once;
        const cudaError_t e = once([](int) {
            const int most = 8 * scratch_bytes(1024);
            const cudaError_t err = cudaFuncSetAttribute(
                select_kernel<VPL, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
            return err != cudaSuccess
                       ? err
                       : cudaFuncSetAttribute(select_kernel<VPL, false>,
                                              cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        });
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(exact ? select_kernel<VPL, true> : select_kernel<VPL, false>, grid,
                      dim3(threads), smem, st, a);
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
    a.shift = 5;
    for (int g = 1; g < a.G; g <<= 1) --a.shift;
    a.per = (a.size + (1 << a.shift) - 1) >> a.shift;
    a.scale = r.scale;
    for (int h = 1; h < s.k; h <<= 1) a.half = h;
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
