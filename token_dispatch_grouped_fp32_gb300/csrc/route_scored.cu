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
    int per_group;  // 2^20 / size, rounded up: e * per_group >> 20 is e's group
    float scale;
    int32_t *idx;
    float *w;
    unsigned *zero_word;
};

// A candidate, or a slot of the selection.
struct __align__(8) Ranked {
    float q;
    int id;
};
constexpr Ranked kNobody = {NAN, 0};

// A warp's shared memory: candidates and slots, and for the tokens that they do
// not settle the row of q, with a list of experts and their 64-bit values.
struct Scratch {
    Ranked *slot;         // [32]
    long long *key;       // [E]
    float *row;           // [E]
    uint16_t *id;         // [E]
};
__host__ __device__ inline int scratch_bytes(int E) { return 256 + ((14 * E + 15) & ~15); }
__device__ __forceinline__ Scratch scratch_of(unsigned char *p, int E) {
    return {reinterpret_cast<Ranked *>(p), reinterpret_cast<long long *>(p + 256),
            reinterpret_cast<float *>(p + 256 + 8 * E),
            reinterpret_cast<uint16_t *>(p + 256 + 12 * E)};
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

// The 64-bit values of the n experts in u.id, to u.key.  One logit for all of many
// (a padded row's): one score.
__device__ __noinline__ void values64(const SelectArgs &a, const float *L, float m, bool on_logits,
                                      int n, const Scratch &u) {
    const int lane = threadIdx.x & 31;
    const double z = a.sigmoid || on_logits || m == -INFINITY ? 1.0 : softmax_sum64(L, a.E, m);
    bool same = n > 32;
    float first = 0.f;
    if (same) {
        first = L[u.id[0]];
        for (int p = lane; p < n; p += 32)
            same = same && __float_as_uint(L[u.id[p]]) == __float_as_uint(first);
        same = __all_sync(kAll, same);
    }
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

__device__ __forceinline__ int group_of(const SelectArgs &a, int e) { return e * a.per_group >> 20; }

// The experts for which in(e) holds, in ascending order, to u.id.
template <typename F> __device__ __forceinline__ int list_experts(int E, const Scratch &u, F in) {
    const int lane = threadIdx.x & 31;
    int n = 0;
#pragma unroll 8
    for (int e0 = 0; e0 < E; e0 += 32) {
        const bool is = in(e0 + lane);
        const unsigned b = __ballot_sync(kAll, is);
        if (is) u.id[n + __popc(b & ((1u << lane) - 1u))] = (uint16_t)(e0 + lane);
        n += __popc(b);
    }
    __syncwarp();
    return n;
}

// The best `need` of the groups in `near` (bit g), by their 64-bit scores.  u.row:
// every q; floor32 (lane g: its group's): only values from there up can be of the
// score.
__device__ __noinline__ unsigned groups64(const SelectArgs &a, const float *L, float m,
                                          bool on_logits, unsigned near, int need, float floor32,
                                          const Scratch &u) {
    const int lane = threadIdx.x & 31;
    const int n = list_experts(a.E, u, [&](int e) {
        const int g = group_of(a, min(e, a.E - 1));
        const float f = __shfl_sync(kAll, floor32, g);
        return e < a.E && ((near >> g) & 1u) && !(u.row[e] < f);
    });
    values64(a, L, m, on_logits, n, u);
    const bool is = ((near >> lane) & 1u) != 0;
    long long key = kNaNKey;
    if (is) {
        long long b1 = kNaNKey, b2 = kNaNKey;
        for (int p = 0; p < n; ++p) {
            if (group_of(a, u.id[p]) != lane) continue;
            const long long v = u.key[p];
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
        const long long o = __shfl_sync(kAll, key, h);
        if (((near >> h) & 1u) && (o > key || (o == key && h < lane))) ++ahead;
    }
    return __ballot_sync(kAll, is && ahead < need);
}

// How far two values of q have to be apart for fp32 to rank them.  Sigmoid: the
// exponential 2 ulp and its argument's rounding, 2^-24 |L|, times s (1 - s), and
// |L| s (1 - s) < 0.3; the sum half an ulp, the reciprocal one: below 2^-22 (two
// values 4 * 2^-23).
// Softmax: the argument's two roundings give the exponential 2^-23 |L - m| of
// itself, and x e^-x < 0.4; the exponential 2 ulp, the sum of at most 37 terms in
// series (`terms` of them a lane) half an ulp each, reciprocal and product: below
// (terms + 12) 2^-23 of the largest score 1/z.  q itself is rounded to 2^-24 of its
// size, and so is a sum of two.  With some room.
__device__ __forceinline__ float unit_of(bool sigmoid, int terms, float z) {
    return sigmoid ? 4.5f * 0x1p-23f : 2.f * (terms + 12) * 0x1p-23f * rcp_fast(z);
}
// (true also where either is a NaN or both are infinite)
__device__ __forceinline__ bool too_near(float hi, float lo, float unit) {
    return !(hi - lo > unit + 0x1.2p-23f * fmaxf(fabsf(hi), fabsf(lo)));
}

__device__ __forceinline__ float score32(float L, bool sigmoid, float m, float inv) {
    if (sigmoid) return rcp_fast(1.f + exp2_fast(L * -kLog2e));
    return m == -INFINITY ? 0.f : exp2_fast((L - m) * kLog2e) * inv;
}

// A token's weights and ids.  A lane with `chosen` has the expert `id`, its logit and
// its slot; m, z: softmax without renormalisation.
__device__ __forceinline__ void write_slots(const SelectArgs &a, int64_t t, bool chosen, int slot, int id,
                                            float logit, float m, float z) {
    float w;
    if (a.sigmoid || a.renorm) {
        float s = a.sigmoid ? rcp_fast(1.f + expf(-logit)) : 0.f;
        float sum = 1.f;
        if (a.sigmoid && a.renorm) sum = warp_sum(chosen ? s : 0.f);
        if (a.renorm && (!a.sigmoid || sum < 0x1p-100f)) {
            // shares of exponentials, shifted by the largest chosen logit; so too
            // sigmoids that underflow together, where 1 + exp(L) is 1
            const float top = warp_max(chosen ? logit : NAN);
            s = !chosen || top == -INFINITY ? 0.f : expf(logit - top);
            sum = warp_sum(s);
            if (top == -INFINITY) sum = 1.f;
        }
        w = a.scale * s * rcp_fast(sum);
    } else {
        w = m == -INFINITY ? 0.f : a.scale * expf(logit - m) * rcp_fast(z);
    }
    if (chosen) {
        a.idx[t * a.k + slot] = id;
        a.w[t * a.k + slot] = w;
    }
}

// A token that the fast path below leaves open: ties, values or groups that fp32
// cannot rank, NaN, or more candidates than a warp has lanes.  From the beginning, for any
// sizes: candidates are ranked in fp32 where that settles them, else in fp64.
__device__ __noinline__ void decide(const SelectArgs &a, int64_t t, unsigned char *smem) {
    const int lane = threadIdx.x & 31, E = a.E;
    const Scratch u = scratch_of(smem, E);
    const float *L = a.logits + t * E;
    const bool by_logits = !a.bias && (a.Gk == a.G || !a.top2);
    __syncwarp();
    float m = -INFINITY, z = 1.f;
    if (!a.sigmoid) {
        float top = NAN;
        for (int e = lane; e < E; e += 32) top = fmaxf(top, L[e]);
        top = warp_max(top);
        if (!isnan(top)) m = top;
        z = 0.f;
#pragma unroll 4
        for (int e = lane; e < E; e += 32) z += exp2_fast((L[e] - m) * kLog2e);
        z = warp_sum(z);
    }
    const float unit = by_logits ? 0.f : unit_of(a.sigmoid, (E + 31) / 32, z);
    const float inv = rcp_fast(z);
    for (int e0 = lane; e0 < E; e0 += 256) {
        float q[8], b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = min(e0 + 32 * i, E - 1);
            q[i] = L[e];
            b[i] = a.bias ? a.bias[e] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (!by_logits) q[i] = score32(q[i], a.sigmoid, m, inv);
            if (a.bias) q[i] += b[i];
            if (e0 + 32 * i < E) u.row[e0 + 32 * i] = q[i];
        }
    }
    __syncwarp();
    unsigned kept = 1u;
    if (a.Gk < a.G) {
        float b1 = NAN, b2 = NAN, score = NAN, floor32 = NAN, mag = 0.f;
        if (lane < a.G) {
            for (int i = 0; i < a.size; ++i) {
                const float x = u.row[lane * a.size + i];
                b2 = fmaxf(b2, x > b1 ? b1 : isnan(b1) ? NAN : x);
                b1 = fmaxf(b1, x);
            }
            const bool sum = a.top2 && a.size > 1;
            score = sum ? b1 + b2 : b1;
            floor32 = isnan(score) ? NAN : sum ? b2 : b1;
            if (!by_logits) floor32 -= unit + 0x1p-22f * fabsf(floor32);
            mag = isnan(score) ? 0.f : fabsf(b1) + (sum ? fabsf(b2) : 0.f);
        }
        float cur = score, bound = NAN;  // the Gk-th largest score
        for (int j = 0; j < a.Gk;) {
            const float top = warp_max(cur);
            if (isnan(top)) break;
            bound = top;
            j += __popc(__ballot_sync(kAll, cur == top));
            if (cur == top) cur = NAN;
        }
        const float off = by_logits ? 0.f : 2.f * unit + 0x1.2p-22f * warp_max(mag);
        const unsigned reach = __ballot_sync(kAll, lane < a.G && !(score < bound - off));
        kept = reach;
        if (__popc(reach) != a.Gk) {
            const unsigned sure = __ballot_sync(kAll, lane < a.G && score > bound + off);
            kept = sure | groups64(a, L, m, by_logits, reach & ~sure, a.Gk - __popc(sure), floor32, u);
        }
        if (!by_logits && !a.bias) {  // the order inside the groups is that of the logits
            for (int e = lane; e < E; e += 32) u.row[e] = L[e];
            __syncwarp();
        }
    }
    const bool exact = by_logits || !a.bias;
    auto stays = [&](int e) { return e < E && ((kept >> group_of(a, min(e, E - 1))) & 1u); };
    float best = NAN, bound = NAN;
#pragma unroll 4
    for (int e = lane; e < E; e += 32)
        if (stays(e)) best = fmaxf(best, u.row[e]);
    for (int j = 0; j < a.k; ++j) {
        bound = warp_max(best);
        if (best == bound) best = NAN;
    }
    if (isnan(bound)) bound = -INFINITY;  // fewer lanes than that: every value, and NaN
    const float floor32 = exact ? bound : bound - (unit + 0x1p-21f * fabsf(bound));
    const int n = list_experts(E, u, [&](int e) { return stays(e) && !(u.row[min(e, E - 1)] < floor32); });
    u.slot[lane] = kNobody;
    __syncwarp();
    // (few candidates that are not logits: two of them are too near, mostly)
    bool open = !exact && n <= 64;
    for (int p = lane; p < n && !open; p += 32) {
        const float q = u.row[u.id[p]];
        int ahead = 0;
        for (int o = 0; o < n; ++o) {
            const float x = u.row[u.id[o]];
            if (x > q || (x == q && o < p)) ++ahead;
            if (!exact && o != p && x >= q) open |= too_near(x, q, unit);
        }
        // (only neighbours of the first k matter; a NaN is for the 64-bit keys)
        if (isnan(q)) open = true;
        else if (ahead < a.k) u.slot[ahead] = {q, u.id[p]};
    }
    open = __any_sync(kAll, open);
    __syncwarp();
    if (open) {
        values64(a, L, m, exact, n, u);
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
    }
    const bool chosen = lane < a.k;
    const int id = chosen ? u.slot[lane].id : 0;
    write_slots(a, t, chosen, lane, id, L[id], m, z);
    __syncwarp();
}

// A warp per token, several tokens one after the other where there are many.
// VPL: values a lane has room for (>= a.per).  EXACT: the ranking is that of the
// logits themselves (no bias, and no group sums).
//
// The k-th largest of the lanes' maxima is a bound that k values reach, and few
// more (with k = 8 and 8 values a lane about 10, with k = 16 about 21): these
// candidates are gathered in shared memory, one a lane, and each counts those ahead
// of it, instead of k rounds of a warp maximum with its removal.  What this leaves
// open goes to decide(), after every 32 tokens: a call inside their loop cost it
// spills (T = 131072, E = 128: 43 us to 62).  Blocks of one warp: what depends on the
// token is uniform, which the compiler sees.
template <int VPL, bool EXACT, bool GROUPS>
__global__ void __launch_bounds__(32, VPL <= 8 ? 32 : 16)
select_kernel(const SelectArgs a, const __grid_constant__ SelectArgs cold) {
    pdl_entry();
    if (a.zero_word != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.zero_word = 0u;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x;
    const int E = a.E;
    const int group = GROUPS ? lane >> a.shift : 0;
    const int r = GROUPS ? lane & ((1 << a.shift) - 1) : lane;
    const int e0 = group * a.size + r * a.per;
    const int count = group < a.G ? max(0, min(a.per, a.size - r * a.per)) : 0;
    const bool whole = VPL % 4 == 0 && a.per == VPL && (E & 3) == 0 && (a.size & 3) == 0;
    const unsigned below = (1u << lane) - 1u;
    Ranked *few = reinterpret_cast<Ranked *>(smem);  // up to 32 VPL candidates

    for (int64_t t0 = blockIdx.x; t0 < a.T; t0 += 32 * (int64_t)gridDim.x) {
    unsigned left = 0u;  // of the tokens t0 + i * gridDim.x
    for (int i32 = 0; i32 < 32; ++i32) {
        const int64_t t = t0 + i32 * (int64_t)gridDim.x;
        if (t >= a.T) break;
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
        __syncwarp();  // (the row as written, and the last token's candidates as read)

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
            if (a.sigmoid) {
#pragma unroll
                for (int i = 0; i < VPL; ++i) v[i] = score32(v[i], true, 0.f, 0.f);
            } else {  // (m == -INF, a row without scores: its NaN are for decide())
                const float inv = rcp_fast(z);
#pragma unroll
                for (int i = 0; i < VPL; ++i) v[i] = exp2_fast((v[i] - m) * kLog2e) * inv;
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
        const float unit = EXACT ? 0.f : unit_of(a.sigmoid, VPL, z);
        const bool exact = EXACT || (GROUPS && !a.bias);  // v are logits, from here on

        float best;
        bool decided = true;
        if constexpr (GROUPS) {
            float score, mag = 0.f;
            if (EXACT || !a.top2 || a.size == 1) {
                best = v[0];
#pragma unroll
                for (int i = 1; i < VPL; ++i) best = fmaxf(best, v[i]);
                score = best;
                for (int o = 1; o < (1 << a.shift); o <<= 1)
                    score = fmaxf(score, __shfl_xor_sync(kAll, score, o));
                if (!EXACT) mag = fabsf(score);
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
                // (no second number, or an excluded expert: for decide())
                score = group < a.G && b2 > -INFINITY ? b1 + b2 : NAN;
                if (!isnan(score)) mag = fabsf(b1) + fabsf(b2);
            }
            // a score that Gk groups reach: if no more come near it, they stay
            float cur = score, bound = NAN;
            for (int j = 0; j < a.Gk; ++j) {
                bound = warp_max(cur);
                if (cur == bound) cur = NAN;
            }
            // (a sum has the errors of its two values and its own rounding)
            const float off = EXACT ? 0.f : 2.f * unit + 0x1.2p-22f * warp_max(mag);
            decided = __popc(__ballot_sync(kAll, r == 0 && group < a.G && !(score < bound - off))) == a.Gk;
            // without a bias the order inside the groups is that of the logits
            if (!EXACT && !a.bias) {
                best = NAN;
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    v[i] = i < count ? L[e0 + i] : NAN;
                    best = fmaxf(best, v[i]);
                }
            }
            if (!(score >= bound)) {
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
        float bound = NAN;
#pragma unroll 4
        for (int j = 0; j < a.k; ++j) {
            bound = warp_max(best);
            if (best == bound) best = NAN;
        }
        if (isnan(bound)) bound = -INFINITY;  // fewer lanes than that: every value
        // the values that the chosen ones are among, and those too near to rank
        const float floor32 = exact ? bound : bound - (unit + 0x1p-21f * fabsf(bound));
        int n = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool in = v[i] >= floor32;
            const unsigned b = __ballot_sync(kAll, in);
            if (VPL > 8 && b == 0u) continue;
            if (in) few[n + __popc(b & below)] = {v[i], e0 + i};
            n += __popc(b);
        }
        decided = decided && n >= a.k && n <= 32;
        __syncwarp();
        const Ranked mine = lane < n ? few[lane] : kNobody;
        // (loops of fixed length: with n for their limit, which is uniform but not
        // known to be, each of their warp operations took three times the instructions)
        unsigned ahead_of_me = 0u;  // (a NaN is ahead of none)
        auto rank = [&](int p) {
            const unsigned b = __ballot_sync(kAll, mine.q > __shfl_sync(kAll, mine.q, p));
            if (lane == p) ahead_of_me = b;
        };
#pragma unroll
        for (int p = 0; p < 12; ++p) rank(p);
        if (n > 12)
#pragma unroll
            for (int p = 12; p < 32; ++p) rank(p);
        const int ahead = __popc(ahead_of_me);
        const bool chosen = lane < n && ahead < a.k;
        // equal values have the same place
        decided &= __popc(__reduce_or_sync(kAll, lane < n ? 1u << ahead : 0u)) == n;
        if (!exact) {
            __syncwarp();
            if (lane < n) few[ahead] = mine;
            __syncwarp();
            const bool behind = chosen && ahead + 1 < n;
            const float next = few[behind ? ahead + 1 : 0].q;
            decided &= !__any_sync(kAll, behind && too_near(mine.q, next, unit));
        }
        if (decided) write_slots(a, t, chosen, ahead, mine.id,
                                 exact ? mine.q : chosen ? L[mine.id] : 0.f, m, z);
        if (!decided) left |= 1u << i32;
    }
    while (left) {
        const int i = __ffs(left) - 1;
        left &= left - 1u;
        decide(cold, t0 + i * (int64_t)gridDim.x, smem);
    }
    }
}

// Long batches: LANES lanes a token, 32 / LANES tokens a warp, N float4 of values a
// lane, k <= 8, no groups.  The same steps as above, at a fraction of the
// instructions a token, since a step of a reduction, a vote or a rank serves all of a
// warp's tokens: the bound from the maxima of half a lane's values each, candidates
// counted and placed by a prefix sum over the lanes, and two or four of them a lane.
constexpr int kManyK = 8, kManyFew = 32;

struct Segment {  // a token's shared memory; 200 words apart: no bank conflicts
    Ranked few[kManyFew];     // candidates, NaN behind them
    Ranked sorted[kManyFew];  // by rank; NaN where equal values leave a gap
    uint32_t pad[72];
};
static_assert(sizeof(Segment) % 128 == 32, "");

template <int LANES, bool MAX> __device__ __forceinline__ float segment_all(float v) {
#pragma unroll
    for (int o = LANES / 2; o >= 1; o >>= 1) {
        const float u = __shfl_xor_sync(kAll, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    return v;
}

template <int LANES, int N, bool EXACT>
__global__ void __launch_bounds__(32, 24)
select_many_kernel(const SelectArgs a, const __grid_constant__ SelectArgs cold) {
    pdl_entry();
    if (a.zero_word != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.zero_word = 0u;
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int kTokens = 32 / LANES, V = 4 * N;
    const int lane = threadIdx.x, seg = lane / LANES, l = lane % LANES, E = a.E;
    Segment &s = reinterpret_cast<Segment *>(smem)[seg];

    const int64_t stride = (int64_t)gridDim.x * kTokens;
    for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < a.T; t0 += LANES * stride) {
        unsigned left = 0u;  // bit LANES * seg + i: token t0 + i * stride + seg
        for (int i = 0; i < LANES; ++i) {
            const int64_t t = t0 + i * stride + seg;
            if (t - seg >= a.T) break;
            const bool there = t < a.T;
            float *L = a.logits + t * E;
            float v[V];  // NaN: no expert
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int e = 4 * (l + LANES * n);
                float4 x = make_float4(NAN, NAN, NAN, NAN);
                if (there && e < E) {
                    if (a.nparts > 0) {
                        const float *p = a.partial + t * E + e;
                        x = *reinterpret_cast<const float4 *>(p);
                        for (int z = 1; z < a.nparts; ++z) {
                            const float4 y = *reinterpret_cast<const float4 *>(p + z * a.T * E);
                            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                        }
                        if (a.logit_bias) {
                            const float4 y = *reinterpret_cast<const float4 *>(a.logit_bias + e);
                            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                        }
                        *reinterpret_cast<float4 *>(L + e) = x;
                    } else {
                        x = *reinterpret_cast<const float4 *>(L + e);
                    }
                }
                v[4 * n] = x.x;
                v[4 * n + 1] = x.y;
                v[4 * n + 2] = x.z;
                v[4 * n + 3] = x.w;
            }
            __syncwarp();  // (the last token's shared memory as read)
#pragma unroll
            for (int c = 2 * l; c < kManyFew; c += 2 * LANES) {
                const float4 none = make_float4(NAN, 0.f, NAN, 0.f);
                *reinterpret_cast<float4 *>(s.few + c) = none;
                *reinterpret_cast<float4 *>(s.sorted + c) = none;
            }

            float m = -INFINITY, z = 1.f;
            if (!a.sigmoid && (!EXACT || !a.renorm)) {
                float top = v[0];
#pragma unroll
                for (int j = 1; j < V; ++j) top = fmaxf(top, v[j]);
                top = segment_all<LANES, true>(top);
                if (!isnan(top)) m = top;
                z = 0.f;
#pragma unroll
                for (int n = 0; n < N; ++n)
                    if (4 * (l + LANES * n) < E)
#pragma unroll
                        for (int j = 0; j < 4; ++j) z += exp2_fast((v[4 * n + j] - m) * kLog2e);
                z = segment_all<LANES, false>(z);
            }
            if constexpr (!EXACT) {
                if (a.sigmoid) {
#pragma unroll
                    for (int j = 0; j < V; ++j) v[j] = score32(v[j], true, 0.f, 0.f);
                } else {
                    const float inv = rcp_fast(z);
#pragma unroll
                    for (int j = 0; j < V; ++j) v[j] = exp2_fast((v[j] - m) * kLog2e) * inv;
                }
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int e = 4 * (l + LANES * n);
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (e < E) x = __ldg(reinterpret_cast<const float4 *>(a.bias + e));
                    v[4 * n] += x.x;
                    v[4 * n + 1] += x.y;
                    v[4 * n + 2] += x.z;
                    v[4 * n + 3] += x.w;
                }
            }
            const float unit = EXACT ? 0.f : unit_of(a.sigmoid, V, z);

            float b0 = v[0], b1 = v[V / 2], bound = NAN;
#pragma unroll
            for (int j = 1; j < V / 2; ++j) {
                b0 = fmaxf(b0, v[j]);
                b1 = fmaxf(b1, v[V / 2 + j]);
            }
#pragma unroll
            for (int j = 0; j < kManyK; ++j) {
                if (j >= a.k) break;
                bound = segment_all<LANES, true>(fmaxf(b0, b1));
                if (b0 == bound) b0 = NAN;
                if (b1 == bound) b1 = NAN;
            }
            if (isnan(bound)) bound = -INFINITY;
            const float floor32 = EXACT ? bound : bound - (unit + 0x1p-21f * fabsf(bound));
            int mine = 0;
#pragma unroll
            for (int j = 0; j < V; ++j) mine += v[j] >= floor32;
            int upto = mine;  // with the lanes below
#pragma unroll
            for (int o = 1; o < LANES; o <<= 1) {
                const int u = __shfl_up_sync(kAll, upto, o, LANES);
                if (l >= o) upto += u;
            }
            const int n = __shfl_sync(kAll, upto, LANES - 1, LANES);
            int at = upto - mine;
            __syncwarp();
            if (n <= kManyFew) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (v[j] >= floor32) s.few[at++] = {v[j], 4 * (l + LANES * (j / 4)) + j % 4};
            }
            __syncwarp();
            // ranks, by the values behind each: by the sign of a difference, two a packed sum
            constexpr int kHold = kManyFew / LANES;  // candidates a lane: 4, or 2
            Ranked c[kHold];
            int behind[kHold];
#pragma unroll
            for (int j = 0; j < kHold; ++j) {
                c[j] = s.few[l + LANES * j];
                behind[j] = 0;
            }
            auto rank = [&](int p, int j) {
                const float4 x = *reinterpret_cast<const float4 *>(s.few + p);  // (q, id) twice
                const float2 d = add2(make_float2(x.x, x.z), make_float2(-c[j].q, -c[j].q));
                behind[j] += (int)(__float_as_uint(d.x) >> 31) + (int)(__float_as_uint(d.y) >> 31);
            };
#pragma unroll
            for (int p = 0; p < 16; p += 2) {
                rank(p, 0);
                rank(p, 1);
            }
            if (__any_sync(kAll, n > 16)) {  // (uniform)
#pragma unroll
                for (int p = 0; p < kManyFew; p += 2)
#pragma unroll
                    for (int j = p < 16 ? 2 : 0; j < kHold; ++j) rank(p, j);
            }
#pragma unroll
            for (int j = 0; j < kHold; ++j)
                if (l + LANES * j < n && n <= kManyFew) s.sorted[n - 1 - behind[j]] = c[j];
            __syncwarp();
            const bool slot = l < a.k;
            const Ranked chosen = s.sorted[l];
            const float q = chosen.q, next = s.sorted[l + 1].q;
            const bool bad = there && slot &&
                             (n > kManyFew || isnan(q) ||
                              (l + 1 < n && (EXACT ? !(q > next) : too_near(q, next, unit))));
            unsigned open = __ballot_sync(kAll, bad);
#pragma unroll
            for (int o = LANES / 2; o >= 1; o >>= 1) open |= open >> o;  // each segment's any, in its bit 0
            open &= LANES == 8 ? 0x01010101u : 0x00010001u;
            left |= open << i;

            const bool write = there && slot && ((open >> (LANES * seg)) & 1u) == 0u;
            const int id = write ? chosen.id : 0;
            const float logit = !write ? -INFINITY : EXACT ? q : L[id];
            float w;
            if (a.sigmoid || a.renorm) {
                float x = a.sigmoid ? rcp_fast(1.f + expf(-logit)) : 0.f;
                float sum = 1.f;
                if (a.sigmoid && a.renorm) sum = segment_all<LANES, false>(slot ? x : 0.f);
                if (a.renorm && __any_sync(kAll, !a.sigmoid || (write && sum < 0x1p-100f))) {
                    // (as in write_slots; for all of the warp's tokens, if one needs it)
                    const float top = segment_all<LANES, true>(logit);
                    const bool here = !a.sigmoid || sum < 0x1p-100f;
                    const float y = !write || top == -INFINITY ? 0.f : expf(logit - top);
                    const float shares = segment_all<LANES, false>(y);
                    if (here) {
                        x = y;
                        sum = top == -INFINITY ? 1.f : shares;
                    }
                }
                w = a.scale * x * rcp_fast(sum);
            } else {
                w = m == -INFINITY ? 0.f : a.scale * expf(logit - m) * rcp_fast(z);
            }
            if (write) {
                a.idx[t * a.k + l] = id;
                a.w[t * a.k + l] = w;
            }
        }
        while (left) {
            const int bit = __ffs(left) - 1;
            left &= left - 1u;
            decide(cold, t0 + bit % LANES * stride + bit / LANES, smem);
        }
    }
}

template <int LANES, int N>
cudaError_t launch_many(const SelectArgs &a, bool exact, cudaStream_t st) {
    constexpr int kTokens = 32 / LANES;
    const size_t smem = std::max<size_t>(scratch_bytes(a.E), sizeof(Segment) * kTokens);
    const dim3 grid((unsigned)std::min<int64_t>((a.T + kTokens - 1) / kTokens,
                                                (int64_t)device_sm_count() * 24));
    return launch_pdl(exact ? select_many_kernel<LANES, N, true> : select_many_kernel<LANES, N, false>,
                      grid, dim3(32), smem, st, a, a);
}
// From this many tokens on (measured below).
constexpr int64_t kManyTokens = 16384;
bool takes_many(const SelectArgs &a) {
    return a.Gk == a.G && a.k <= kManyK && a.E % 4 == 0 && a.E >= 32 && a.E <= 256 && a.T >= kManyTokens;
}

template <int VPL, bool EXACT, bool GROUPS>
cudaError_t launch_select_t(const SelectArgs &a, cudaStream_t st) {
    const size_t smem = std::max<size_t>(scratch_bytes(a.E), sizeof(Ranked) * (32 * VPL + 4));
    // as many blocks as stay resident, then more tokens a block
    const dim3 grid((unsigned)std::min<int64_t>(a.T, (int64_t)device_sm_count() * 32));
    return launch_pdl(select_kernel<VPL, EXACT, GROUPS>, grid, dim3(32), smem, st, a, a);
}
template <int VPL> cudaError_t launch_select_v(const SelectArgs &a, bool exact, cudaStream_t st) {
    if (a.Gk < a.G)
        return exact ? launch_select_t<VPL, true, true>(a, st) : launch_select_t<VPL, false, true>(a, st);
    return exact ? launch_select_t<VPL, true, false>(a, st) : launch_select_t<VPL, false, false>(a, st);
}

// ------------------------- gradient to the logits --------------------------
//   softmax, renormalised:  dl[idx_j] = w_j (d_j - S/c)
//   softmax:                dl[e]     = s_e (c g_e - S),  g_e = d_j where e = idx_j
//   sigmoid, renormalised:  dl[idx_j] = w_j (d_j - S/c) (1 - s_j)
//   sigmoid:                dl[idx_j] = w_j d_j (1 - s_j)
// with S = sum_j w_j d_j.  LANES lanes per token: its row's chosen entries in shared
// memory, zero elsewhere, then written whole, W columns a lane at a time (four where
// E allows it).  The fewer lanes a token, the fewer steps its sums take; with
// eight columns a lane T = 131072, E = 128 (softmax, all logits) takes 16 lanes, X us against
// 34.7 with 32, bound by HBM.
constexpr int kGradThreads = 256;

struct GradArgs {
    const float *logits;
    const int32_t *idx;
    const float *w, *dw;
    int64_t T;
    int E, k;
    ScoreGrad f;
    float *dl;
};

template <int LANES> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

template <int W> struct Columns;
template <> struct Columns<4> { using V = float4; };
template <> struct Columns<1> { using V = float; };

// DENSE: softmax that is not renormalised, N times W columns a lane
template <bool DENSE, int W, int LANES, int N>
__global__ void __launch_bounds__(kGradThreads)
logits_grad_kernel(const GradArgs a, DevStatus ds) {
    pdl_wait();
    using V = typename Columns<W>::V;
    extern __shared__ __align__(16) float rows[];
    const int E = a.E, l = threadIdx.x % LANES, own = threadIdx.x / LANES;
    const int stride = (E + 3) & ~3;
    const int64_t t = (int64_t)blockIdx.x * (kGradThreads / LANES) + own;
    const bool there = t < a.T;
    float *row = rows + own * stride;
    for (int c = W * l; c < E; c += W * LANES)
#pragma unroll
        for (int i = 0; i < W; ++i) row[c + i] = 0.f;
    const float *L = a.logits + t * E;
    float *o = a.dl + t * E;
    // the logits first: nothing waits for them but the last sums
    float v[N][W];
    if constexpr (DENSE) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = (l + LANES * n) * W;
            if (there && c < E) {
                *reinterpret_cast<V *>(v[n]) = *reinterpret_cast<const V *>(L + c);
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i) v[n][i] = -INFINITY;
            }
        }
    }
    float S = 0.f;
    int e[32 / LANES];  // this lane's slots l, l + LANES, ...
    float wj[32 / LANES], dj[32 / LANES];
#pragma unroll
    for (int q = 0; q < 32 / LANES; ++q) {
        const int j = l + LANES * q;
        e[q] = -1;
        wj[q] = dj[q] = 0.f;
        if (there && j < a.k) {
            e[q] = a.idx[t * a.k + j];
            wj[q] = a.w[t * a.k + j];
            dj[q] = a.dw[t * a.k + j];
            if ((unsigned)e[q] >= (unsigned)E) {
                raise_error(ds, kErrBadRouting);
                e[q] = -1;
                wj[q] = dj[q] = 0.f;
            }
        }
        S += wj[q] * dj[q];
    }
    S = lanes_sum<LANES>(S);
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 32 / LANES; ++q)
        if (e[q] >= 0)
            row[e[q]] = DENSE ? a.f.scale * dj[q]
                              : a.f.chosen(wj[q], dj[q], S, a.f.sigmoid ? L[e[q]] : 0.f);
    __syncwarp();
    if constexpr (!DENSE) {
        if (there)
            for (int c = W * l; c < E; c += W * LANES)
                *reinterpret_cast<V *>(o + c) = *reinterpret_cast<const V *>(row + c);
    } else {
        float m = -INFINITY, z = 0.f;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < W; ++i) m = fmaxf(m, v[n][i]);
#pragma unroll
        for (int q = LANES / 2; q >= 1; q >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, q));
        if (m == -INFINITY) m = 0.f;  // all masked: exponentials of 0, and no scores
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < W; ++i) {
                v[n][i] = exp2_fast((v[n][i] - m) * kLog2e);
                z += v[n][i];
            }
        z = lanes_sum<LANES>(z);
        const float inv = z > 0.f || isnan(z) ? 1.f / z : 0.f;
        if (!there) return;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = (l + LANES * n) * W;
            if (c >= E) continue;
            float g[W];
            *reinterpret_cast<V *>(g) = *reinterpret_cast<const V *>(row + c);
#pragma unroll
            for (int i = 0; i < W; ++i) g[i] = v[n][i] * inv * (g[i] - S);
            *reinterpret_cast<V *>(o + c) = *reinterpret_cast<const V *>(g);
        }
    }
}

template <bool DENSE, int W, int LANES, int N>
cudaError_t launch_grad(const GradArgs &a, const DevStatus &ds, cudaStream_t st) {
    constexpr int kTokens = kGradThreads / LANES;
    const dim3 grid((unsigned)((a.T + kTokens - 1) / kTokens));
    const size_t smem = sizeof(float) * kTokens * (size_t)((a.E + 3) & ~3);
    return launch_pdl(logits_grad_kernel<DENSE, W, LANES, N>, grid, dim3(kGradThreads), smem, st, a, ds);
}

template <bool DENSE> cudaError_t launch_grad_any(const GradArgs &a, const DevStatus &ds, cudaStream_t st) {
    if (a.E % 4 == 0) {  // two float4 a lane, and from E = 257 on more
        if (a.E <= 64) return launch_grad<DENSE, 4, 8, 2>(a, ds, st);
        if (a.E <= 128) return launch_grad<DENSE, 4, 16, 2>(a, ds, st);
        if (a.E <= 256 || !DENSE) return launch_grad<DENSE, 4, 32, 2>(a, ds, st);
        if (a.E <= 512) return launch_grad<DENSE, 4, 32, 4>(a, ds, st);
        return launch_grad<DENSE, 4, 32, 8>(a, ds, st);
    }
    if (a.E <= 64) return launch_grad<DENSE, 1, 8, 8>(a, ds, st);
    if (a.E <= 128) return launch_grad<DENSE, 1, 16, 8>(a, ds, st);
    if (a.E <= 256 || !DENSE) return launch_grad<DENSE, 1, 32, 8>(a, ds, st);
    if (a.E <= 512) return launch_grad<DENSE, 1, 32, 16>(a, ds, st);
    return launch_grad<DENSE, 1, 32, 32>(a, ds, st);
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
    a.per_group = (1 << 20) / a.size + 1;  // (e < 1024: off by less than 1 / size)
    a.shift = 5;
    for (int g = 1; g < a.G; g <<= 1) --a.shift;
    a.per = (a.size + (1 << a.shift) - 1) >> a.shift;
    a.scale = r.scale;
    a.idx = idx;
    a.w = w;
    a.zero_word = zero_word;
    const bool exact = !bias && (a.Gk == a.G || !a.top2);
    cudaError_t e;
    if (takes_many(a)) {
        if (a.E <= 64) e = launch_many<8, 2>(a, exact, st);
        else if (a.E <= 128) e = launch_many<8, 4>(a, exact, st);
        else e = launch_many<16, 4>(a, exact, st);
    }
    else if (a.per <= 1) e = launch_select_v<1>(a, exact, st);
    else if (a.per <= 2) e = launch_select_v<2>(a, exact, st);
    else if (a.per <= 4) e = launch_select_v<4>(a, exact, st);
    else if (a.per <= 8) e = launch_select_v<8>(a, exact, st);
    else if (a.per <= 16) e = launch_select_v<16>(a, exact, st);
    else if (a.per <= 32) e = launch_select_v<32>(a, exact, st);
    else if (exact) e = launch_select_t<64, true, true>(a, st);  // few lanes a group: 9 to 31 groups
    else e = launch_select_t<64, false, true>(a, st);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_logits_grad(const Shape &s, const ScoreGrad &f, const float *logits,
                               const int32_t *idx, const float *w, const float *dw, float *dlogits,
                               const DevStatus &ds, cudaStream_t st) {
    const GradArgs a = {logits, idx, w, dw, s.T, s.E, s.k, f, dlogits};
    const cudaError_t e = f.dense ? launch_grad_any<true>(a, ds, st) : launch_grad_any<false>(a, ds, st);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_balance(const int32_t *counts, int64_t layers, int E, float rate, float *bias,
                           float *imbalance, cudaStream_t st) {
    const cudaError_t e = launch_pdl(balance_kernel, dim3((unsigned)layers), dim3(kBalanceThreads), 0,
                                     st, counts, E, rate, bias, imbalance);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
