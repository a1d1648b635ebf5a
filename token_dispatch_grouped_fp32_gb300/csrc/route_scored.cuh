// route_scored.cuh -- what the selections of route_scored.cu and route_scored_many.cu
// share: the device code of one token that fp32 leaves open, and of its weights.
#pragma once

#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {

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
    int pending_at;  // where in the shared memory a warp keeps what it could not rank
    int32_t *idx;
    float *w;
    unsigned *zero_word;
};

// Long batches (route_scored_many.cu): whether, and their launch.
bool select_takes_many(const SelectArgs &a, bool exact);
cudaError_t launch_select_many(const SelectArgs &a, bool exact, cudaStream_t st);

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

// A candidate, or a slot of the selection.
struct __align__(8) Ranked {
    float q;
    int id;
};
constexpr Ranked kNobody = {NAN, 0};

// A warp's shared memory: candidates and slots, and for the tokens that they do
// not settle the row of q, with a list of experts and their 64-bit values.
struct Scratch {
    int *slot;            // [32]
    long long *key;       // [E]
    float *row;           // [E]
    uint16_t *id;         // [E]
};
__host__ __device__ inline int scratch_bytes(int E) { return 256 + ((14 * E + 15) & ~15); }
__device__ __forceinline__ Scratch scratch_of(unsigned char *p, int E) {
    return {reinterpret_cast<int *>(p), reinterpret_cast<long long *>(p + 256),
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

// The code from here to write_chosen runs for a token in a thousand, and for those of a
// padded batch, which are all ties: mostly it is read from memory for the one time that
// a multiprocessor runs it, so it is kept short, with loops as they stand.

// (a padded row's logits are alike, and most often 0)
__device__ __noinline__ double exp64(double x) { return x == 0.0 ? 1.0 : exp(x); }

// sum of exp(L - m) over a row
__device__ __noinline__ double softmax_sum64(const float *L, int E, float m) {
    double z = 0.0;
#pragma unroll 1
    for (int e = threadIdx.x & 31; e < E; e += 32) z += exp64((double)L[e] - (double)m);
#pragma unroll 1
    for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
    return z;
}
// the score of a logit (or the logit itself)
__device__ __noinline__ double score64(bool on_logits, bool sigmoid, float L, float m, double z) {
    if (on_logits) return (double)L;
    if (!sigmoid && m == -INFINITY) return 0.0;
    const double e = exp64(sigmoid ? -(double)L : (double)L - (double)m);
    return (sigmoid ? 1.0 : e) / (sigmoid ? 1.0 + e : z);
}

// The 64-bit values of the n experts in u.id, to u.key.  One logit for all of many
// (a padded row's): one score.
__device__ __noinline__ void values64(const SelectArgs &a, const float *L, float m, bool on_logits,
                                      int n, const Scratch &u) {
    const int lane = threadIdx.x & 31;
    const double z = a.sigmoid || on_logits || m == -INFINITY ? 1.0 : softmax_sum64(L, a.E, m);
    bool same = n > 32;
    double s = 0.0;
    if (same) {
        const float first = L[u.id[0]];
#pragma unroll 1
        for (int p = lane; p < n; p += 32)
            same = same && __float_as_uint(L[u.id[p]]) == __float_as_uint(first);
        same = __all_sync(kAll, same);
        if (same) s = score64(on_logits, a.sigmoid, first, m, z);
    }
#pragma unroll 1
    for (int p = lane; p < n; p += 32) {
        const int e = u.id[p];
        if (!same) s = score64(on_logits, a.sigmoid, L[e], m, z);
        u.key[p] = key_of(a.bias ? s + (double)a.bias[e] : s);
    }
    __syncwarp();
}

__device__ __forceinline__ int group_of(const SelectArgs &a, int e) { return e * a.per_group >> 20; }

// The experts for which in(e) holds, in ascending order, to u.id.
template <typename F> __device__ __forceinline__ int list_experts(int E, const Scratch &u, F in) {
    const int lane = threadIdx.x & 31;
    int n = 0;
#pragma unroll 1
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
        int p = 0, end = n;  // the first of the group's experts
#pragma unroll 1
        while (p < end) {
            const int mid = (p + end) >> 1;
            if (u.id[mid] < lane * a.size) p = mid + 1; else end = mid;
        }
#pragma unroll 1
        for (; p < n && u.id[p] < (lane + 1) * a.size; ++p) {
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
#pragma unroll 1
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

// What the errors of a group's score b1 + b2 go by; an excluded group's, -INF, has none.
__device__ __forceinline__ float size_of_score(float score, float b1, float b2) {
    return score > -INFINITY ? fabsf(b1) + fabsf(b2) : 0.f;
}

__device__ __forceinline__ float score32(float L, bool sigmoid, float m, float inv) {
    if (sigmoid) return rcp_fast(1.f + exp2_fast(L * -kLog2e));
    return m == -INFINITY ? 0.f : exp2_fast((L - m) * kLog2e) * inv;
}

// A token's weights and ids.  A lane with `chosen` has the expert `id`, its logit and
// its slot; m, z: softmax without renormalisation (m: a NaN where a logit of the row is one).
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
    if (isnan(m)) w = NAN;
    if (chosen) {
        a.idx[t * a.k + slot] = id;
        a.w[t * a.k + slot] = w;
    }
}

// A row's largest logit (a NaN where one is) and the sum of its exponentials.
__device__ __forceinline__ void softmax32(const float *L, int E, float *m, float *z) {
    const int lane = threadIdx.x & 31;
    float top = NAN, sum = 0.f;
    bool nan = false;
#pragma unroll 1
    for (int e = lane; e < E; e += 32) {
        top = fmaxf(top, L[e]);
        nan |= isnan(L[e]);
    }
    top = warp_max(top);
    *m = __any_sync(kAll, nan) ? NAN : top;
#pragma unroll 1
    for (int e = lane; e < E; e += 32) sum += exp2_fast((L[e] - *m) * kLog2e);
    *z = warp_sum(sum);
}

// Order-preserving whole-number image of a number, and back.
__device__ __forceinline__ int key32(float v) {
    const int b = __float_as_int(v + 0.f);
    return b >= 0 ? b : (int)(0x80000000u - (unsigned)b);
}
__device__ __forceinline__ float value32(int key) {
    return __int_as_float(key >= 0 ? key : (int)(0x80000000u - (unsigned)key));
}
__device__ __forceinline__ int largest(int v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ long long largest(long long v) {
    const int hi = __reduce_max_sync(kAll, (int)(v >> 32));
    const unsigned lo = __reduce_max_sync(kAll, (int)(v >> 32) == hi ? (unsigned)v : 0u);
    return (long long)(((unsigned long long)(unsigned)hi << 32) | lo);
}
// The `rounds` largest of more than 32 keys, one after the other, equal ones by id: the
// first k to u.slot.  Lane r returns the r-th; *last: the last one.  The keys taken are
// lost.  (Many candidates are ties, as in a padded row: ranking each against all
// others took 577 us for T = 8192, E = 256, half of them padded; now 38.)
template <typename K>
__device__ __noinline__ K pick(int k, int n, int rounds, K *key, const Scratch &u, K *last) {
    const int lane = threadIdx.x & 31;
    constexpr K kTaken = sizeof(K) == 4 ? (K)INT32_MIN : (K)INT64_MIN;
    K mine = kTaken, best = kTaken;
    int at = 0;
    auto scan = [&] {
        best = kTaken;
#pragma unroll 1
        for (int p = lane; p < n; p += 32) {
            const K v = key[p];
            if (v > best) {
                best = v;
                at = p;
            }
        }
    };
    scan();
#pragma unroll 1
    for (int r = 0; r < rounds; ++r) {
        const K top = largest(best);
        const int p = __reduce_min_sync(kAll, best == top ? at : INT32_MAX);
        if (lane == r) mine = top;
        *last = top;
        if ((p & 31) == lane) {
            if (r < k) u.slot[r] = u.id[p];
            key[p] = kTaken;
            scan();
        }
        __syncwarp();
    }
    return mine;
}

// Ranks of the n experts in u.id by u.key, equal ones by id: the first k to u.slot.
__device__ __forceinline__ void rank64(int k, int n, const Scratch &u) {
    const int p = threadIdx.x & 31;  // n <= 32
    if (p < n) {
        const long long v = u.key[p];
        const int id = u.id[p];
        int ahead = 0;
#pragma unroll 1
        for (int o = 0; o < n; ++o) {
            const long long w = u.key[o];
            if (w > v || (w == v && u.id[o] < id)) ++ahead;
        }
        if (ahead < k) u.slot[ahead] = id;
    }
    __syncwarp();
}
// ... and from there to the outputs.
__device__ __forceinline__ void write_chosen(const SelectArgs &a, int64_t t, const float *L, float m,
                                             float z, const Scratch &u) {
    const int lane = threadIdx.x & 31;
    const bool chosen = lane < a.k;
    const int id = chosen ? u.slot[lane] : 0;
    write_slots(a, t, chosen, lane, id, L[id], m, z);
    __syncwarp();
}

// A token that the fast path below leaves open: ties, values or groups that fp32
// cannot rank, NaN, or more candidates than a warp has lanes.  From the beginning, for any
// sizes: candidates are ranked in fp32 where that settles them, else in fp64.
__device__ __noinline__ void decide(const SelectArgs &a, int64_t t, unsigned char *smem) {
    const int lane = threadIdx.x & 31, E = a.E;
    const Scratch u = scratch_of(smem, E);
    const float *L = a.logits + t * E;
    const bool by_logits = !a.bias && (a.Gk == a.G || !a.top2);
    float m = -INFINITY, z = 1.f;
    if (!a.sigmoid) softmax32(L, E, &m, &z);
    const float unit = by_logits ? 0.f : unit_of(a.sigmoid, (E + 31) / 32, z);
    const float inv = rcp_fast(z);
#pragma unroll 1
    for (int e = lane; e < E; e += 32) {
        float q = L[e];
        if (!by_logits) {
            q = score32(q, a.sigmoid, m, inv);
            if (a.bias) q += a.bias[e];
        }
        u.row[e] = q;
    }
    __syncwarp();
    unsigned kept = 1u;
    if (a.Gk < a.G) {
        float b1 = NAN, b2 = NAN, score = NAN, floor32 = NAN, mag = 0.f;
        // a group's lanes share its experts, and lane g has its score
        auto second = [](float x, float y) { return isnan(x) || isnan(y) ? NAN : fminf(x, y); };
        const int g = lane >> a.shift, r = lane & ((1 << a.shift) - 1);
        if (g < a.G) {
#pragma unroll 1
            for (int i = r * a.per; i < min(a.size, (r + 1) * a.per); ++i) {
                const float x = u.row[g * a.size + i];
                b2 = fmaxf(b2, second(x, b1));
                b1 = fmaxf(b1, x);
            }
        }
#pragma unroll 1
        for (int o = 1; o < (1 << a.shift); o <<= 1) {
            const float o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
            b2 = fmaxf(fmaxf(b2, o2), second(b1, o1));
            b1 = fmaxf(b1, o1);
        }
        b1 = __shfl_sync(kAll, b1, lane << a.shift);
        b2 = __shfl_sync(kAll, b2, lane << a.shift);
        if (lane < a.G) {
            const bool sum = a.top2 && a.size > 1;
            score = sum ? b1 + b2 : b1;
            floor32 = isnan(score) ? NAN : sum ? b2 : b1;
            if (!by_logits) floor32 -= unit + 0x1p-22f * fabsf(floor32);
            mag = size_of_score(score, b1, sum ? b2 : 0.f);
        }
        float cur = score, bound = NAN;  // the Gk-th largest score
#pragma unroll 1
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
#pragma unroll 1
            for (int e = lane; e < E; e += 32) u.row[e] = L[e];
            __syncwarp();
        }
    }
    const bool exact = by_logits || !a.bias;
    auto stays = [&](int e) { return e < E && ((kept >> group_of(a, min(e, E - 1))) & 1u); };
    float best = NAN, bound = NAN;
#pragma unroll 1
    for (int e = lane; e < E; e += 32)
        if (stays(e)) best = fmaxf(best, u.row[e]);
#pragma unroll 1
    for (int j = 0; j < a.k; ++j) {
        bound = warp_max(best);
        if (best == bound) best = NAN;
    }
    if (isnan(bound)) bound = -INFINITY;  // fewer lanes than that: every value, and NaN
    const float floor32 = exact ? bound : bound - (unit + 0x1p-21f * fabsf(bound));
    const int n = list_experts(E, u, [&](int e) { return stays(e) && !(u.row[min(e, E - 1)] < floor32); });
    bool open = false;
    if (n <= 32) {
        const float q = lane < n ? u.row[u.id[lane]] : 0.f;
        int ahead = 0;
#pragma unroll 1
        for (int o = 0; o < n; ++o) {
            const float x = u.row[u.id[o]];
            if (x > q || (x == q && o < lane)) ++ahead;
            if (!exact && o != lane && x >= q) open |= too_near(x, q, unit);
        }
        open |= isnan(q);  // (for the 64-bit keys)
        open &= lane < n;
        if (lane < n && ahead < a.k) u.slot[ahead] = u.id[lane];
    } else {
        int *key = reinterpret_cast<int *>(u.key);
#pragma unroll 1
        for (int p = lane; p < n; p += 32) {
            const float q = u.row[u.id[p]];
            open |= isnan(q);
            key[p] = key32(q);
        }
        __syncwarp();
        if (!__any_sync(kAll, open)) {
            int last;
            const int rounds = min(n, a.k + 1);
            const int top = pick(a.k, n, rounds, key, u, &last);
            const int next = __shfl_down_sync(kAll, top, 1);
            if (!exact && lane + 1 < rounds)
                open = too_near(value32(top), value32(lane == 31 ? last : next), unit);
        }
    }
    open = __any_sync(kAll, open);
    __syncwarp();
    if (open) {
        values64(a, L, m, exact, n, u);
        long long last;
        if (n <= 32) rank64(a.k, n, u);
        else pick(a.k, n, a.k, u.key, u, &last);
    }
    write_chosen(a, t, L, m, z, u);
}

// A token whose candidates are known, and too near one another to rank: n <= 32 of
// them.  (They are kept until a warp has passed its tokens, or has no more room.)
constexpr int kPending = 8;
struct Pending {
    int64_t t[kPending];
    int n[kPending];
    uint16_t id[kPending][32];
};
__device__ __noinline__ void settle(const SelectArgs &a, const Pending &p, int i, unsigned char *smem) {
    const int lane = threadIdx.x & 31, n = p.n[i];
    const int64_t t = p.t[i];
    const Scratch u = scratch_of(smem, a.E);
    const float *L = a.logits + t * a.E;
    float m = -INFINITY, z = 1.f;
    if (!a.sigmoid) softmax32(L, a.E, &m, &z);
    if (lane < n) u.id[lane] = p.id[i][lane];
    __syncwarp();
    values64(a, L, m, !a.bias, n, u);
    rank64(a.k, n, u);
    write_chosen(a, t, L, m, z, u);
}

}  // namespace
}  // namespace moe
