// route_scored.cu -- the router with scores of its own: softmax or sigmoid of
// the logits, a balance bias that acts on the choice and not on the weights,
// groups of experts, top-k, renormalised and scaled weights.
//
//   s_e = exp(L_e) / sum_i exp(L_i)   or   1 / (1 + exp(-L_e))
//   q_e = s_e + b_e           the choice is made on q (without b: on L, the same order)
//   u_g = max of q in group g, or the sum of its two largest; the best Gk stay
//   w_j = c s_j / (sum of s over the chosen k, or 1)
//
// The choice is that of 64-bit values of q: fp32 values are ranked first, and a
// token whose ranking they cannot settle (two of its values closer than their
// errors, about one token in 1,000 at E = 256) is decided again in fp64.
#include "route_scored.cuh"

namespace moe {
namespace {

// A warp per token, several tokens one after the other where there are many.
// VPL: values a lane has room for (>= a.per).  EXACT: the ranking is that of the
// logits themselves (no bias, and no group sums).
//
// The k-th largest of the lanes' maxima is a bound that k values reach, and few
// more (with k = 8 and 8 values a lane about 10, with k = 16 about 21): these
// candidates are gathered in shared memory, one a lane, and each counts those ahead
// of it, instead of k rounds of a warp maximum with its removal.  What this leaves
// open goes to decide(), after every 32 tokens: a call inside their loop cost it
// spills (then 62 us for T = 131072, E = 128 instead of 43).  Blocks of one warp: what depends on the
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

    Pending &pend = *reinterpret_cast<Pending *>(smem + a.pending_at);
    int64_t t = blockIdx.x;
    while (t < a.T) {
        const int64_t t0 = t;
        unsigned left = 0u;  // of the tokens t0 + i * gridDim.x, those for decide()
        int pending = 0;     // and for settle()
        for (int i32 = 0; i32 < 32 && t < a.T && pending < kPending; ++i32, t += gridDim.x) {
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
            // a NaN among softmax's logits makes every weight one: for decide(), as is a row
            // of -INF (without an exact ranking both are, for their NaN in `unit`)
            bool odd = false;
            if (EXACT && !a.sigmoid) {
                float sum = z;
                if (a.renorm) {  // (no z; logits that overflow both ways go there too)
                    sum = 0.f;
#pragma unroll
                    for (int i = 0; i < VPL; ++i)
                        if (i < count) sum += v[i];
                }
                odd = __any_sync(kAll, isnan(sum));
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
                    if (!EXACT) mag = size_of_score(score, score, 0.f);
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
                    // (no second number, or an excluded expert: below every sum of two; decide()
                    // knows more, where such groups are to be kept)
                    score = group >= a.G ? NAN : b2 > -INFINITY ? b1 + b2 : -INFINITY;
                    mag = size_of_score(score, b1, b2);
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
            const bool listed = decided && !odd && n >= a.k && n <= 32;
            decided = listed;
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
            if (!decided && listed) {
                pend.id[pending][lane] = (uint16_t)mine.id;
                if (lane == 0) {
                    pend.t[pending] = t;
                    pend.n[pending] = n;
                }
                ++pending;
            } else if (!decided) {
                left |= 1u << i32;
            }
        }
        __syncwarp();
        for (int i = 0; i < pending; ++i) settle(cold, pend, i, smem);
        while (left) {
            const int i = __ffs(left) - 1;
            left &= left - 1u;
            decide(cold, t0 + i * (int64_t)gridDim.x, smem);
        }
    }
}

template <int VPL, bool EXACT, bool GROUPS>
cudaError_t launch_select_t(const SelectArgs &a, cudaStream_t st) {
    SelectArgs b = a;
    b.pending_at = std::max(scratch_bytes(a.E), (int)sizeof(Ranked) * 32 * VPL);
    const size_t smem = b.pending_at + sizeof(Pending);
    // as many blocks as stay resident, then more tokens a block
    const dim3 grid((unsigned)std::min<int64_t>(a.T, (int64_t)device_sm_count() * 32));
    return launch_pdl(select_kernel<VPL, EXACT, GROUPS>, grid, dim3(32), smem, st, b, b);
}
template <int VPL> cudaError_t launch_select_v(const SelectArgs &a, bool exact, cudaStream_t st) {
    if (a.Gk < a.G)
        return exact ? launch_select_t<VPL, true, true>(a, st) : launch_select_t<VPL, false, true>(a, st);
    return exact ? launch_select_t<VPL, true, false>(a, st) : launch_select_t<VPL, false, false>(a, st);
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
    if (select_takes_many(a, exact)) e = launch_select_many(a, exact, st);
    else if (a.per <= 4) e = launch_select_v<4>(a, exact, st);
    else if (a.per <= 8) e = launch_select_v<8>(a, exact, st);
    else if (a.per <= 16) e = launch_select_v<16>(a, exact, st);
    else if (a.per <= 32) e = launch_select_v<32>(a, exact, st);
    else if (exact) e = launch_select_t<64, true, true>(a, st);  // few lanes a group: 9 to 31 groups
    else e = launch_select_t<64, false, true>(a, st);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
