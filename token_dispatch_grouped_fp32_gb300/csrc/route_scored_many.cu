// route_scored_many.cu -- the selection of route_scored.cu for long batches.
#include "route_scored.cuh"

namespace moe {
namespace {

// Long batches: eight lanes a token, four tokens a warp, N float4 of values a
// lane, k <= 8.  The same steps as a warp's per token, at a fraction of the
// instructions, since a step of a reduction, a vote or a rank serves all of a warp's
// tokens: the bound from the maxima of a half or a quarter of a lane's values each,
// candidates counted and placed by a prefix sum over the lanes, and four of them a
// lane.  T = 131072, k = 8, sigmoid with bias: E = 128 32 us, 60 with a warp a token
// (its bytes take 11); E = 256 47 and 76; E = 128 in four groups 46 and 79.  What is
// left is instructions (0.66 of the issue slots); code that a token seldom needs is
// kept out of the loop, which has to fit the instruction cache (49 us when it did
// not, 26 with the present loop, for E = 64).
constexpr int kLanes = 8, kManyK = 8, kManyFew = 32;
constexpr int kGroupParts = 4;  // (fewer of the lanes have values then)

struct Segment {  // a token's shared memory; 200 words apart: no bank conflicts
    Ranked few[kManyFew];     // candidates, NaN behind them
    Ranked sorted[kManyFew];  // by rank; NaN where equal values leave a gap
    uint32_t pad[72];
};
static_assert(sizeof(Segment) % 128 == 32, "");

template <bool MAX> __device__ __forceinline__ float segment_all(float v) {
#pragma unroll
    for (int o = kLanes / 2; o >= 1; o >>= 1) {
        const float u = __shfl_xor_sync(kAll, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    return v;
}

template <int N, bool EXACT, bool SIGMOID, bool GROUPS>
__global__ void __launch_bounds__(32, N <= 4 ? 24 : 20)
select_many_kernel(const SelectArgs a, const __grid_constant__ SelectArgs cold) {
    pdl_entry();
    if (a.zero_word != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.zero_word = 0u;
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int kTokens = 32 / kLanes, V = 4 * N, kParts = GROUPS ? kGroupParts : 2;
    const int lane = threadIdx.x, seg = lane / kLanes, l = lane % kLanes, E = a.E;
    Segment &s = reinterpret_cast<Segment *>(smem)[seg];
    // this lane's experts, four at a time: 4 (l + kLanes n) on, or with groups, whose
    // lanes follow one another, `per` consecutive ones
    const int mine0 = GROUPS ? l * a.per : 4 * l, mine_end = GROUPS ? mine0 + a.per : E;
    constexpr int kNext = GROUPS ? 4 : 4 * kLanes;

    const int64_t stride = (int64_t)gridDim.x * kTokens;
    Pending &pend = *reinterpret_cast<Pending *>(smem + a.pending_at);
    int64_t first = (int64_t)blockIdx.x * kTokens;
    while (first < a.T) {
        const int64_t t0 = first;
        unsigned left = 0u;  // bit kLanes * seg + i: token t0 + i * stride + seg is for decide()
        int pending = 0;     // and for settle()
        for (int i = 0; i < kLanes && first < a.T && pending <= kPending - kTokens; ++i, first += stride) {
            const int64_t t = first + seg;
            const bool there = t < a.T;
            const float *L = a.logits + t * E;
            float v[V];  // NaN: no expert
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int e = mine0 + kNext * n;
                float4 x = make_float4(NAN, NAN, NAN, NAN);
                if (there && e < mine_end) x = *reinterpret_cast<const float4 *>(L + e);
                v[4 * n] = x.x;
                v[4 * n + 1] = x.y;
                v[4 * n + 2] = x.z;
                v[4 * n + 3] = x.w;
            }
            __syncwarp();  // (the last token's shared memory as read)
#pragma unroll
            for (int c = 2 * l; c < kManyFew; c += 2 * kLanes) {
                const float4 none = make_float4(NAN, 0.f, NAN, 0.f);
                *reinterpret_cast<float4 *>(s.few + c) = none;
                *reinterpret_cast<float4 *>(s.sorted + c) = none;
            }

            float m = -INFINITY, z = 1.f;
            if (!SIGMOID && (!EXACT || !a.renorm)) {
                float top = v[0];
#pragma unroll
                for (int j = 1; j < V; ++j) top = fmaxf(top, v[j]);
                top = segment_all<true>(top);
                if (!isnan(top)) m = top;
                z = 0.f;
#pragma unroll
                for (int n = 0; n < N; ++n)
                    if (mine0 + kNext * n < mine_end)
#pragma unroll
                        for (int j = 0; j < 4; ++j) z += exp2_fast((v[4 * n + j] - m) * kLog2e);
                z = segment_all<false>(z);
            }
            // a NaN among softmax's logits makes every weight one: for decide() (as is a row of
            // -INF that is not renormalised, and sums that overflow both ways; without an exact
            // ranking such rows are for their NaN in `unit`)
            bool start_over = false;
            if (EXACT && !SIGMOID) {
                float2 sum = make_float2(z, 0.f);
                if (a.renorm)  // (no z)
#pragma unroll
                    for (int j = 0; j < V; j += 4)
                        if (mine0 + kNext * (j / 4) < mine_end)
                            sum = add2(add2(sum, make_float2(v[j], v[j + 1])), make_float2(v[j + 2], v[j + 3]));
                const unsigned odd = __ballot_sync(kAll, isnan(sum.x + sum.y) && there);
                start_over = (odd >> (kLanes * seg)) & ((1u << kLanes) - 1u);
            }
            if constexpr (!EXACT) {
                if (SIGMOID) {
#pragma unroll
                    for (int j = 0; j < V; ++j) v[j] = score32(v[j], true, 0.f, 0.f);
                } else {
                    const float inv = rcp_fast(z);
#pragma unroll
                    for (int j = 0; j < V; ++j) v[j] = exp2_fast((v[j] - m) * kLog2e) * inv;
                }
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int e = mine0 + kNext * n;
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (e < mine_end) x = __ldg(reinterpret_cast<const float4 *>(a.bias + e));
                    v[4 * n] += x.x;
                    v[4 * n + 1] += x.y;
                    v[4 * n + 2] += x.z;
                    v[4 * n + 3] += x.w;
                }
            }
            const float unit = EXACT ? 0.f : unit_of(SIGMOID, V, z);

            float bound = NAN;
            if constexpr (GROUPS) {
                const int in_group = 1 << a.shift;  // lanes
                float score, mag = 0.f;
                if (EXACT || !a.top2) {
                    score = v[0];
#pragma unroll
                    for (int j = 1; j < V; ++j) score = fmaxf(score, v[j]);
                    for (int o = 1; o < in_group; o <<= 1)
                        score = fmaxf(score, __shfl_xor_sync(kAll, score, o));
                    mag = size_of_score(score, score, 0.f);
                } else {
                    float h1 = -INFINITY, h2 = -INFINITY;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        h2 = fmaxf(h2, v[j] > h1 ? h1 : v[j]);
                        h1 = fmaxf(h1, v[j]);
                    }
                    for (int o = 1; o < in_group; o <<= 1) {
                        const float o1 = __shfl_xor_sync(kAll, h1, o), o2 = __shfl_xor_sync(kAll, h2, o);
                        h2 = fmaxf(fmaxf(h2, o2), fminf(h1, o1));
                        h1 = fmaxf(h1, o1);
                    }
                    score = h2 > -INFINITY ? h1 + h2 : -INFINITY;  // (as in select_kernel)
                    mag = size_of_score(score, h1, h2);
                }
                float cur = score;
                for (int j = 0; j < a.Gk; ++j) {
                    bound = segment_all<true>(cur);
                    if (cur == bound) cur = NAN;
                }
                const float off = EXACT ? 0.f
                                        : 2.f * unit + 0x1.2p-22f * segment_all<true>(mag);
                const unsigned reach = __ballot_sync(kAll, (l & (in_group - 1)) == 0 && !(score < bound - off));
                start_over |= __popc((reach >> (kLanes * seg)) & ((1u << kLanes) - 1u)) != a.Gk;
                if (!(score >= bound))
#pragma unroll
                    for (int j = 0; j < V; ++j) v[j] = NAN;
                bound = NAN;
            }
            // the maxima of a part of the lane's values each
            float part[kParts];
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                part[p] = v[V / kParts * p];
#pragma unroll
                for (int j = 1; j < V / kParts; ++j) part[p] = fmaxf(part[p], v[V / kParts * p + j]);
            }
#pragma unroll
            for (int j = 0; j < kManyK; ++j) {
                if (j >= a.k) break;
                float top = fmaxf(part[0], part[1]);
#pragma unroll
                for (int p = 2; p < kParts; ++p) top = fmaxf(top, part[p]);
                bound = segment_all<true>(top);
#pragma unroll
                for (int p = 0; p < kParts; ++p)
                    if (part[p] == bound) part[p] = NAN;
            }
            if (isnan(bound)) bound = -INFINITY;
            const float floor32 = EXACT ? bound : bound - (unit + 0x1p-21f * fabsf(bound));
            int mine = 0;
#pragma unroll
            for (int j = 0; j < V; ++j) mine += v[j] >= floor32;
            int upto = mine;  // with the lanes below
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) {
                const int u = __shfl_up_sync(kAll, upto, o, kLanes);
                if (l >= o) upto += u;
            }
            const int n = __shfl_sync(kAll, upto, kLanes - 1, kLanes);
            int at = upto - mine;
            __syncwarp();
            if (n <= kManyFew) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (v[j] >= floor32) s.few[at++] = {v[j], mine0 + kNext * (j / 4) + j % 4};
            }
            __syncwarp();
            // ranks, by the values behind each: by the sign of a difference, two a packed sum
            constexpr int kHold = kManyFew / kLanes;  // candidates a lane
            Ranked c[kHold];
            int behind[kHold];
#pragma unroll
            for (int j = 0; j < kHold; ++j) {
                c[j] = s.few[l + kLanes * j];
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
            if (__any_sync(kAll, n > 16)) {  // (uniform; in few instructions)
#pragma unroll 1
                for (int p = 0; p < kManyFew; p += 2) {
                    if (p >= 16) {
                        rank(p, 0);
                        rank(p, 1);
                    }
#pragma unroll
                    for (int j = 2; j < kHold; ++j) rank(p, j);
                }
            }
#pragma unroll
            for (int j = 0; j < kHold; ++j)
                if (l + kLanes * j < n && n <= kManyFew) s.sorted[n - 1 - behind[j]] = c[j];
            __syncwarp();
            const bool slot = l < a.k;
            const Ranked chosen = s.sorted[l];
            const float q = chosen.q, next = s.sorted[l + 1].q;
            const bool bad = there && slot &&
                             (start_over || n > kManyFew || isnan(q) ||
                              (l + 1 < n && (EXACT ? !(q > next) : too_near(q, next, unit))));
            unsigned open = __ballot_sync(kAll, bad);
#pragma unroll
            for (int o = kLanes / 2; o >= 1; o >>= 1) open |= open >> o;  // each segment's any, in its bit 0
            open &= 0x01010101u;
            if (open) {  // (uniform)
                const unsigned many =
                    __ballot_sync(kAll, l == 0 && (start_over || n < a.k || n > kManyFew));
                left |= (open & many) << i;
                const unsigned listed = open & ~many;
                const int at_pend = pending + __popc(listed & ((1u << kLanes * seg) - 1u));
                if ((listed >> (kLanes * seg)) & 1u) {
#pragma unroll
                    for (int c = l; c < kManyFew; c += kLanes) pend.id[at_pend][c] = (uint16_t)s.few[c].id;
                    if (l == 0) {
                        pend.t[at_pend] = t;
                        pend.n[at_pend] = n;
                    }
                }
                pending += __popc(listed);
            }

            const bool write = there && slot && ((open >> (kLanes * seg)) & 1u) == 0u;
            const int id = write ? chosen.id : 0;
            const float logit = !write ? -INFINITY : EXACT ? q : L[id];
            float w;
            if (SIGMOID || a.renorm) {
                float x = SIGMOID ? rcp_fast(1.f + expf(-logit)) : 0.f;
                float sum = 1.f;
                if (SIGMOID && a.renorm) sum = segment_all<false>(slot ? x : 0.f);
                if (a.renorm && __any_sync(kAll, !SIGMOID || (write && sum < 0x1p-100f))) {
                    // (as in write_slots; for all of the warp's tokens, if one needs it)
                    const float top = segment_all<true>(logit);
                    const bool here = !SIGMOID || sum < 0x1p-100f;
                    const float y = !write || top == -INFINITY ? 0.f : expf(logit - top);
                    const float shares = segment_all<false>(y);
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
        __syncwarp();
        for (int i = 0; i < pending; ++i) settle(cold, pend, i, smem);
        while (left) {
            const int bit = __ffs(left) - 1;
            left &= left - 1u;
            decide(cold, t0 + bit % kLanes * stride + bit / kLanes, smem);
        }
    }
}

template <int N, bool GROUPS>
cudaError_t launch_many(const SelectArgs &a, bool exact, cudaStream_t st) {
    constexpr int kTokens = 32 / kLanes;
    SelectArgs b = a;
    if (GROUPS) {  // the lanes of a group, in a segment
        b.shift = 0;
        while ((a.G << (b.shift + 1)) <= kLanes) ++b.shift;
        b.per = a.size >> b.shift;
    }
    b.pending_at = std::max(scratch_bytes(a.E), (int)sizeof(Segment) * kTokens);
    const size_t smem = b.pending_at + sizeof(Pending);
    const dim3 grid((unsigned)std::min<int64_t>((a.T + kTokens - 1) / kTokens,
                                                (int64_t)device_sm_count() * (N <= 4 ? 24 : 20)));
    auto kernel = a.sigmoid ? (exact ? select_many_kernel<N, true, true, GROUPS>
                                     : select_many_kernel<N, false, true, GROUPS>)
                            : (exact ? select_many_kernel<N, true, false, GROUPS>
                                     : select_many_kernel<N, false, false, GROUPS>);
    return launch_pdl(kernel, grid, dim3(32), smem, st, b, a);
}
// From this many tokens on, where there are several for each lane's place (T = 4096,
// E = 128: 3.7 us and 4.6 with a warp a token; 2048: 2.8 and 2.7; E = 256 3.8 and 4.6,
// 3.1 and 2.7).  Groups of 256 experts, whose lanes are fewer, from eight times as
// many (eight groups by their maxima: T = 16384 11.1 and 11.0, 32768 17.0 and 19.1;
// by the sum of two: 18.6 and 16.4, 26.8 and 27.0, 131072 91 and 100).
constexpr int64_t kManyTokens = 4096;

}  // namespace

bool select_takes_many(const SelectArgs &a, bool exact) {
    if (a.nparts > 0 || a.k > kManyK || a.E % 4 != 0 || a.E < 32 || a.E > 256 || a.T < kManyTokens)
        return false;
    if (a.Gk == a.G) return true;
    // groups: a power of two, whole lanes of a multiple of four experts, and a rank
    // that is that of the values in hand
    const int lanes = a.G <= 8 ? 8 / a.G : 0;
    return lanes > 0 && (a.G & (a.G - 1)) == 0 && a.size % (4 * lanes) == 0 && (exact || a.bias) && a.size > 1 &&
           a.Gk * lanes * kGroupParts >= 2 * a.k && (a.E <= 128 || a.T >= 8 * kManyTokens);
}

cudaError_t launch_select_many(const SelectArgs &a, bool exact, cudaStream_t st) {
    if (a.Gk < a.G)
        return a.E <= 128 ? launch_many<4, true>(a, exact, st) : launch_many<8, true>(a, exact, st);
    if (a.E <= 64) return launch_many<2, false>(a, exact, st);
    if (a.E <= 128) return launch_many<4, false>(a, exact, st);
    return launch_many<8, false>(a, exact, st);
}

}  // namespace moe
