// adamw.cu -- one AdamW step over many tensors, states in fp32 or in 8 bits.
//
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - step_size m / (sqrt(v) inv_sqrt_bc2 + eps)
//
// The tensors are cut into blocks of 256 elements, the unit of an 8-bit state's
// scale: a warp takes one, eight consecutive elements a lane, so that the block's
// largest magnitudes are two warp reductions and every access is a vector.  Chunks
// of 64 such blocks are dealt to the thread blocks; the tensors' addresses
// travel as kernel parameters, as in clip.cu.
//
// m and v are formed by rounded products and sums in a fixed order (no fused
// multiply-adds): a scale is a power of two that depends on the last bit of the
// largest magnitude, and so repeats wherever the same formula is evaluated.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = 256;                // elements under one scale
constexpr int kChunk = 64 * kBlock;        // elements a thread block takes at a time
constexpr int kGrid = 152 * 8;
constexpr int kTable = 300;                // tensors per launch
constexpr int kMapped = 1024;              // chunks with a map of their own

struct Entry {
    void *p;
    const void *g;
    void *m, *v;
    float *ms, *rs, *master;
    int64_t numel, block0;  // block0: number of its first block, counted over the list
    int end;                // chunks of the tensors up to and with this one
    float wd;
    uint8_t p_bf16, g_bf16, vec;
};
struct Table {
    int n, chunks, mapped;
    uint16_t tensor_of[kMapped];
    Entry t[kTable];
};

struct Step {
    float b1, c1, b2, c2, eps, max_norm;  // c1 = 1 - b1, c2 = 1 - b2
    int stochastic, skip_nonfinite;
    moe_adamw_scalars_t sc;
    const moe_adamw_scalars_t *dev;
    const float *norm;
};

// ------------------------------ random bits --------------------------------
// Words of a 32-bit product, xor'ed: the whole generator.  A block's two key words
// come from its number and the seed; an element's bits from those and its place.
// (Checked for uniform bits, and for correlation between neighbours, blocks and
// seeds: none beyond chance in 10^7 numbers.)
constexpr uint32_t kK0 = 0x9E3779B1u, kK1 = 0xD6E8FEB9u, kK2 = 0xA24BAED5u, kK3 = 0xCA5A8263u;
__device__ __forceinline__ uint32_t fold(uint32_t a, uint32_t k) {
    const uint64_t p = (uint64_t)a * k;
    return (uint32_t)(p >> 32) ^ (uint32_t)p;
}
struct Key {
    uint32_t x, y;
};
__device__ __forceinline__ Key block_key(int64_t block, uint32_t lo, uint32_t hi) {
    uint32_t x = fold((uint32_t)block + kK0, kK1);
    x = fold(x ^ lo, kK2);
    x = fold(x + hi + (uint32_t)((uint64_t)block >> 32), kK3);
    return {x, fold(x ^ kK0, kK3)};
}
__device__ __forceinline__ uint32_t random_bits(Key k, int place) {
    return fold(fold(k.x + kK0 * (uint32_t)place, kK2) ^ k.y, kK1);
}

// fp32 to bf16, up or down by 16 random bits (NaN stays NaN)
__device__ __forceinline__ uint32_t bf16_bits(float v, uint32_t u) {
    const uint32_t b = __float_as_uint(v);
    return isnan(v) ? 0x7fffu : (b + (u & 0xffffu)) >> 16;
}

// |y| <= 256 to a neighbouring e4m3 value, as a float: the low 20 mantissa bits
// go, up or down by 16 random bits.  Below 2^-6 the steps are 2^-9 throughout,
// those of the values from 2^-6 to 2^-5: with 2^-6 added, the same.
__device__ __forceinline__ float to_e4m3(float y, uint32_t random20) {
    const float low = fabsf(y) < 0x1p-6f ? copysignf(0x1p-6f, y) : 0.f;
    const uint32_t z = (__float_as_uint(y + low) + random20) & ~0xFFFFFu;
    return __uint_as_float(z) - low;
}

template <typename T> struct Eight;  // eight consecutive elements as floats
template <> struct Eight<float> {
    static __device__ __forceinline__ void load(const float *p, float (&v)[8]) {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        const float4 b = *reinterpret_cast<const float4 *>(p + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&v)[8]) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
};
template <> struct Eight<__nv_bfloat16> {
    static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&v)[8]) {
        unpack16(*reinterpret_cast<const uint4 *>(p), v, static_cast<const __nv_bfloat16 *>(nullptr));
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[8]) {
        stg16(p, pack16(v, static_cast<const __nv_bfloat16 *>(nullptr)));
    }
};
template <> struct Eight<__nv_fp8_e4m3> {
    static __device__ __forceinline__ float2 two(uint32_t c) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3);
        return __half22float2(__half2(h));
    }
    static __device__ __forceinline__ uint32_t code(float a, float b) {
        return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    }
    static __device__ __forceinline__ void load(const __nv_fp8_e4m3 *p, float (&v)[8]) {
        const uint2 c = *reinterpret_cast<const uint2 *>(p);
        float2 f = two(c.x);
        v[0] = f.x; v[1] = f.y;
        f = two(c.x >> 16);
        v[2] = f.x; v[3] = f.y;
        f = two(c.y);
        v[4] = f.x; v[5] = f.y;
        f = two(c.y >> 16);
        v[6] = f.x; v[7] = f.y;
    }
    static __device__ __forceinline__ void store(__nv_fp8_e4m3 *p, const float (&v)[8]) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(code(v[0], v[1]) | code(v[2], v[3]) << 16,
                                                   code(v[4], v[5]) | code(v[6], v[7]) << 16);
    }
};

// n of the lane's eight elements (all: a vector where the tensor allows it)
template <typename T>
__device__ __forceinline__ void load8(const T *p, int n, bool vec, float (&v)[8]) {
    if (vec && n == 8) {
        Eight<T>::load(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? (float)p[i] : 0.f;
}
template <typename T>
__device__ __forceinline__ void store8(T *p, int n, bool vec, const float (&v)[8]) {
    if (vec && n == 8) {
        Eight<T>::store(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = T(v[i]);
}

// 2^(e - 7) and its reciprocal for a block whose largest magnitude has these bits
__device__ __forceinline__ float scale_of(uint32_t largest, float *inverse) {
    const uint32_t e = max((largest >> 23) & 0xffu, 8u) - 7u;  // biased; at least 2^-126
    *inverse = __uint_as_float((254u - e) << 23);
    return __uint_as_float(e << 23);
}

// A block's states to 8 bits, in place.  x: 0 beyond the tensor's end; u: the elements'
// random bits.  ROOT: the roots, no positive one of which becomes zero.
template <bool ROOT>
__device__ __forceinline__ float quantise(float (&x)[8], uint32_t largest, const uint32_t (&u)[8]) {
    float inv;
    const float scale = scale_of(largest, &inv);
    if (largest >= 0x7f800000u) {  // uniform: a NaN or an infinity in the block
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= inv;
        return scale;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t r = ROOT ? ((u[i] >> 12) & 0xFFFF0u) | 8u : ((u[i] >> 4) & 0xFFFF0u) | 8u;
        const float y = to_e4m3(x[i] * inv, r);
        x[i] = ROOT && x[i] > 0.f ? fmaxf(y, 0x1p-9f) : y;
    }
    return scale;
}

// One block of 256 elements by a warp.
template <typename TP, typename TG, bool MASTER, bool SMALL>
__device__ __forceinline__ void step_block(const Entry &t, const Step &s, const moe_adamw_scalars_t &sc,
                                           float coef, int64_t block) {
    using TS = std::conditional_t<SMALL, __nv_fp8_e4m3, float>;
    const int lane = threadIdx.x & 31;
    const int64_t at = block * kBlock + 8 * lane;
    const int n = (int)max((int64_t)0, min((int64_t)8, t.numel - at));
    const bool vec = t.vec;
    float p[8], g[8], m[8], v[8];
    if constexpr (MASTER) load8(t.master + at, n, vec, p);
    else load8(static_cast<const TP *>(t.p) + at, n, vec, p);
    load8(static_cast<const TG *>(t.g) + at, n, vec, g);
    load8(static_cast<const TS *>(t.m) + at, n, vec, m);
    load8(static_cast<const TS *>(t.v) + at, n, vec, v);
    const float decay = fmaf(-sc.lr, t.wd, 1.f);
    if constexpr (SMALL) {
        const float ms = t.ms[block], rs = t.rs[block];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m[i] *= ms;
            const float r = v[i] * rs;
            v[i] = __fmul_rn(r, r);
        }
    }
    uint32_t top_m = 0u;
    float r[8], top_v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float gi = g[i] * coef;
        m[i] = __fadd_rn(__fmul_rn(m[i], s.b1), __fmul_rn(gi, s.c1));
        v[i] = __fadd_rn(__fmul_rn(v[i], s.b2), __fmul_rn(__fmul_rn(gi, gi), s.c2));
        r[i] = __fsqrt_rn(v[i]);
        p[i] = fmaf(-sc.step_size, __fdividef(m[i], fmaf(r[i], sc.inv_sqrt_bc2, s.eps)), p[i] * decay);
        if constexpr (SMALL) {
            top_m = max(top_m, __float_as_uint(m[i]) & 0x7fffffffu);
            top_v = v[i] > top_v || isnan(v[i]) ? v[i] : top_v;
        }
    }
    Key key = {0u, 0u};
    uint32_t u[8];
    const bool round = SMALL || (sizeof(TP) == 2 && !MASTER && s.stochastic);
    if (round) {
        key = block_key(t.block0 + block, sc.seed_lo, sc.seed_hi);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = random_bits(key, 8 * lane + i);
    }
    if constexpr (MASTER) store8(t.master + at, n, vec, p);
    if (sizeof(TP) == 2 && !MASTER && s.stochastic) {
        uint16_t *o = static_cast<uint16_t *>(t.p) + at;
        if (vec && n == 8) {
            uint32_t h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = bf16_bits(p[i], u[i]);
            stg16(o, make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16,
                                h[6] | h[7] << 16));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) o[i] = (uint16_t)bf16_bits(p[i], u[i]);
        }
    } else {
        store8(static_cast<TP *>(t.p) + at, n, vec, p);
    }
    if constexpr (SMALL) {
        top_m = __reduce_max_sync(kAll, top_m);
        // (the root's order is its square's)
        const uint32_t top_r = __reduce_max_sync(kAll, __float_as_uint(__fsqrt_rn(top_v)) & 0x7fffffffu);
        const float ms = quantise<false>(m, top_m, u);
        const float rs = quantise<true>(r, top_r, u);
        store8(static_cast<TS *>(t.m) + at, n, vec, m);
        store8(static_cast<TS *>(t.v) + at, n, vec, r);
        if (lane == 0) {
            t.ms[block] = ms;
            t.rs[block] = rs;
        }
    } else {
        store8(static_cast<float *>(t.m) + at, n, vec, m);
        store8(static_cast<float *>(t.v) + at, n, vec, v);
    }
}

template <bool SMALL>
__global__ void __launch_bounds__(kThreads)
adamw_kernel(const __grid_constant__ Table tab, const __grid_constant__ Step s) {
    pdl_wait();
    const moe_adamw_scalars_t sc = s.dev ? *s.dev : s.sc;
    float coef = 1.f;
    if (s.norm) {
        const float norm = *s.norm;
        if (s.skip_nonfinite && !isfinite(norm)) return;
        coef = s.max_norm / (norm + 1e-6f);
        coef = coef > 1.f ? 1.f : coef;  // a NaN norm stays NaN
    }
    const int wid = threadIdx.x >> 5;
    for (int c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
        int lo = 0, hi = tab.n - 1;
        if (tab.mapped) lo = hi = tab.tensor_of[c];
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (tab.t[mid].end > c) hi = mid; else lo = mid + 1;
        }
        const Entry &t = tab.t[lo];
        const int64_t blocks = (t.numel + kBlock - 1) / kBlock;
        const int64_t all = (t.numel + kChunk - 1) / kChunk;
        const int64_t first = (c - (t.end - all)) * (kChunk / kBlock);
        const int64_t last = min(blocks, first + kChunk / kBlock);
        const int kind = t.p_bf16 ? (t.master ? 2 : 1) : 0;
        for (int64_t b = first + wid; b < last; b += kWarps) {
            if (kind == 0) {
                if (t.g_bf16) step_block<float, __nv_bfloat16, false, SMALL>(t, s, sc, coef, b);
                else step_block<float, float, false, SMALL>(t, s, sc, coef, b);
            } else if (kind == 1) {
                if (t.g_bf16) step_block<__nv_bfloat16, __nv_bfloat16, false, SMALL>(t, s, sc, coef, b);
                else step_block<__nv_bfloat16, float, false, SMALL>(t, s, sc, coef, b);
            } else {
                if (t.g_bf16) step_block<__nv_bfloat16, __nv_bfloat16, true, SMALL>(t, s, sc, coef, b);
                else step_block<__nv_bfloat16, float, true, SMALL>(t, s, sc, coef, b);
            }
        }
    }
}

int64_t chunks_of(int64_t numel) { return (numel + kChunk - 1) / kChunk; }

bool vectors(const moe_adamw_tensor_t &t) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(t.param) | reinterpret_cast<uintptr_t>(t.grad) |
                          reinterpret_cast<uintptr_t>(t.exp_avg) |
                          reinterpret_cast<uintptr_t>(t.exp_avg_sq) |
                          reinterpret_cast<uintptr_t>(t.master);
    return (all & 15) == 0;
}

}  // namespace

int64_t adamw_chunk() { return kChunk; }

cudaError_t launch_adamw(const moe_adamw_tensor_t *ts, int64_t n, const moe_adamw_scalars_t &sc,
                         const moe_adamw_scalars_t *dev, const moe_adamw_hyper_t &h,
                         const float *norm, cudaStream_t st) {
    Step s = {};
    s.b1 = (float)h.beta1;
    s.c1 = (float)(1.0 - h.beta1);
    s.b2 = (float)h.beta2;
    s.c2 = (float)(1.0 - h.beta2);
    s.eps = (float)h.eps;
    s.max_norm = h.max_norm;
    s.stochastic = h.stochastic;
    s.skip_nonfinite = h.skip_nonfinite;
    s.sc = sc;
    s.dev = dev;
    s.norm = norm;
    Table tab;
    for (const bool small : {false, true}) {
        int64_t block0 = 0, i = 0;
        while (i < n) {
            tab.n = 0;
            int end = 0;
            for (; i < n && tab.n < kTable; ++i) {
                const moe_adamw_tensor_t &t = ts[i];
                const int64_t first = block0;
                block0 += (t.numel + kBlock - 1) / kBlock;
                if (t.numel == 0 || (t.state_dtype == MOE_E4M3) != small) continue;
                const int from = end;
                end += (int)chunks_of(t.numel);
                for (int c = from; c < end && c < kMapped; ++c) tab.tensor_of[c] = (uint16_t)tab.n;
                tab.t[tab.n++] = {t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.exp_avg_scale,
                                  t.exp_avg_sq_scale, t.master, t.numel, first, end, t.weight_decay,
                                  t.param_dtype == MOE_BF16, t.grad_dtype == MOE_BF16, vectors(t)};
            }
            if (tab.n == 0) continue;
            tab.chunks = end;
            tab.mapped = end <= kMapped;
            const cudaError_t e = launch_pdl(small ? adamw_kernel<true> : adamw_kernel<false>,
                                             dim3(std::min(kGrid, end)), dim3(kThreads), 0, st, tab, s);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaGetLastError();
}

}  // namespace moe
