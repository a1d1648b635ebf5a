// adamw.cu -- one AdamW step over many tensors, states in fp32 or in 8 bits.
//
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - step_size m / (sqrt(v) inv_sqrt_bc2 + eps)
//
// The tensors are cut into blocks of 256 elements, the unit of an 8-bit state's
// scale: a warp takes one, eight consecutive elements a lane, so that the block's
// largest magnitudes are two warp reductions and every access is a vector.  A
// thread block takes a chunk of 8 to 256 such blocks; the tensors' addresses
// travel as kernel parameters, as in clip.cu.
//
// fp32 states are bound by HBM (64 M bf16 parameters: 210 us, 0.99 of the copy
// rate).  8-bit states by the instructions of two roundings an element: 129 us
// (0.74; fp32 parameters, which move more, 160: 0.95; 1.4 G bf16 ones 0.82).  A ring of asynchronous copies
// into shared memory took 148 to 155 us, values of the next block held in registers
// 161 to 205, and a prefetch into L2 158: the loads are not what it waits for.
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
// Blocks a chunk, one to 32 a warp.  Every chunk has to be found and its scales
// read, and in the last round of chunks some multiprocessors have none: the first costs
// blocks / chunk, the second a chunk, and their sum is least where the chunk
// goes by the root of the blocks (8-bit states: 64 M parameters 131 us with chunks
// of 64, 132 of 128, 141 of 256; 1.4 G 2741 of 64, 2607 of 256; 3 M in ragged tensors 10.9
// of 8, 9.5 of 16).  kSquare: from 0.5 M to 512 M elements, in one tensor and in 40 ragged
// ones, its chunk takes at most 2 % more time than the best of a quarter, half, double and
// four times that.  A thread block for each: 64 M took
// 137 us with a grid of eight an SM, which cannot even out what they take.
constexpr int kMostBlocks = 32 * kWarps;
constexpr int kSquare = 76;
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
struct Step {
    float b1, c1, b2, c2, eps, max_norm;  // c1 = 1 - b1, c2 = 1 - b2
    float minus_zero;
    int stochastic, skip_nonfinite;
    moe_adamw_scalars_t sc;
    const moe_adamw_scalars_t *dev;
    const float *norm;
};

// Tensors per launch: what a kernel's parameters hold beside the rest.
constexpr int kParameterBytes = 32764;
constexpr int kTable = (kParameterBytes - (int)sizeof(Step) - 16 - 2 * kMapped) / (int)sizeof(Entry);
struct Table {
    int n, chunks, mapped, chunk_blocks;
    uint16_t tensor_of[kMapped];
    Entry t[kTable];
};
static_assert(sizeof(Table) + sizeof(Step) <= kParameterBytes, "");

// ------------------------------ random bits --------------------------------
// Words of a 32-bit product, xor'ed: the whole generator.  A block's two key words
// come from its number and the seed; an element's bits from those and its place.
// (Checked for uniform bits, and for correlation between neighbours, blocks and
// seeds: none beyond chance in 10^7 numbers.)  kK0 is the prime next to 2^32 over the
// golden ratio; the others are the leading 32 bits of 64-bit multipliers that published
// mixing functions use, made odd.
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
// (with the highest bit of m's flipped, which costs nothing here)
constexpr uint32_t kFlip = 0x00800000u;
__device__ __forceinline__ uint32_t random_bits(Key k, int place) {
    return fold(fold(k.x + kK0 * (uint32_t)place, kK2) ^ k.y, kK1) ^ kFlip;
}

// Two fp32 values to bf16, up or down by 16 random bits each (the low ones of u and
// w): the bits plus those, without their last 16; a NaN stays one.
__device__ __forceinline__ uint32_t bf16_pair(float2 v, uint32_t u, uint32_t w) {
    uint32_t d;
    asm("cvt.rs.bf16x2.f32 %0, %1, %2, %3;"
        : "=r"(d) : "f"(v.y), "f"(v.x), "r"(__byte_perm(u, w, 0x5410)));
    return d;
}

// The largest magnitude of three; a NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The smallest magnitude of three.
__device__ __forceinline__ float min_abs(float a, float b, float c) {
    float d;
    asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }

// Root and reciprocal to 1 ulp.  FLUSH: squares below 2^-126 count as 0.
template <bool FLUSH> __device__ __forceinline__ float root(float v) {
    float r;
    if constexpr (FLUSH) asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    else asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Eight consecutive elements as they lie in memory, and as floats.
template <typename T> struct Eight {
    uint4 c;
    __device__ __forceinline__ void load(const T *p) { c = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(T *p) const { stg16(p, c); }
};
template <> struct Eight<float> {
    uint4 c, d;
    __device__ __forceinline__ void load(const float *p) {
        c = *reinterpret_cast<const uint4 *>(p);
        d = *reinterpret_cast<const uint4 *>(p + 4);
    }
    __device__ __forceinline__ void store(float *p) const {
        stg16(p, c);
        stg16(p + 4, d);
    }
};
template <> struct Eight<__nv_fp8_e4m3> {
    uint2 c;
    __device__ __forceinline__ void load(const __nv_fp8_e4m3 *p) { c = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void store(__nv_fp8_e4m3 *p) const { *reinterpret_cast<uint2 *>(p) = c; }
};
__device__ __forceinline__ float2 pair_of(uint32_t a, uint32_t b) {
    return make_float2(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ void unpack(const Eight<float> &e, float2 (&v)[4]) {
    v[0] = pair_of(e.c.x, e.c.y);
    v[1] = pair_of(e.c.z, e.c.w);
    v[2] = pair_of(e.d.x, e.d.y);
    v[3] = pair_of(e.d.z, e.d.w);
}
__device__ __forceinline__ void unpack(const Eight<__nv_bfloat16> &e, float2 (&v)[4]) {
    const uint32_t w[4] = {e.c.x, e.c.y, e.c.z, e.c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair_of(w[i] << 16, w[i] & 0xffff0000u);
}
__device__ __forceinline__ float2 e4m3_pair(uint32_t c) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3);
    return __half22float2(__half2(h));
}
__device__ __forceinline__ void unpack(const Eight<__nv_fp8_e4m3> &e, float2 (&v)[4]) {
    v[0] = e4m3_pair(e.c.x);
    v[1] = e4m3_pair(e.c.x >> 16);
    v[2] = e4m3_pair(e.c.y);
    v[3] = e4m3_pair(e.c.y >> 16);
}
__device__ __forceinline__ void pack(const float2 (&v)[4], Eight<float> *e) {
    e->c = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                      __float_as_uint(v[1].y));
    e->d = make_uint4(__float_as_uint(v[2].x), __float_as_uint(v[2].y), __float_as_uint(v[3].x),
                      __float_as_uint(v[3].y));
}
__device__ __forceinline__ void pack(const float2 (&v)[4], Eight<__nv_bfloat16> *e) {
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&e->c);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[i].x, v[i].y);
}
__device__ __forceinline__ uint32_t e4m3_code(float2 a, float2 b) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16;
}
__device__ __forceinline__ void pack(const float2 (&v)[4], Eight<__nv_fp8_e4m3> *e) {
    e->c = make_uint2(e4m3_code(v[0], v[1]), e4m3_code(v[2], v[3]));
}

// ... n of them, an element at a time (0 for the others: the zero of every type)
template <typename T> struct Bits;
template <> struct Bits<float> { using U = uint32_t; };
template <> struct Bits<__nv_bfloat16> { using U = uint16_t; };
template <> struct Bits<__nv_fp8_e4m3> { using U = uint8_t; };
template <typename T> __device__ __forceinline__ uint32_t some_word(const T *p, int n, int w) {
    using U = typename Bits<T>::U;
    constexpr int kIn = 4 / sizeof(T);
    const U *q = reinterpret_cast<const U *>(p);
    uint32_t x = 0u;
#pragma unroll
    for (int j = 0; j < kIn; ++j)
        if (w * kIn + j < n) x |= (uint32_t)q[w * kIn + j] << (8 * sizeof(T) * j);
    return x;
}
template <typename T> __device__ __forceinline__ void put_word(T *p, int n, int w, uint32_t x) {
    using U = typename Bits<T>::U;
    constexpr int kIn = 4 / sizeof(T);
    U *q = reinterpret_cast<U *>(p);
#pragma unroll
    for (int j = 0; j < kIn; ++j)
        if (w * kIn + j < n) q[w * kIn + j] = (U)(x >> (8 * sizeof(T) * j));
}
template <typename T> __device__ __forceinline__ void load_some(const T *p, int n, Eight<T> *e) {
    e->c.x = some_word(p, n, 0);
    e->c.y = some_word(p, n, 1);
    if constexpr (sizeof(T) > 1) {
        e->c.z = some_word(p, n, 2);
        e->c.w = some_word(p, n, 3);
    }
    if constexpr (sizeof(T) == 4)
        e->d = make_uint4(some_word(p, n, 4), some_word(p, n, 5), some_word(p, n, 6), some_word(p, n, 7));
}
template <typename T> __device__ __forceinline__ void store_some(T *p, int n, const Eight<T> &e) {
    put_word(p, n, 0, e.c.x);
    put_word(p, n, 1, e.c.y);
    if constexpr (sizeof(T) > 1) {
        put_word(p, n, 2, e.c.z);
        put_word(p, n, 3, e.c.w);
    }
    if constexpr (sizeof(T) == 4) {
        put_word(p, n, 4, e.d.x);
        put_word(p, n, 5, e.d.y);
        put_word(p, n, 6, e.d.z);
        put_word(p, n, 7, e.d.w);
    }
}

// The biased exponent of 2^(e - 7), at least that of 2^-126, for a block whose largest
// magnitude has these bits; and for the roots of one whose largest value has.
__device__ __forceinline__ uint32_t scale_exponent(uint32_t largest) {
    return max(largest >> 23, 8u) - 7u;
}
__device__ __forceinline__ uint32_t root_scale_exponent(uint32_t largest) {
    // half of v's exponent, rounded down; just below an even power the root, rounded
    // to the nearest, is the next one.  (Below 2^-126 the roots are 0.)
    const int e = (int)((largest + 1u) >> 23) - 127;
    return largest < 0x00800000u ? 1u : (uint32_t)((e >> 1) + 127 - 7);
}

// 16 random bits (of a root: the high ones; else bits 8 to 23) as the bits of
// 2^23 + their number.
template <bool ROOT> __device__ __forceinline__ uint32_t number(uint32_t u) {
    return __byte_perm(u ^ kFlip, 0x4B000000u, ROOT ? 0x7432 : 0x7421);
}
// ... and as a signed fraction of 2^32, centred: 2^16 (number - 2^15 + 1/2).
template <bool ROOT> __device__ __forceinline__ int centred(uint32_t u) {
    return ROOT ? (int)((u & 0xffff0000u) ^ (0x80008000u ^ kFlip)) : (int)__byte_perm(u, 0x8000u, 0x2154);
}

// (a block with magnitudes below the normal ones; apart, for its registers)
struct Values {
    float2 x[4];
    uint32_t u[8];
};
template <bool ROOT> __device__ __noinline__ Values small_ones(Values a) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = a.x[i];
        // to a neighbouring e4m3 value (|y| <= 256).  power: 2^e <= |y|, at least 2^-6, below
        // which the steps are those from there up: a step is power / 8.  A random part
        // of a step in (-1/2, 1/2), of 16 bits, is added to the magnitude, and the sum
        // rounded to steps by adding and taking away 1.5 * 2^23 of them.  (Four packed
        // operations; by integer sums on the bits it took seven or eight of the ALU,
        // which is what bounds this kernel.)
        const float2 power = make_float2(
            fmaxf(__uint_as_float(__float_as_uint(y.x) & 0x7f800000u), 0x1p-6f),
            fmaxf(__uint_as_float(__float_as_uint(y.y) & 0x7f800000u), 0x1p-6f));
        const float2 f = pair_of(number<ROOT>(a.u[2 * i]), number<ROOT>(a.u[2 * i + 1]));
        // (number + 1/2) 2^-19 - 1/16, to 2^-27: 2^23 and 1/2 do not fit one float, but
        // 2^23 2^-19 (1 - 2^-24) lacks 2^-20
        float2 part = fma2(f, two(0x1p-19f * (1.f - 0x1p-24f)), two(-16.0625f + 0x1p-19f));
        if (!ROOT) {  // away from zero by the same numbers on either side
            part.x = __uint_as_float(__float_as_uint(part.x) ^ (__float_as_uint(y.x) & 0x80000000u));
            part.y = __uint_as_float(__float_as_uint(part.y) ^ (__float_as_uint(y.y) & 0x80000000u));
        }
        const float2 sum = fma2(power, two(1.5f * 0x1p20f), fma2(part, power, y));
        float2 q = fma2(power, two(-1.5f * 0x1p20f), sum);
        if (ROOT) {  // (2^-9 if y is not 0)
            const float2 least = make_float2(__saturatef(y.x * 0x1p126f), __saturatef(y.y * 0x1p126f));
            const float2 l = mul2(least, two(0x1p-9f));
            q = make_float2(fmaxf(q.x, l.x), fmaxf(q.y, l.y));
        }
        a.x[i] = q;
    }
    return a;
}

// A block's states to 8 bits, in place, by a scale of biased exponent e.  x: 0 beyond
// the tensor's end; u: the elements' random bits.
// ROOT: the roots, no positive one of which becomes zero.
template <bool ROOT>
__device__ __forceinline__ float quantise(float2 (&x)[4], uint32_t e, const uint32_t (&u)[8]) {
    const float inv = __uint_as_float((254u - e) << 23), scale = __uint_as_float(e << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], two(inv));
    float low = min_abs(x[0].x, x[0].y, x[1].x);
    low = min_abs(low, x[1].y, x[2].x);
    low = min_abs(low, x[2].y, x[3].x);
    low = min_abs(low, low, x[3].y);
    if (__all_sync(kAll, low >= 0x1p-6f)) {
        // Normal numbers of e4m3, nineteen blocks of twenty: their last 20 bits are a part
        // of a step, and a random one in (-1/2, 1/2) is added to them; the conversion
        // rounds to the nearest.  (64 M bf16 parameters 137 us, by the way below alone 144.)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = pair_of(__float_as_uint(x[i].x) + (uint32_t)(centred<ROOT>(u[2 * i]) >> 12),
                           __float_as_uint(x[i].y) + (uint32_t)(centred<ROOT>(u[2 * i + 1]) >> 12));
        return scale;
    }
    const Values a = small_ones<ROOT>({{x[0], x[1], x[2], x[3]}, {u[0], u[1], u[2], u[3], u[4], u[5], u[6], u[7]}});
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a.x[i];
    return scale;
}

// Eight states of a block with NaN or infinite ones to 8 bits: the scale is that of its
// largest finite magnitude, and the others are rounded as they are without those.  A
// NaN is stored as one, an infinite m as the largest value, an infinite root as kInfiniteRoot.
constexpr uint8_t kInfiniteRoot = 0xff;  // a negative NaN
template <bool ROOT>
__device__ __forceinline__ float set_apart(const float (&x)[8], const uint32_t (&u)[8],
                                           Eight<__nv_fp8_e4m3> *to) {
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = isfinite(x[j]) ? fmaxf(top, fabsf(x[j])) : top;
    const uint32_t e = scale_exponent(__reduce_max_sync(kAll, __float_as_uint(top)));
    const float inv = __uint_as_float((254u - e) << 23);
    float y[8];
    Values a;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        y[j] = isfinite(x[j]) ? x[j] * inv : 0.f;
        a.u[j] = u[j];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) a.x[i] = make_float2(y[2 * i], y[2 * i + 1]);
    a = small_ones<ROOT>(a);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float &q = j & 1 ? a.x[j / 2].y : a.x[j / 2].x;
        if (!isfinite(x[j])) q = ROOT ? NAN : x[j];
    }
    pack(a.x, to);
    if (ROOT)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (isinf(x[j])) (j < 4 ? to->c.x : to->c.y) |= 0x80u << (8 * (j % 4));
    return __uint_as_float(e << 23);
}

// What a lane reads of a block of 256 elements.
template <typename TP, typename TG, bool SMALL> struct Block {
    using TS = std::conditional_t<SMALL, __nv_fp8_e4m3, float>;
    Eight<TP> p;
    Eight<TG> g;
    Eight<TS> m, v;
};

// A block of 8-bit states with one that is not finite: the same operations, apart from the
// others for their registers (the branch there costs them 1 to 3 %; with the bad elements
// handled where the others are, 6 to 8 % for more spills).  Returns the new scales.
template <typename TP, typename TG, bool MASTER>
__device__ __noinline__ float2 seldom_block(const Entry &t, const Step &s, float coef, int64_t b,
                                            float ms, float rs, Key key) {
    const moe_adamw_scalars_t sc = s.dev ? *s.dev : s.sc;
    const int lane = threadIdx.x & 31;
    const int64_t at = b * kBlock + 8 * lane;
    const int n = (int)max((int64_t)0, min((int64_t)8, t.numel - at));
    float m[8], r[8];
    uint32_t u[8];
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {
        m[j] = r[j] = 0.f;
        u[j] = random_bits(key, 8 * lane + j);
        if (j >= n) continue;
        const __nv_fp8_e4m3 *mp = static_cast<const __nv_fp8_e4m3 *>(t.m) + at + j;
        const __nv_fp8_e4m3 *rp = static_cast<const __nv_fp8_e4m3 *>(t.v) + at + j;
        const float root0 = __fmul_rn((float)*rp, rs);
        const float v0 = rp->__x == kInfiniteRoot ? INFINITY : __fmul_rn(root0, root0);
        const float g = __fmul_rn((float)static_cast<const TG *>(t.g)[at + j], coef);
        m[j] = __fadd_rn(__fmul_rn(__fmul_rn((float)*mp, ms), s.b1), __fmul_rn(g, s.c1));
        r[j] = root<true>(__fadd_rn(__fmul_rn(v0, s.b2), __fmul_rn(__fmul_rn(g, g), s.c2)));
        TP *const p = (MASTER ? reinterpret_cast<TP *>(t.master) : static_cast<TP *>(t.p)) + at + j;
        const float q = __fmul_rn(m[j], reciprocal(__fmaf_rn(r[j], sc.inv_sqrt_bc2, s.eps)));
        const float x = __fmaf_rn(-sc.step_size, q, __fmul_rn((float)*p, fmaf(-sc.lr, t.wd, 1.f)));
        if constexpr (sizeof(TP) == 4) *p = x;
        else if (s.stochastic) *reinterpret_cast<uint16_t *>(p) = (uint16_t)bf16_pair(make_float2(x, x), u[j], u[j]);
        else *p = __float2bfloat16_rn(x);
        if constexpr (MASTER) static_cast<__nv_bfloat16 *>(t.p)[at + j] = __float2bfloat16_rn(x);
    }
    Eight<__nv_fp8_e4m3> to;
    const float new_ms = set_apart<false>(m, u, &to);
    store_some(static_cast<__nv_fp8_e4m3 *>(t.m) + at, n, to);
    const float new_rs = set_apart<true>(r, u, &to);
    store_some(static_cast<__nv_fp8_e4m3 *>(t.v) + at, n, to);
    return make_float2(new_ms, new_rs);
}

// The blocks b, b + kWarps, ... before `last` of a tensor, by a warp.  TP: the
// stepped parameter's type (a master copy's: fp32).
template <typename TP, typename TG, bool MASTER, bool SMALL>
__device__ __forceinline__ void step_chunk(const Entry &t, const Step &s, const moe_adamw_scalars_t &sc,
                                           float coef, int64_t first, int64_t last) {
    using B = Block<TP, TG, SMALL>;
    using TS = typename B::TS;
    const int lane = threadIdx.x & 31;
    int64_t b = first + (threadIdx.x >> 5);
    if (b >= last) return;
    TP *const stepped = MASTER ? reinterpret_cast<TP *>(t.master) : static_cast<TP *>(t.p);
    const float decay = fmaf(-sc.lr, t.wd, 1.f);
    const bool round_p = sizeof(TP) == 2 && s.stochastic;
    // the key and the scales of block b + i kWarps, in lane i (a scale that each block
    // waited for itself cost a round to memory: 64 M bf16 parameters 187 us, then 155)
    const int64_t mine = b + lane * kWarps;
    float ms = 0.f, rs = 0.f;
    if (SMALL && mine < last) {
        ms = t.ms[mine];
        rs = t.rs[mine];
    }
    Key keys = {0u, 0u};
    if (SMALL || round_p) keys = block_key(t.block0 + b + lane * kWarps, sc.seed_lo, sc.seed_hi);

    // (whole: vectors)
    auto fetch = [&](B &r, int64_t block, bool whole) {
        const int64_t at = block * kBlock + 8 * lane;
        if (whole) {
            r.p.load(stepped + at);
            r.g.load(static_cast<const TG *>(t.g) + at);
            r.m.load(static_cast<const TS *>(t.m) + at);
            r.v.load(static_cast<const TS *>(t.v) + at);
        } else {
            const int n = (int)max((int64_t)0, min((int64_t)8, t.numel - at));
            load_some(stepped + at, n, &r.p);
            load_some(static_cast<const TG *>(t.g) + at, n, &r.g);
            load_some(static_cast<const TS *>(t.m) + at, n, &r.m);
            load_some(static_cast<const TS *>(t.v) + at, n, &r.v);
        }
    };
    // a product that is rounded: the compiler fuses a packed product with the sum that
    // takes it, for all its .rn, but not one that is a multiply-add itself
    auto product = [&](float2 a, float b) { return fma2(a, two(b), two(s.minus_zero)); };
    const int64_t full = t.vec ? t.numel / kBlock : 0;
    for (int i = 0; b < last; ++i, b += kWarps) {
        B now;
        fetch(now, b, b < full);

        float2 p[4], g[4], m[4], v[4], r[4];
        unpack(now.p, p);
        unpack(now.g, g);
        unpack(now.m, m);
        unpack(now.v, v);
        if constexpr (SMALL) {
            const float old_ms = __shfl_sync(kAll, ms, i), old_rs = __shfl_sync(kAll, rs, i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                m[j] = mul2(m[j], two(old_ms));
                v[j] = mul2(v[j], two(old_rs));
                v[j] = mul2(v[j], v[j]);
            }
        }
        float top_m = 0.f, top_v = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 gj = mul2(g[j], two(coef));
            m[j] = add2(product(m[j], s.b1), product(gj, s.c1));
            v[j] = add2(product(v[j], s.b2), product(mul2(gj, gj), s.c2));
            r[j] = make_float2(root<SMALL>(v[j].x), root<SMALL>(v[j].y));
            const float2 d = fma2(r[j], two(sc.inv_sqrt_bc2), two(s.eps));
            const float2 q = mul2(m[j], make_float2(reciprocal(d.x), reciprocal(d.y)));
            p[j] = fma2(two(-sc.step_size), q, mul2(p[j], two(decay)));
            if constexpr (SMALL) {
                top_m = max_abs(top_m, m[j].x, m[j].y);
                top_v = max_abs(top_v, v[j].x, v[j].y);
            }
        }
        uint32_t u[8];
        if (SMALL || round_p) {
            const Key key = {__shfl_sync(kAll, keys.x, i), __shfl_sync(kAll, keys.y, i)};
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = random_bits(key, 8 * lane + j);
        }
        uint32_t largest_m = 0u, largest_v = 0u;
        if constexpr (SMALL) {
            largest_m = __reduce_max_sync(kAll, __float_as_uint(top_m));
            largest_v = __reduce_max_sync(kAll, __float_as_uint(top_v));
            if (max(largest_m, largest_v) >= 0x7f800000u) {  // (uniform) a NaN or an infinity
                const Key key = {__shfl_sync(kAll, keys.x, i), __shfl_sync(kAll, keys.y, i)};
                const float2 scales = seldom_block<TP, TG, MASTER>(t, s, coef, b, __shfl_sync(kAll, ms, i),
                                                                   __shfl_sync(kAll, rs, i), key);
                if (lane == i) {
                    ms = scales.x;
                    rs = scales.y;
                }
                continue;
            }
        }
        // (each is stored as soon as it is known: registers)
        const int64_t at = b * kBlock + 8 * lane;
        const int n = (int)max((int64_t)0, min((int64_t)8, t.numel - at));
        auto put = [&](auto *to, const auto &x) {
            if (b < full) x.store(to + at);
            else store_some(to + at, n, x);
        };
        Eight<TP> op;
        if (sizeof(TP) == 2 && round_p) {
            if constexpr (sizeof(TP) == 2)
                op.c = make_uint4(bf16_pair(p[0], u[0], u[1]), bf16_pair(p[1], u[2], u[3]),
                                  bf16_pair(p[2], u[4], u[5]), bf16_pair(p[3], u[6], u[7]));
        } else {
            pack(p, &op);
        }
        put(stepped, op);
        if constexpr (MASTER) {
            Eight<__nv_bfloat16> copy;
            pack(p, &copy);
            put(static_cast<__nv_bfloat16 *>(t.p), copy);
        }
        Eight<TS> state;
        if constexpr (SMALL) {
            const float new_ms = quantise<false>(m, scale_exponent(largest_m), u);
            pack(m, &state);
            put(static_cast<TS *>(t.m), state);
            const float new_rs = quantise<true>(r, root_scale_exponent(largest_v), u);
            pack(r, &state);
            put(static_cast<TS *>(t.v), state);
            if (lane == i) {
                ms = new_ms;
                rs = new_rs;
            }
        } else {
            pack(m, &state);
            put(static_cast<TS *>(t.m), state);
            pack(v, &state);
            put(static_cast<TS *>(t.v), state);
        }
    }
    if constexpr (SMALL) {
        if (mine < last) {
            t.ms[mine] = ms;
            t.rs[mine] = rs;
        }
    }
}

// Blocks an SM: with 8-bit states four (64 M parameters 137 us; three took 152, and
// five, for which registers spill, 153); with fp32 states three (213 us against 236
// with four, whose accesses are spread over more of the memory's rows).
template <bool SMALL>
__global__ void __launch_bounds__(kThreads, SMALL ? 4 : 3)
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
    const int c = blockIdx.x;
    int lo = 0, hi = tab.n - 1;
    if (tab.mapped) lo = hi = tab.tensor_of[c];
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (tab.t[mid].end > c) hi = mid; else lo = mid + 1;
    }
    const Entry &t = tab.t[lo];
    const int64_t blocks = (t.numel + kBlock - 1) / kBlock;
    const int64_t all = (blocks + tab.chunk_blocks - 1) / tab.chunk_blocks;
    const int64_t first = (c - (t.end - all)) * tab.chunk_blocks;
    const int64_t last = min(blocks, first + tab.chunk_blocks);
    if (!t.p_bf16) {
        if (t.g_bf16) step_chunk<float, __nv_bfloat16, false, SMALL>(t, s, sc, coef, first, last);
        else step_chunk<float, float, false, SMALL>(t, s, sc, coef, first, last);
    } else if (!t.master) {
        if (t.g_bf16) step_chunk<__nv_bfloat16, __nv_bfloat16, false, SMALL>(t, s, sc, coef, first, last);
        else step_chunk<__nv_bfloat16, float, false, SMALL>(t, s, sc, coef, first, last);
    } else {
        if (t.g_bf16) step_chunk<float, __nv_bfloat16, true, SMALL>(t, s, sc, coef, first, last);
        else step_chunk<float, float, true, SMALL>(t, s, sc, coef, first, last);
    }
}

// launch_pdl without its copy of the 32 KB of parameters (0.4 us a call).
cudaError_t launch(void (*kernel)(Table, Step), int grid, Table &tab, Step &s, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[] = {&tab, &s};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(kernel), args);
}

int64_t blocks_of(int64_t numel) { return (numel + kBlock - 1) / kBlock; }

bool vectors(const moe_adamw_tensor_t &t) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(t.param) | reinterpret_cast<uintptr_t>(t.grad) |
                          reinterpret_cast<uintptr_t>(t.exp_avg) |
                          reinterpret_cast<uintptr_t>(t.exp_avg_sq) |
                          reinterpret_cast<uintptr_t>(t.master);
    return (all & 15) == 0;
}

}  // namespace

int64_t adamw_chunk() { return kWarps * kBlock; }

cudaError_t launch_adamw(const moe_adamw_tensor_t *ts, int64_t n, const moe_adamw_scalars_t &sc,
                         const moe_adamw_scalars_t *dev, const moe_adamw_hyper_t &h,
                         const float *norm, cudaStream_t st) {
    Step s = {};
    s.b1 = (float)h.beta1;
    s.c1 = (float)(1.0 - h.beta1);
    s.b2 = (float)h.beta2;
    s.c2 = (float)(1.0 - h.beta2);
    s.eps = (float)h.eps;
    s.minus_zero = -0.f;
    s.max_norm = h.max_norm;
    s.stochastic = h.stochastic;
    s.skip_nonfinite = h.skip_nonfinite;
    s.sc = sc;
    s.dev = dev;
    s.norm = norm;
    Table tab;
    int64_t blocks = 0;
    for (int64_t i = 0; i < n; ++i) blocks += blocks_of(ts[i].numel);
    tab.chunk_blocks = kWarps;
    while (tab.chunk_blocks < kMostBlocks &&
           (int64_t)tab.chunk_blocks * tab.chunk_blocks * kSquare < blocks)
        tab.chunk_blocks *= 2;
    for (const bool small : {false, true}) {
        int64_t block0 = 0, i = 0;
        while (i < n) {
            tab.n = 0;
            int end = 0;
            for (; i < n && tab.n < kTable; ++i) {
                const moe_adamw_tensor_t &t = ts[i];
                const int64_t first = block0;
                block0 += blocks_of(t.numel);
                if (t.numel == 0 || (t.state_dtype == MOE_E4M3) != small) continue;
                const int from = end;
                end += (int)((blocks_of(t.numel) + tab.chunk_blocks - 1) / tab.chunk_blocks);
                for (int c = from; c < end && c < kMapped; ++c) tab.tensor_of[c] = (uint16_t)tab.n;
                tab.t[tab.n++] = {t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.exp_avg_scale,
                                  t.exp_avg_sq_scale, t.master, t.numel, first, end, t.weight_decay,
                                  t.param_dtype == MOE_BF16, t.grad_dtype == MOE_BF16, vectors(t)};
            }
            if (tab.n == 0) continue;
            tab.chunks = end;
            tab.mapped = end <= kMapped;
            const cudaError_t e = launch(small ? adamw_kernel<true> : adamw_kernel<false>, end, tab, s, st);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaGetLastError();
}

}  // namespace moe
