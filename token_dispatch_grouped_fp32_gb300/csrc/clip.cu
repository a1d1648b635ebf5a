// clip.cu -- the global norm of many gradient tensors, and their clipped
// copies:  N = sqrt(sum of all squares),  out = g * min(1, max_norm / (N + 1e-6)).
//
// Launch 1 (norm_kernel): the tensors are cut into chunks of kChunk elements;
// block b sums the squares of chunks b, b + grid, ... (a thread's 64 of a chunk
// in fp32, with their scale adjusted where they leave its range; doubles beyond)
// and writes one double.  Launch 2 (scale_kernel): every block adds the partial
// sums of launch 1 in the same order, so each has the same norm and no block
// waits for another, and scales its chunks.  The tensors' addresses and sizes
// travel as kernel parameters: no copy to the device, and the calls can be
// captured in a graph.
//
// Bound by HBM where the set exceeds L2: three passes over its bytes (1.41 G
// elements of a Mixtral-shaped layer, 8.46 GB: 1266 us, 0.98 of the copy rate).
// 300 tensors of up to 20,000 elements: 10.3 us, two launches and their chains
// of table, data and norm (25.7 with 912 blocks whatever the chunks, and the
// table in separate arrays).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 16384;
constexpr int kBlocks = 152 * 6;
constexpr int kTable = 512;    // tensors per launch
constexpr int kMapped = 1024;  // chunks with a map of their own

// One tensor: a whole 32 bytes, so that a block finds it in one line.
struct Entry {
    const void *src;
    void *dst;
    int64_t numel;
    int end;   // chunks of the tensors up to and with this one
    int bf16;
};
struct Table {
    int n, chunks;
    // where the table's chunks are few (most tensors one chunk): the tensor
    // of every chunk, so that a block finds its own in one load
    int mapped;
    uint16_t tensor_of[kMapped];
    Entry t[kTable];
};

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double s[kThreads / 32];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
    for (int i = 0; i < kThreads / 32; ++i) t += s[i];
    __syncthreads();
    return t;
}

struct Chunk {
    Entry t;
    int64_t first;
    int count;
};
__device__ __forceinline__ Chunk find_chunk(const Table &t, int c) {
    int lo = 0, hi = t.n - 1;
    if (t.mapped) lo = hi = t.tensor_of[c];
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (t.t[mid].end > c) hi = mid; else lo = mid + 1;
    }
    Chunk k;
    k.t = t.t[lo];
    const int all = (int)((k.t.numel + kChunk - 1) / kChunk);
    k.first = (int64_t)(c - (k.t.end - all)) * kChunk;
    k.count = (int)min((int64_t)kChunk, k.t.numel - k.first);
    return k;
}

// This thread's share of the sum of (scale g)^2 over a chunk; any: the bits set in
// its elements, but for their signs.
template <typename TA, bool SCALED>
__device__ __forceinline__ float thread_squares(const TA *p, int n, float scale, uint32_t *any) {
    constexpr int EPV = 16 / sizeof(TA);
    const int head = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(TA));
    float s = 0.f;
    uint32_t bits = 0;
    auto one = [&](TA g) {
        const float v = SCALED ? scale * Act<TA>::to_f(g) : Act<TA>::to_f(g);
        bits |= __float_as_uint(v) & 0x7fffffffu;
        s = fmaf(v, v, s);
    };
    if ((int)threadIdx.x < head) one(p[threadIdx.x]);
    const int nv = (n - head) / EPV;
    const TA *q = p + head;
#pragma unroll 4
    for (int i = threadIdx.x; i < nv; i += kThreads) {
        const uint4 raw = ldg16(q + (int64_t)i * EPV);
        float v[EPV];
        unpack16(raw, v, static_cast<const TA *>(nullptr));
        if (!SCALED)
            bits |= (raw.x | raw.y | raw.z | raw.w) & (sizeof(TA) == 2 ? 0x7fff7fffu : 0x7fffffffu);
#pragma unroll
        for (int j = 0; j < EPV; ++j) {
            if (SCALED) v[j] *= scale;
            s = fmaf(v[j], v[j], s);
        }
    }
    const int tail = head + nv * EPV + threadIdx.x;
    if (tail < n) one(p[tail]);
    *any = bits;
    return s;
}

// ... without a scale, and where that sum left fp32's range, again with a power of
// two that is taken out afterwards.  A sum that overflowed: all terms are within
// 2^96 then, and what underflows is below 2^-110 of it.  A sum below 2^-100 that
// is not of zeros alone: every element is below 2^-50, and the smallest
// subnormal's square becomes 2^-98.  From 2^-100 up, what a square lost by
// underflow is below 2^-43 of the sum.  The zeros of an expert without rows stay
// on the first pass.
template <typename TA> __device__ __forceinline__ double chunk_squares(const TA *p, int n) {
    uint32_t any, unused;
    const float s = thread_squares<TA, false>(p, n, 1.f, &any);
    if (any == 0 || (s >= 0x1p-100f && s < INFINITY)) return s;
    const bool small = s < 0x1p-100f;  // else an overflow, an infinity or a NaN
    return (double)thread_squares<TA, true>(p, n, small ? 0x1p100f : 0x1p-80f, &unused) *
           (small ? 0x1p-200 : 0x1p160);
}

// The scale as a product of two factors, the second 1 or, where the scale itself
// would be subnormal (a norm near fp32's end), a power of two.  Two factors take
// the simple loop: in the vector loop the second one cost the whole Mixtral-shaped
// set 6 % (1266 us to 1346), whatever its value.
struct Scale {
    float a, b;
};
__device__ __forceinline__ Scale scale_for(float max_norm, float nrm) {
    const float c = max_norm / (nrm + 1e-6f);
    if (c < 0x1p-100f) return {max_norm * 0x1p100f / (nrm + 1e-6f), 0x1p-100f};
    return {c > 1.f ? 1.f : c, 1.f};  // a NaN norm stays NaN
}

template <typename TA>
__device__ __forceinline__ void chunk_scale(const TA *p, TA *o, int n, const Scale &scale) {
    constexpr int EPV = 16 / sizeof(TA);
    const unsigned mp = reinterpret_cast<uintptr_t>(p) & 15, mo = reinterpret_cast<uintptr_t>(o) & 15;
    if (mp != mo || scale.b != 1.f) {  // no common 16-byte boundary, or two factors
        for (int i = threadIdx.x; i < n; i += kThreads)
            o[i] = Act<TA>::from_f(Act<TA>::to_f(p[i]) * scale.a * scale.b);
        return;
    }
    const float coef = scale.a;
    const int head = min(n, (int)((16 - mp) & 15) / (int)sizeof(TA));
    if ((int)threadIdx.x < head) o[threadIdx.x] = Act<TA>::from_f(Act<TA>::to_f(p[threadIdx.x]) * coef);
    const int nv = (n - head) / EPV;
    constexpr int U = 4;  // loads before the first store (o may be p)
    for (int i0 = threadIdx.x; i0 < nv; i0 += U * kThreads) {
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * kThreads < nv)
                raw[u] = *reinterpret_cast<const uint4 *>(p + head + (int64_t)(i0 + u * kThreads) * EPV);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u * kThreads >= nv) continue;
            float v[EPV];
            unpack16(raw[u], v, static_cast<const TA *>(nullptr));
#pragma unroll
            for (int j = 0; j < EPV; ++j) v[j] *= coef;
            stg16(o + head + (int64_t)(i0 + u * kThreads) * EPV,
                  pack16(v, static_cast<const TA *>(nullptr)));
        }
    }
    const int tail = head + nv * EPV + threadIdx.x;
    if (tail < n) o[tail] = Act<TA>::from_f(Act<TA>::to_f(p[tail]) * coef);
}

__global__ void __launch_bounds__(kThreads)
norm_kernel(const __grid_constant__ Table t, int add, double *__restrict__ part) {
    pdl_wait();
    double sum = 0.0;
    for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const Chunk k = find_chunk(t, c);
        sum += k.t.bf16
                   ? chunk_squares(static_cast<const __nv_bfloat16 *>(k.t.src) + k.first, k.count)
                   : chunk_squares(static_cast<const float *>(k.t.src) + k.first, k.count);
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) part[blockIdx.x] = add ? part[blockIdx.x] + sum : sum;
}

__global__ void __launch_bounds__(kThreads)
scale_kernel(const __grid_constant__ Table t, const double *__restrict__ part, int parts,
             float max_norm, float *__restrict__ norm) {
    pdl_wait();
    double sum = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) sum += part[i];
    const float nrm = (float)sqrt(block_sum(sum));
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = nrm;
    const Scale scale = scale_for(max_norm, nrm);
    // from the last chunk: what launch 1 read last is still in the L2 cache
    // (the Mixtral-shaped layer's gradients: 1350 us forward, 1277 us backward)
    for (int c = t.chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
        const Chunk k = find_chunk(t, c);
        if (k.t.dst == nullptr) continue;
        if (k.t.bf16)
            chunk_scale(static_cast<const __nv_bfloat16 *>(k.t.src) + k.first,
                        static_cast<__nv_bfloat16 *>(k.t.dst) + k.first, k.count, scale);
        else
            chunk_scale(static_cast<const float *>(k.t.src) + k.first,
                        static_cast<float *>(k.t.dst) + k.first, k.count, scale);
    }
}

int chunks_of(const moe_grad_t &g) { return (int)((g.numel + kChunk - 1) / kChunk); }

void fill(const moe_grad_t *g, int64_t n, Table *t) {
    int end = 0;
    for (int64_t i = 0; i < n; ++i) {
        const int first = end;
        end += chunks_of(g[i]);
        t->t[i] = {g[i].grad, g[i].out, g[i].numel, end, g[i].dtype == MOE_BF16};
        for (int c = first; c < end && c < kMapped; ++c) t->tensor_of[c] = (uint16_t)i;
    }
    t->n = (int)n;
    t->chunks = end;
    t->mapped = end <= kMapped;
}

}  // namespace

size_t clip_scratch_bytes() { return sizeof(double) * kBlocks; }
int64_t clip_chunk() { return kChunk; }

cudaError_t launch_clip(const moe_grad_t *g, int64_t n, float max_norm, float *norm, void *ws,
                        cudaStream_t st) {
    Table t;
    double *part = static_cast<double *>(ws);
    // as many blocks as the longest launch has chunks: each writes a partial sum
    int most = 1;
    for (int64_t i = 0; i < n; i += kTable) {
        int c = 0;
        for (int64_t j = i; j < std::min<int64_t>(n, i + kTable); ++j) c += chunks_of(g[j]);
        most = std::max(most, c);
    }
    const int blocks = std::min(kBlocks, most);
    for (int64_t i = 0; i == 0 || i < n; i += kTable) {
        fill(g + i, std::min<int64_t>(kTable, n - i), &t);
        launch_pdl(norm_kernel, dim3(blocks), dim3(kThreads), 0, st, t, i > 0 ? 1 : 0, part);
    }
    for (int64_t i = 0; i == 0 || i < n; i += kTable) {
        if (n > kTable) fill(g + i, std::min<int64_t>(kTable, n - i), &t);
        launch_pdl(scale_kernel, dim3(blocks), dim3(kThreads), 0, st, t, (const double *)part, blocks,
                   max_norm, norm);
    }
    return cudaGetLastError();
}

}  // namespace moe
