// The norm of all gradients together and their scaling to a largest norm, over lists of
// tensors of any sizes.  The list travels in the kernel's parameters: no table is copied to
// the device, so a call enqueues kernels alone and can be captured.  Both are HBM-bound: a 7B layer's 233 million fp32
// values 138 us for the norm, 207 us scaled into bf16 (6.75 TB/s, the copy rate) and 331 in place (5.6 TB/s), 1036
// matrices of at most 128 x 3584 in bf16 73 us (6.0 TB/s).  What is left for short lists are about 6 us of launch, first
// loads and the last block's sum, and 5 more for the 32 KB of parameters of long ones.
#include "act8.cuh"
#include "grads.h"
#include "kernels.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
// Blocks per SM: 32 KB of loads in flight each (256 threads, 8 loads of 16 bytes) cover HBM's latency.
constexpr int kFit = 4;
constexpr int kWords = 32;   // of a chunk per thread

// A thread's groups of a chunk as loaded: group i is its i-th of every kThreads-th.
template <bool BF16>
struct Groups {
    static constexpr int kPer = BF16 ? 4 : 8, kCount = kWords / kPer;
    static_assert(kCount * kThreads == (BF16 ? kChunkGroups16 : kChunkGroups32), "the chunk's groups");
    uint32_t r[kWords];
    // Groups from g0 on of a gradient whose first group begins `pad` values before it; zero outside it.  vec: whole
    // groups are aligned to 16 bytes.
    __device__ __forceinline__ void load(const GradEntry& e, long long g0, bool vec) {
        const long long first = (g0 + threadIdx.x) * 8 - e.pad;
        if (vec && g0 * 8 >= e.pad && (g0 + kCount * kThreads) * 8 - e.pad <= e.count) {   // the whole chunk
#pragma unroll
            for (int i = 0; i < kCount; ++i) whole(e.p, first + i * 8ll * kThreads, r + i * kPer);
            return;
        }
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const long long at = first + i * 8ll * kThreads;
            if (vec && at >= 0 && at + 8 <= e.count) {
                whole(e.p, at, r + i * kPer);
            } else {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = at + j >= 0 && at + j < e.count ? load_one<BF16>(e.p, at + j) : 0.f;
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    r[i * kPer + j] =
                        BF16 ? bf16_bits(v[2 * j]) | bf16_bits(v[2 * j + 1]) << 16 : __float_as_uint(v[j]);
            }
        }
    }
    static __device__ __forceinline__ uint32_t bf16_bits(float v) { return __float_as_uint(v) >> 16; }
    static __device__ __forceinline__ void whole(const void* p, long long at, uint32_t* w) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * (BF16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < kPer / 4; ++i) {
            const uint4 a = __ldcs(q + i);
            w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
        }
    }
    __device__ __forceinline__ void get(int i, float (&v)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (BF16)
                v[j] = j & 1 ? bf16_hi(r[i * kPer + j / 2]) : bf16_lo(r[i * kPer + j / 2]);
            else
                v[j] = __uint_as_float(r[i * kPer + j % kPer]);
        }
    }
};

template <bool BF16>
__device__ __forceinline__ void store_eight(void* p, long long start, long long count, const float (&v)[8]) {
    if (start >= 0 && start + 8 <= count) {   // aligned by the groups' layout
        uint4* q = reinterpret_cast<uint4*>(static_cast<char*>(p) + start * (BF16 ? 2 : 4));
        if (BF16) {
            q[0] = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
        } else {
            const uint4* w = reinterpret_cast<const uint4*>(v);
            q[0] = w[0], q[1] = w[1];
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (start + j >= 0 && start + j < count) store_one<BF16>(p, start + j, v[j]);
}

// Squares of a thread's values of a chunk in 64 bits, read again.
template <bool BF16>
__device__ __noinline__ double chunk_squares_wide(const void* p, long long first, long long count) {
    double d = 0.0;
    for (int i = 0; i < Groups<BF16>::kCount; ++i)
        for (int j = 0; j < 8; ++j) {
            const long long at = first + i * 8ll * kThreads + j;
            const double v = at >= 0 && at < count ? (double)load_one<BF16>(p, at) : 0.0;
            d += v * v;
        }
    return d;
}
// The same, in fp32 by four sums of at most 16 values; where one of them is beyond the range in which every square
// that counts is exact to 2^-24 (an overflow, or values below 2^-45), in 64 bits, so that the norm is right for
// gradients of any scale.  Sums of zeros that are exact are the common case among small ones.
template <bool BF16>
__device__ __forceinline__ double chunk_squares(const GradEntry& e, long long g0) {
    Groups<BF16> g;
    g.load(e, g0, true);
    float s[4] = {};
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < g.kCount; ++i) {
        float v[8];
        g.get(i, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[(i * 8 + j) & 3] = fmaf(v[j], v[j], s[(i * 8 + j) & 3]);
#pragma unroll
        for (int j = 0; j < g.kPer; ++j) any |= BF16 ? g.r[i * g.kPer + j] & 0x7fff7fffu : g.r[i * g.kPer + j] << 1;
    }
    const float least = fminf(fminf(s[0], s[1]), fminf(s[2], s[3])), sum = (s[0] + s[1]) + (s[2] + s[3]);
    if ((least > 8.0e-28f && sum <= 3.0e38f) || any == 0) return sum;
    return chunk_squares_wide<BF16>(e.p, (g0 + threadIdx.x) * 8 - e.pad, e.count);
}

// The chunks of this block, one after another, and the gradient that each lies in.
struct ChunkWalk {
    uint32_t c, to;
    int i;
    template <typename Table>
    __device__ __forceinline__ explicit ChunkWalk(const Table& t)
        : c((uint32_t)((uint64_t)t.chunks * blockIdx.x / gridDim.x)),
          to((uint32_t)((uint64_t)t.chunks * (blockIdx.x + 1) / gridDim.x)), i(t.start[blockIdx.x]) {}
    template <typename Table>
    __device__ __forceinline__ const GradEntry& entry(const Table& t) {
        while (i + 1 < t.n && t.e[i + 1].first <= c) ++i;
        return t.e[i];
    }
};

__device__ __forceinline__ double block_sum(double d) {
    __shared__ double part[kThreads / 32];
#pragma unroll
    for (int k = 16; k > 0; k /= 2) d += __shfl_xor_sync(0xffffffffu, d, k);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = d;
    __syncthreads();
    d = part[0];
#pragma unroll
    for (int k = 1; k < kThreads / 32; ++k) d += part[k];
    return d;
}

// Block b sums a contiguous share of the chunks; the block that comes last adds up all blocks' sums in
// their order, so the same gradients give the same bits.
template <int N>
__global__ void __launch_bounds__(kThreads, kFit) k_grad_norm(const __grid_constant__ GradTable<N, false> t, double* partial,
                                                        double* running, int* arrived, float* norm, int first, int last) {
    pdl_trigger();
    pdl_wait();
    double sum = 0.0;
    for (ChunkWalk w(t); w.c < w.to; ++w.c) {
        const GradEntry& e = w.entry(t);
        const long long k = w.c - e.first;
        sum += e.bf16 ? chunk_squares<true>(e, k * kChunkGroups16) : chunk_squares<false>(e, k * kChunkGroups32);
    }
    sum = block_sum(sum);
    __shared__ bool is_last;
    if (threadIdx.x == 0) {
        partial[blockIdx.x] = sum;
        __threadfence();
        is_last = atomicAdd(arrived, 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    double all = 0.0;
    for (int b = threadIdx.x; b < (int)gridDim.x; b += kThreads) all += __ldcg(partial + b);
    __syncthreads();
    all = block_sum(all);
    if (threadIdx.x == 0) {
        if (!first) all += *running;
        *running = all;
        *arrived = 0;
        if (last) *norm = (float)sqrt(all);
    }
}

template <bool IN16, bool OUT16>
__device__ __forceinline__ void chunk_scale(const GradEntry& e, void* out, long long g0, float f) {
    Groups<IN16> g;
    g.load(e, g0, ((reinterpret_cast<uintptr_t>(e.p) - e.pad * (IN16 ? 2 : 4)) & 15) == 0);
#pragma unroll
    for (int i = 0; i < g.kCount; ++i) {
        float v[8];
        g.get(i, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= f;
        store_eight<OUT16>(out, (g0 + i * kThreads + threadIdx.x) * 8 - e.pad, e.count, v);
    }
}

// out = g times max_norm / norm where the norm is finite and beyond max_norm, else g itself; in place
// nothing is read or written then.
template <int N>
__global__ void __launch_bounds__(kThreads, kFit) k_grad_clip(const __grid_constant__ GradTable<N, true> t, const float* norm,
                                                        float max_norm, int in_place) {
    pdl_trigger();
    pdl_wait();
    const float x = *norm;
    const float f = x > max_norm && x <= 3.402823466e38f ? max_norm / x : 1.f;
    if (in_place && f == 1.f) return;
    for (ChunkWalk w(t); w.c < w.to; ++w.c) {
        const GradEntry& e = w.entry(t);
        const long long k = w.c - e.first;
        if (e.bf16)
            e.out_bf16 ? chunk_scale<true, true>(e, t.out[w.i], k * kChunkGroups16, f)
                       : chunk_scale<true, false>(e, t.out[w.i], k * kChunkGroups16, f);
        else
            e.out_bf16 ? chunk_scale<false, true>(e, t.out[w.i], k * kChunkGroups32, f)
                       : chunk_scale<false, false>(e, t.out[w.i], k * kChunkGroups32, f);
    }
}

template <int N>
cudaError_t norm_of(const GradList& l, int from, int to, const GradNormArgs& a, bool last, cudaStream_t s) {
    GradTable<N, false> t;
    const int blocks = l.table(from, to, kFit * a.sm_count, &t);
    return launch_pdl(k_grad_norm<N>, dim3(blocks), dim3(kThreads), 0, s, t, a.partial, a.running, a.arrived, a.norm,
                      from == 0, (int)last);
}
template <int N>
cudaError_t clip_of(const GradList& l, int from, int to, const float* norm, float max_norm, int sm_count,
                    cudaStream_t s) {
    GradTable<N, true> t;
    const int blocks = l.table(from, to, kFit * sm_count, &t);
    return launch_pdl(k_grad_clip<N>, dim3(blocks), dim3(kThreads), 0, s, t, norm, max_norm, (int)l.in_place);
}

}  // namespace

cudaError_t launch_grad_norm(const GradList& l, const GradNormArgs& a, cudaStream_t s) {
    for (int from = 0; from == 0 || from < l.n; from += kTableNorm) {
        const int to = std::min(l.n, from + kTableNorm);
        const bool last = to == l.n;
        const cudaError_t e = to - from <= kTableFew    ? norm_of<kTableFew>(l, from, to, a, last, s)
                              : to - from <= kTableSome ? norm_of<kTableSome>(l, from, to, a, last, s)
                                                        : norm_of<kTableNorm>(l, from, to, a, last, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_grad_clip(const GradList& l, const float* norm, float max_norm, int sm_count, cudaStream_t s) {
    for (int from = 0; from < l.n; from += kTableClip) {
        const int to = std::min(l.n, from + kTableClip);
        const cudaError_t e = to - from <= kTableFew    ? clip_of<kTableFew>(l, from, to, norm, max_norm, sm_count, s)
                              : to - from <= kTableSome ? clip_of<kTableSome>(l, from, to, norm, max_norm, sm_count, s)
                                                        : clip_of<kTableClip>(l, from, to, norm, max_norm, sm_count, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace muon
