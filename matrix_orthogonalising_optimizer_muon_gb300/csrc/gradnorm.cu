// The norm of all gradients together and their scaling to a largest norm, over lists of
// tensors of any sizes.  The list travels in the kernel's parameters: no table is copied to
// the device, so a call enqueues kernels alone and can be captured.
#include "act8.cuh"
#include "grads.h"
#include "kernels.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kUnrollGroups = kChunkGroups / kThreads;   // of eight values per thread and chunk

// Eight values of a gradient from element `start` on, zero outside [0, count).
template <bool BF16>
__device__ __forceinline__ void load_eight(const void* p, long long start, long long count, bool vec, float (&v)[8]) {
    if (vec && start >= 0 && start + 8 <= count) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + start * (BF16 ? 2 : 4));
        if (BF16) {
            const uint4 a = q[0];
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
        } else {
            const uint4 a = q[0], b = q[1];
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = start + j >= 0 && start + j < count ? load_one<BF16>(p, start + j) : 0.f;
}

template <bool BF16>
__device__ __forceinline__ void store_eight(void* p, long long start, long long count, const float (&v)[8]) {
    if (start >= 0 && start + 8 <= count) {   // aligned by the chunks' layout
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

// Squares of a chunk's values.  fp32 sums of one thread's run; a run whose sum is beyond the range where every
// square that counts is exact to 2^-24 (an overflow, or values below 2^-45) is summed again in 64 bits, so that
// the norm is right for gradients of any scale.
template <bool BF16>
__device__ __forceinline__ double chunk_squares(const GradEntry& e, long long g0) {
    float v[kUnrollGroups][8];
#pragma unroll
    for (int k = 0; k < kUnrollGroups; ++k)
        load_eight<BF16>(e.p, (g0 + k * kThreads + threadIdx.x) * 8 - e.pad, e.count, true, v[k]);
    float s = 0.f;
    uint32_t any = 0;
#pragma unroll
    for (int k = 0; k < kUnrollGroups; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s = fmaf(v[k][j], v[k][j], s);
            any |= __float_as_uint(v[k][j]) << 1;
        }
    if (any == 0) return 0.0;
    if (s > 8.0e-28f && s <= 3.0e38f) return s;
    double d = 0.0;
#pragma unroll
    for (int k = 0; k < kUnrollGroups; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) d += (double)v[k][j] * (double)v[k][j];
    return d;
}

// Index of the gradient that chunk c lies in.
template <int N>
__device__ __forceinline__ int find_entry(const GradTable<N>& t, uint32_t c) {
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.e[mid].first <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

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
__global__ void __launch_bounds__(kThreads) k_grad_norm(const __grid_constant__ GradTable<N> t, double* partial,
                                                        double* running, int* arrived, float* norm, int first, int last) {
    pdl_trigger();
    pdl_wait();
    const uint32_t from = (uint32_t)((uint64_t)t.chunks * blockIdx.x / gridDim.x);
    const uint32_t to = (uint32_t)((uint64_t)t.chunks * (blockIdx.x + 1) / gridDim.x);
    double sum = 0.0;
    int i = from < to ? find_entry(t, from) : 0;
    for (uint32_t c = from; c < to; ++c) {
        while (i + 1 < t.n && t.e[i + 1].first <= c) ++i;
        const GradEntry& e = t.e[i];
        const long long g0 = (long long)(c - e.first) * kChunkGroups;
        sum += e.bf16 ? chunk_squares<true>(e, g0) : chunk_squares<false>(e, g0);
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
__device__ __forceinline__ void chunk_scale(const GradEntry& e, long long g0, float f) {
    const bool vec = ((reinterpret_cast<uintptr_t>(e.p) - e.pad * (IN16 ? 2 : 4)) & 15) == 0;
    float v[kUnrollGroups][8];
#pragma unroll
    for (int k = 0; k < kUnrollGroups; ++k)
        load_eight<IN16>(e.p, (g0 + k * kThreads + threadIdx.x) * 8 - e.pad, e.count, vec, v[k]);
#pragma unroll
    for (int k = 0; k < kUnrollGroups; ++k) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] *= f;
        store_eight<OUT16>(e.out, (g0 + k * kThreads + threadIdx.x) * 8 - e.pad, e.count, v[k]);
    }
}

// out = g times max_norm / norm where the norm is finite and beyond max_norm, else g itself; in place
// nothing is read or written then.
template <int N>
__global__ void __launch_bounds__(kThreads) k_grad_clip(const __grid_constant__ GradTable<N> t, const float* norm,
                                                        float max_norm, int in_place) {
    pdl_trigger();
    pdl_wait();
    const float x = *norm;
    const float f = x > max_norm && x <= 3.402823466e38f ? max_norm / x : 1.f;
    if (in_place && f == 1.f) return;
    const uint32_t from = (uint32_t)((uint64_t)t.chunks * blockIdx.x / gridDim.x);
    const uint32_t to = (uint32_t)((uint64_t)t.chunks * (blockIdx.x + 1) / gridDim.x);
    int i = from < to ? find_entry(t, from) : 0;
    for (uint32_t c = from; c < to; ++c) {
        while (i + 1 < t.n && t.e[i + 1].first <= c) ++i;
        const GradEntry& e = t.e[i];
        const long long g0 = (long long)(c - e.first) * kChunkGroups;
        if (e.bf16)
            e.out_bf16 ? chunk_scale<true, true>(e, g0, f) : chunk_scale<true, false>(e, g0, f);
        else
            e.out_bf16 ? chunk_scale<false, true>(e, g0, f) : chunk_scale<false, false>(e, g0, f);
    }
}

template <int N>
cudaError_t norm_of(const GradList& l, int from, int to, const GradNormArgs& a, bool last, cudaStream_t s) {
    GradTable<N> t;
    l.table(from, to, &t);
    const int blocks = (int)std::min<long long>(t.chunks, 4ll * a.sm_count);
    return launch_pdl(k_grad_norm<N>, dim3(std::max(blocks, 1)), dim3(kThreads), 0, s, t, a.partial, a.running, a.arrived,
                      a.norm, from == 0, (int)last);
}
template <int N>
cudaError_t clip_of(const GradList& l, int from, int to, const float* norm, float max_norm, int sm_count,
                    cudaStream_t s) {
    GradTable<N> t;
    l.table(from, to, &t);
    const int blocks = (int)std::min<long long>(t.chunks, 4ll * sm_count);
    return launch_pdl(k_grad_clip<N>, dim3(std::max(blocks, 1)), dim3(kThreads), 0, s, t, norm, max_norm, (int)l.in_place);
}

}  // namespace

cudaError_t launch_grad_norm(const GradList& l, const GradNormArgs& a, cudaStream_t s) {
    for (int from = 0; from == 0 || from < l.n; from += kTableMost) {
        const int to = std::min(l.n, from + kTableMost);
        const bool last = to == l.n;
        const cudaError_t e = to - from <= kTableFew ? norm_of<kTableFew>(l, from, to, a, last, s)
                                                     : norm_of<kTableMost>(l, from, to, a, last, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_grad_clip(const GradList& l, const float* norm, float max_norm, int sm_count, cudaStream_t s) {
    for (int from = 0; from < l.n; from += kTableMost) {
        const int to = std::min(l.n, from + kTableMost);
        const cudaError_t e = to - from <= kTableFew ? clip_of<kTableFew>(l, from, to, norm, max_norm, sm_count, s)
                                                     : clip_of<kTableMost>(l, from, to, norm, max_norm, sm_count, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace muon
