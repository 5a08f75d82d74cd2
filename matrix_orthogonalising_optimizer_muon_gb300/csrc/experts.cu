// Tokens in their experts' order and back: the order itself (a stable counting sort of the
// chosen experts), the move of rows into it, their weighted sum per token, and its gradients.
#include <algorithm>

#include "act8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace muon {
namespace {

// ------------------------------------------------------------------ order
// slots[i] = offsets[ids[i]] + number of h < i with ids[h] = ids[i].  One cluster: CTA r takes a
// contiguous share of the ids, its warps contiguous shares of that.  Pass 1 counts each warp's ids by
// expert in shared memory; the counts of earlier warps, earlier CTAs (read from their shared memory)
// and smaller experts give each warp its first slot per expert; pass 2 deals the slots out, 32 ids at
// a time, neighbours with the same expert by their rank among the warp's lanes.
constexpr int kOrderThreads = 1024;
constexpr int kOrderCounts = 32768;   // counts in shared memory: warps x experts

__device__ __forceinline__ int remote_int(uint32_t local_saddr, uint32_t rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(local_saddr, rank)) : "memory");
    return v;
}

__global__ void __launch_bounds__(kOrderThreads) k_expert_order(const OrderArgs a, int warps, int ctas) {
    extern __shared__ int smem[];
    const int E = a.experts;
    int* count = smem;                    // [warps][E]
    int* total = smem + warps * E;        // [E]: this CTA's counts
    int* base = total + E;                // [E]: the CTA's first slot
    __shared__ int chunk[kOrderThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = ctas > 1 ? (int)cluster_ctarank() : 0;
    pdl_trigger();
    pdl_wait();

    for (int i = threadIdx.x; i < warps * E; i += kOrderThreads) count[i] = 0;
    __syncthreads();
    // shares of 32 ids, as even as that allows
    const long long groups = (a.n + 31) / 32, parts = (long long)ctas * warps, w = (long long)rank * warps + warp;
    const long long from = groups * w / parts * 32, to = min(groups * (w + 1) / parts * 32, a.n);
    int* mine = count + warp * E;
    if (warp < warps) {
        for (long long i = from + lane; i < to; i += 32) {
            const int id = a.ids[i];
            if ((unsigned)id < (unsigned)E) atomicAdd(mine + id, 1);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kOrderThreads) {   // counts of earlier warps
        int sum = 0;
        for (int k = 0; k < warps; ++k) {
            const int c = count[k * E + e];
            count[k * E + e] = sum;
            sum += c;
        }
        total[e] = sum;
    }
    if (ctas > 1)
        cluster_sync();
    else
        __syncthreads();
    // counts of earlier CTAs and of smaller experts: a scan over the experts, kOrderThreads at a time
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += kOrderThreads) {
        const int e = e0 + threadIdx.x;
        int before = 0, all = 0;
        if (e < E) {
            if (ctas > 1) {
                for (int r = 0; r < ctas; ++r) {
                    const int c = remote_int(smem_u32(total + e), r);
                    before += r < rank ? c : 0;
                    all += c;
                }
            } else {
                all = total[e];
            }
        }
        int scan = all;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, scan, d);
            if (lane >= d) scan += o;
        }
        if (lane == 31) chunk[warp] = scan;
        __syncthreads();
        int lower = carry, whole = 0;
        for (int k = 0; k < kOrderThreads / 32; ++k) {
            lower += k < warp ? chunk[k] : 0;
            whole += chunk[k];
        }
        carry += whole;
        if (e < E) {
            const int first = lower + scan - all;
            base[e] = first + before;
            if (rank == 0) a.offsets[e] = first;
        }
        __syncthreads();
    }
    if (rank == 0 && threadIdx.x == 0) a.offsets[E] = carry;
    if (warp < warps) {
        for (int e = lane; e < E; e += 32) mine[e] += base[e];
        __syncwarp();
        for (long long i0 = from; i0 < to; i0 += 32) {
            const long long i = i0 + lane;
            int id = i < to ? a.ids[i] : -1;
            if ((unsigned)id >= (unsigned)E) id = -1;
            const unsigned peers = __match_any_sync(0xffffffffu, id);
            const int rk = __popc(peers & ((1u << lane) - 1));
            int slot = -1;
            if (id >= 0) slot = mine[id] + rk;
            __syncwarp();
            if (id >= 0 && rk == 0) mine[id] += __popc(peers);
            __syncwarp();
            if (i < to) a.slots[i] = slot;
        }
    }
    if (ctas > 1) cluster_sync();   // no CTA leaves while another reads its counts
}

// ------------------------------------------------------------------ rows
constexpr int kThreads = 256;
constexpr int kSms = 152;
using Walk = RowWalk<kThreads>;
template <bool VEC>
constexpr int kMode = VEC ? kAligned : kShifted;

// A slot as a row of the experts' tensor, or -1.
__device__ __forceinline__ int slot_row(const MoveArgs& a, uint32_t token, int j) {
    const int s = a.slots[(uint64_t)token * a.choices + j];
    return (uint32_t)s < a.rows ? s : -1;
}

// out[slots[t, j], :] = x[t, :]: a warp loads a piece of a token's row once and stores it once per choice.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) k_dispatch(const MoveArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (Walk w(a.cols); w.row < a.tokens; w.next()) {
        Raw<BF16, kMode<VEC>> raw[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) raw[k].load(row_ptr(a.x, w.row), w.col + k * kSeg, a.cols, lane);
        for (int j = 0; j < a.choices; ++j) {
            const int s = slot_row(a, w.row, j);
            if (s < 0) continue;
#pragma unroll
            for (int k = 0; k < kUnroll; ++k)
                if (w.col + k * kSeg < a.cols)
                    seg_store_words<BF16, kMode<VEC>>(row_ptr(a.y, s), w.col + k * kSeg, a.cols, lane, raw[k].r);
        }
    }
}

// x[t, :] = sum over j of weights[t, j] y[slots[t, j], :], in fp32, j ascending.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) k_combine(const MoveArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (Walk w(a.cols); w.row < a.tokens; w.next()) {
        float acc[kUnroll][8] = {};
        for (int j = 0; j < a.choices; ++j) {
            const int s = slot_row(a, w.row, j);
            if (s < 0) continue;
            const float f = a.weights ? a.weights[(uint64_t)w.row * a.choices + j] : 1.f;
            Raw<BF16, kMode<VEC>> raw[kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) raw[k].load(row_ptr(a.y, s), w.col + k * kSeg, a.cols, lane);
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                float v[8];
                raw[k].get(v);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[k][i] = fmaf(f, v[i], acc[k][i]);
            }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (w.col + k * kSeg < a.cols)
                seg_store<BF16, kMode<VEC>>(row_ptr(a.x, w.row), w.col + k * kSeg, a.cols, lane, acc[k]);
    }
}

// dy[slots[t, j], :] = weights[t, j] x[t, :] and dweights[t, j] = x[t, :] . y[slots[t, j], :]: `span` warps
// share a token's columns, their sums meet in shared memory and are added in order.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) k_combine_backward(const MoveArgs a, int span) {
    __shared__ float part[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = kThreads / 32 / span, q = warp % span;
    pdl_trigger();
    pdl_wait();
    for (uint32_t t0 = blockIdx.x * per; t0 < a.tokens; t0 += gridDim.x * per) {
        const uint32_t t = t0 + warp / span;
        for (int j = 0; j < a.choices; ++j) {
            const int s = t < a.tokens ? slot_row(a, t, j) : -1;
            float sum = 0.f;
            if (s >= 0) {
                const float f = a.weights[(uint64_t)t * a.choices + j];
                for (int c0 = q * kSeg; c0 < a.cols; c0 += span * kSeg) {
                    Raw<BF16, kMode<VEC>> xr, yr;
                    float x[8], y[8];
                    xr.load(row_ptr(a.x, t), c0, a.cols, lane);
                    if (a.dweights) yr.load(row_ptr(a.y, s), c0, a.cols, lane);
                    xr.get(x);
                    if (a.dweights) {
                        yr.get(y);
#pragma unroll
                        for (int i = 0; i < 8; ++i) sum = fmaf(x[i], y[i], sum);
                    }
                    if (a.dy.p) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] *= f;
                        seg_store<BF16, kMode<VEC>>(row_ptr(a.dy, s), c0, a.cols, lane, x);
                    }
                }
            }
            if (a.dweights) {
#pragma unroll
                for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                if (lane == 0) part[warp] = sum;
                __syncthreads();
                if (q == 0 && lane == 0 && t < a.tokens) {
                    float all = part[warp];
                    for (int k = 1; k < span; ++k) all += part[warp + k];
                    a.dweights[(uint64_t)t * a.choices + j] = all;
                }
                __syncthreads();
            }
        }
    }
}

unsigned blocks_for(long long units, int fit) {
    const long long b = (units + kThreads / 32 - 1) / (kThreads / 32);
    return (unsigned)std::min<long long>(b, 4ll * fit * kSms);
}
unsigned row_blocks(const MoveArgs& a, int fit) {
    return blocks_for((long long)a.tokens * ((a.cols + Walk::kWidth - 1) / Walk::kWidth), fit);
}

}  // namespace

cudaError_t launch_expert_order(const OrderArgs& a, cudaStream_t s) {
    int warps = kOrderThreads / 32;
    while (warps * a.experts > kOrderCounts) warps /= 2;
    const int ctas = a.n <= 8192 ? 1 : 8;
    const size_t bytes = (size_t)(warps + 2) * a.experts * sizeof(int);
    // per call: an attribute of the current device
    const cudaError_t set =
        cudaFuncSetAttribute(k_expert_order, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (set != cudaSuccess) return set;
    return launch_pdl_cluster(k_expert_order, dim3(ctas), dim3(kOrderThreads), bytes, s, (unsigned)ctas, a, warps, ctas);
}

cudaError_t launch_expert_dispatch(const MoveArgs& a, bool bf16, bool vec, cudaStream_t s) {
    static void (*const k[4])(MoveArgs) = {k_dispatch<false, false>, k_dispatch<false, true>, k_dispatch<true, false>,
                                           k_dispatch<true, true>};
    return launch_pdl(k[(bf16 ? 2 : 0) + (vec ? 1 : 0)], dim3(row_blocks(a, 8)), dim3(kThreads), 0, s, a);
}
cudaError_t launch_expert_combine(const MoveArgs& a, bool bf16, bool vec, cudaStream_t s) {
    static void (*const k[4])(MoveArgs) = {k_combine<false, false>, k_combine<false, true>, k_combine<true, false>,
                                           k_combine<true, true>};
    return launch_pdl(k[(bf16 ? 2 : 0) + (vec ? 1 : 0)], dim3(row_blocks(a, 8)), dim3(kThreads), 0, s, a);
}
cudaError_t launch_expert_combine_backward(const MoveArgs& a, bool bf16, bool vec, cudaStream_t s) {
    static void (*const k[4])(MoveArgs, int) = {k_combine_backward<false, false>, k_combine_backward<false, true>,
                                                k_combine_backward<true, false>, k_combine_backward<true, true>};
    int span = 1;
    while (span < kThreads / 32 && span * kSeg < a.cols) span *= 2;
    return launch_pdl(k[(bf16 ? 2 : 0) + (vec ? 1 : 0)], dim3(blocks_for((long long)a.tokens * span, 8)), dim3(kThreads),
                      0, s, a, span);
}

}  // namespace muon
