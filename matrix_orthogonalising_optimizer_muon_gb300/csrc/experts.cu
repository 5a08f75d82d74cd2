// Tokens in their experts' order and back: the order itself (a stable counting sort of the
// chosen experts), the move of rows into it, their weighted sum per token, and its gradients.
#include <algorithm>
#include <atomic>

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
// a time, neighbours with the same expert by their rank among the warp's lanes.  What bounds it is latency:
// a warp's ids are loaded kBatch groups of 32 at a time and, when that is all it has, kept for pass 2
// (131072 ids of 128 experts: 13.1 to 13.5 us, 512 ids 6).
constexpr int kOrderThreads = 1024;
constexpr int kOrderCounts = 32768;   // counts in shared memory: warps x experts
constexpr int kBatch = 16;

__device__ __forceinline__ int remote_int(uint32_t local_saddr, uint32_t rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(local_saddr, rank)) : "memory");
    return v;
}

// Ids from .. of one batch, -1 for those that are no expert or at and beyond `to`.
__device__ __forceinline__ void load_ids(const OrderArgs& a, long long from, long long to, int lane,
                                         int (&id)[kBatch]) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) id[j] = from + 32 * j + lane < to ? a.ids[from + 32 * j + lane] : -1;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) id[j] = (unsigned)id[j] < (unsigned)a.experts ? id[j] : -1;
}

// Lanes of the warp with the same id < 2^bits: as many votes as bits (the instruction that matches all lanes
// takes a scheduler 200 cycles, 131072 ids 21 us).
__device__ __forceinline__ unsigned same_id(int id, int bits) {
    unsigned peers = 0xffffffffu;
    for (int b = 0; b < bits; ++b) {
        const bool one = id >> b & 1;
        const unsigned with = __ballot_sync(0xffffffffu, one);
        peers &= one ? with : ~with;
    }
    return peers;
}

// 2^lw warps count and deal; 2^lc CTAs in the cluster, at most 16.
__global__ void __launch_bounds__(kOrderThreads) k_expert_order(const OrderArgs a, int lw, int lc) {
    extern __shared__ int smem[];
    const int warps = 1 << lw, ctas = 1 << lc, bits = 32 - __clz(a.experts);   // ids 0 .. experts
    const int E = a.experts, row = warps + 1;   // an expert's counts lie side by side, odd rows against bank conflicts
    int* count = smem;                    // [E][row]
    int* total = smem + E * row;          // [E]: this CTA's counts
    int* base = total + E;                // [E]: the CTA's first slot
    __shared__ int chunk[kOrderThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = ctas > 1 ? (int)cluster_ctarank() : 0;
    for (int i = threadIdx.x; i < E * row; i += kOrderThreads) count[i] = 0;
    pdl_trigger();
    pdl_wait();

    // shares of 32 ids, as even as that allows
    const long long groups = (a.n + 31) / 32, parts = (long long)ctas * warps, w = (long long)rank * warps + warp;
    const long long from = warp < warps ? groups * w / parts * 32 : 0;
    const long long to = warp < warps ? min(groups * (w + 1) / parts * 32, a.n) : 0;
    int id[kBatch];
    if (from < to) load_ids(a, from, to, lane, id);
    __syncthreads();
    for (long long i = from; i < to; i += 32 * kBatch) {
        if (i > from) load_ids(a, i, to, lane, id);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (id[j] >= 0) atomicAdd(count + id[j] * row + warp, 1);
    }
    __syncthreads();
    // counts of earlier warps: `warps` lanes per expert
    const int sub = lane & (warps - 1);
    for (int e0 = warp << (5 - lw); e0 < E; e0 += kOrderThreads >> lw) {
        const int e = e0 + (lane >> lw), c = e < E ? count[e * row + sub] : 0;
        int sum = c;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, sum, d);
            if (sub >= d) sum += o;
        }
        if (e < E) {
            count[e * row + sub] = sum - c;
            if (sub == warps - 1) total[e] = sum;
        }
    }
    if (ctas > 1)
        cluster_sync();
    else
        __syncthreads();
    // counts of earlier CTAs, and of all: a lane per CTA, the sums to base and, for now, the first counts' row end
    for (int i0 = 0; i0 < E * ctas; i0 += kOrderThreads) {
        const int i = i0 + threadIdx.x, e = i >> lc, r = i & (ctas - 1);
        int all = 0;
        if (e < E) all = ctas > 1 ? remote_int(smem_u32(total + e), r) : total[e];
        int before = r < rank ? all : 0;
#pragma unroll
        for (int d = 1; d < 16; d *= 2) {
            const int x = __shfl_xor_sync(0xffffffffu, all, d), y = __shfl_xor_sync(0xffffffffu, before, d);
            if (d < ctas) all += x, before += y;
        }
        if (e < E && r == 0) base[e] = before, count[e * row + warps] = all;
    }
    __syncthreads();
    // smaller experts: a scan, kOrderThreads at a time
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += kOrderThreads) {
        const int e = e0 + threadIdx.x, all = e < E ? count[e * row + warps] : 0;
        int scan = all;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, scan, d);
            if (lane >= d) scan += o;
        }
        if (lane == 31) chunk[warp] = scan;
        __syncthreads();
        int lower = chunk[lane];   // every warp scans the warps' sums
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, lower, d);
            if (lane >= d) lower += o;
        }
        const int mine = warp ? __shfl_sync(0xffffffffu, lower, warp - 1) : 0;
        if (e < E) {
            const int first = carry + mine + scan - all;
            base[e] += first;
            if (rank == 0) a.offsets[e] = first;
        }
        carry += __shfl_sync(0xffffffffu, lower, 31);
        __syncthreads();
    }
    if (rank == 0 && threadIdx.x == 0) a.offsets[E] = carry;
    for (long long i = from; i < to; i += 32 * kBatch) {
        if (to - from > 32 * kBatch) load_ids(a, i, to, lane, id);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (i + 32 * j >= to) break;
            const unsigned peers = same_id(id[j] < 0 ? E : id[j], bits);
            const int rk = __popc(peers & ((1u << lane) - 1));
            int slot = -1;
            int* mine = count + id[j] * row + warp;
            if (id[j] >= 0) slot = base[id[j]] + *mine + rk;
            __syncwarp();
            if (id[j] >= 0 && rk == 0) *mine += __popc(peers);
            __syncwarp();
            if (i + 32 * j + lane < to) a.slots[i + 32 * j + lane] = slot;
        }
    }
    if (ctas > 1) cluster_sync();   // no CTA leaves while another reads its counts
}

// ------------------------------------------------------------------ rows
constexpr int kThreads = 256;
constexpr int kSms = 152;
using Walk = RowWalk<kThreads>;
// Rows that are not aligned: bf16 in shifted pieces, fp32 by value, whose loads are whole lines, too, and need no
// shifts (13384 x 6 rows of 453: 29 us by value, 61 shifted).
template <bool BF16, bool VEC>
constexpr int kMode = VEC ? kAligned : BF16 ? kShifted : kByValue;

// A slot as a row of the experts' tensor, or -1.
__device__ __forceinline__ int slot_row(const MoveArgs& a, uint32_t token, int j) {
    const int s = a.slots[(uint64_t)token * a.choices + j];
    return (uint32_t)s < a.rows ? s : -1;
}

// out[slots[t, j], :] = x[t, :]: a warp loads a piece of a token's row once and stores it once per choice (HBM-bound:
// 8192 x 4 rows of 3584 in bf16 44.1 us, 98 % of the copy rate; in fp32 117, 74 %).
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) k_dispatch(const MoveArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (Walk w(a.cols); w.row < a.tokens; w.next()) {
        Raw<BF16, kMode<BF16, VEC>> raw[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) raw[k].load(row_ptr(a.x, w.row), w.col + k * kSeg, a.cols, lane);
        for (int j = 0; j < a.choices; ++j) {
            const int s = slot_row(a, w.row, j);
            if (s < 0) continue;
#pragma unroll
            for (int k = 0; k < kUnroll; ++k)
                if (w.col + k * kSeg < a.cols) {
                    if constexpr (BF16 || VEC) {
                        seg_store_words<BF16, kMode<BF16, VEC>>(row_ptr(a.y, s), w.col + k * kSeg, a.cols, lane,
                                                                raw[k].r);
                    } else {
                        float v[8];
                        raw[k].get(v);
                        seg_store<BF16, kMode<BF16, VEC>>(row_ptr(a.y, s), w.col + k * kSeg, a.cols, lane, v);
                    }
                }
        }
    }
}

// Choices whose rows are on their way together: with one, the loads do not cover HBM's latency (backward, 8192 x 4
// rows of 3584 in bf16: 101 us, 81 with four, 96 % of the copy rate).
template <bool BF16>
constexpr int kTogether = BF16 ? 4 : 2;

// x[t, :] = sum over j of weights[t, j] y[slots[t, j], :], in fp32, j ascending.  HBM-bound: 8192 x 4 rows of 3584 in
// bf16 48.7 us (89 % of the copy rate), in fp32 84.7.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) k_combine(const MoveArgs a) {
    constexpr int kJ = kTogether<BF16>;
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (Walk w(a.cols); w.row < a.tokens; w.next()) {
        float acc[kUnroll][8] = {};
        for (int j0 = 0; j0 < a.choices; j0 += kJ) {
            int s[kJ];
            Raw<BF16, kMode<BF16, VEC>> raw[kJ][kUnroll];
#pragma unroll
            for (int j = 0; j < kJ; ++j) s[j] = j0 + j < a.choices ? slot_row(a, w.row, j0 + j) : -1;
#pragma unroll
            for (int j = 0; j < kJ; ++j)
#pragma unroll
                for (int k = 0; k < kUnroll; ++k)
                    if (s[j] >= 0) raw[j][k].load(row_ptr(a.y, s[j]), w.col + k * kSeg, a.cols, lane);
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                if (s[j] < 0) continue;
                const float f = a.weights ? a.weights[(uint64_t)w.row * a.choices + j0 + j] : 1.f;
#pragma unroll
                for (int k = 0; k < kUnroll; ++k) {
                    float v[8];
                    raw[j][k].get(v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[k][i] = fmaf(f, v[i], acc[k][i]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (w.col + k * kSeg < a.cols)
                seg_store<BF16, kMode<BF16, VEC>>(row_ptr(a.x, w.row), w.col + k * kSeg, a.cols, lane, acc[k]);
    }
}

// dy[slots[t, j], :] = weights[t, j] x[t, :] and dweights[t, j] = x[t, :] . y[slots[t, j], :]: `span` warps
// share a token's columns, their sums meet in shared memory and are added in order.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) k_combine_backward(const MoveArgs a, int span) {
    constexpr int kJ = kTogether<BF16>, kWarps = kThreads / 32;
    __shared__ float part[2][kWarps][kJ];   // in turn, so that one barrier a round is enough
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = kWarps / span, q = warp % span;
    int round = 0;
    pdl_trigger();
    pdl_wait();
    for (uint32_t t0 = blockIdx.x * per; t0 < a.tokens; t0 += gridDim.x * per) {
        const uint32_t t = t0 + warp / span;
        for (int j0 = 0; j0 < a.choices; j0 += kJ, round ^= 1) {
            int s[kJ];
            float f[kJ], sum[kJ] = {};
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                s[j] = t < a.tokens && j0 + j < a.choices ? slot_row(a, t, j0 + j) : -1;
                f[j] = s[j] >= 0 ? a.weights[(uint64_t)t * a.choices + j0 + j] : 0.f;
            }
            for (int c0 = q * kSeg; t < a.tokens && c0 < a.cols; c0 += span * kSeg) {
                Raw<BF16, kMode<BF16, VEC>> xr, yr[kJ];
                float x[8];
                xr.load(row_ptr(a.x, t), c0, a.cols, lane);
                if (a.dweights) {
#pragma unroll
                    for (int j = 0; j < kJ; ++j)
                        if (s[j] >= 0) yr[j].load(row_ptr(a.y, s[j]), c0, a.cols, lane);
                }
                xr.get(x);
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    if (s[j] < 0) continue;
                    float v[8];
                    if (a.dweights) {
                        yr[j].get(v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) sum[j] = fmaf(x[i], v[i], sum[j]);
                    }
                    if (a.dy.p) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = x[i] * f[j];
                        seg_store<BF16, kMode<BF16, VEC>>(row_ptr(a.dy, s[j]), c0, a.cols, lane, v);
                    }
                }
            }
            if (a.dweights) {
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
#pragma unroll
                    for (int d = 16; d > 0; d /= 2) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], d);
                    if (lane == j) part[round][warp][j] = sum[j];
                }
                __syncthreads();
                if (q == 0 && lane < kJ && t < a.tokens && j0 + lane < a.choices) {
                    float all = part[round][warp][lane];
                    for (int k = 1; k < span; ++k) all += part[round][warp + k][lane];
                    a.dweights[(uint64_t)t * a.choices + j0 + lane] = all;
                }
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

// Shared memory beyond 48 KB and clusters beyond eight CTAs are for attributes of the current device to allow: set per
// call, and the same by every call, as another thread may be between its own setting and its launch.
constexpr int kMostBytes = (8 + 3) * 4096 * (int)sizeof(int), kSixteenBytes = (32 + 3) * 1024 * (int)sizeof(int);
static_assert(kMostBytes >= kSixteenBytes && kMostBytes >= (16 + 3) * 2048 * (int)sizeof(int),
              "the most of any number of experts");
cudaError_t allow_bytes() {
    return cudaFuncSetAttribute(k_expert_order, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostBytes);
}
cudaError_t allow_sixteen() {
    return cudaFuncSetAttribute(k_expert_order, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}
// Whether the current device has room for sixteen CTAs of up to 1024 experts in a cluster, which only eight always
// have; asked once per device.
bool places_sixteen() {
    constexpr int kDevices = 64;
    static std::atomic<signed char> known[kDevices];   // 0: not asked yet
    int dev = 0, clusters = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return false;
    if (const signed char k = known[dev].load(std::memory_order_relaxed)) return k > 0;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(16), cfg.blockDim = dim3(kOrderThreads), cfg.dynamicSmemBytes = kSixteenBytes;
    cfg.attrs = attr, cfg.numAttrs = 1;
    cudaError_t e = allow_bytes();
    if (e == cudaSuccess) e = allow_sixteen();
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&clusters, k_expert_order, &cfg);
    if (e != cudaSuccess) (void)cudaGetLastError(), clusters = 0;
    known[dev].store(clusters > 0 ? 1 : -1, std::memory_order_relaxed);
    return clusters > 0;
}

}  // namespace

cudaError_t launch_expert_order(const OrderArgs& a, cudaStream_t s) {
    int lw = 5;
    while ((a.experts << lw) > kOrderCounts) --lw;
    // One CTA for the smallest (8192 ids of 256: 10.8 us, 8.1 with eight), the largest cluster there is for long ones,
    // whose ranks take longest, unless reading all CTAs' counts takes longer.  us with eight and with sixteen CTAs:
    //   ids     64 experts   128          256          512          1024         4096
    //   32768   8.4   8.5    9.0   9.9   10.2  13.1   12.6  19.8   16.8  28.9
    //   65536  10.6   9.6   11.4  11.0   13.0  14.5   15.6  21.1   20.1  30.4
    //  131072  15.2  11.9   16.3  13.5   18.1  17.1   21.3  24.1   26.2  33.6   51    84
    //  262144  27.0  16.6   28.4  18.3   31.2  22.4   35.3  29.8   40.9  39.8
    // 1048576  91.5  50.1   96.2  53.5    104  60.0    114  70.2    124  82.6
    const bool is_long = a.n >= 256ll * (a.experts + 128) && a.experts <= 1024;
    const int lc = a.n <= 2048 ? 0 : is_long && places_sixteen() ? 4 : 3;
    const size_t bytes = (size_t)((1 << lw) + 3) * a.experts * sizeof(int);
    cudaError_t e = bytes > 48 * 1024 ? allow_bytes() : cudaSuccess;
    if (e == cudaSuccess && lc == 4) e = allow_sixteen();
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(k_expert_order, dim3(1 << lc), dim3(kOrderThreads), bytes, s, 1u << lc, a, lw, lc);
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
    return launch_pdl(k[(bf16 ? 2 : 0) + (vec ? 1 : 0)], dim3(blocks_for((long long)a.tokens * span, 8)),
                      dim3(kThreads), 0, s, a, span);
}

}  // namespace muon
