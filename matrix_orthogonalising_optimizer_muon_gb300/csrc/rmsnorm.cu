// The root-mean-square norm with the residual's addition, forward and backward.
//
// One block per row; warp w of the block holds segments w, w + W, ... of the row (256
// values each, eight per lane) in registers, so every value crosses HBM once each way, which
// bounds both passes.  Measured at 16384 x 3584 bf16 with the residual: forward 82 us for 530 MB
// (6.5 TB/s, 96 % of the measured copy rate), backward from 8 bits 76 us for 413 MB (5.4 TB/s, 80 %:
// 4 us of it are the sum of the blocks' dweight rows, the rest waits on each row's barrier).
#include <algorithm>
#include <type_traits>

#include "act8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kMaxThreads = 512;   // 128 registers per thread: up to eight segments per warp
// Least segments per warp.  Forward: with two a row's block is small enough for many to share an SM,
// one reducing while others load (16384 x 3584 bf16: 82 us, and 88 with the two segments' loads one
// after the other; there 99 with one, 97 with four).
constexpr int kFwdSegs = 2, kBwdSegs = 1;
// Backward: warps per SM, as many as 64 registers allow.  With 28, rows of 15 segments have one block
// per SM instead of two (16384 x 3585 bf16: 254 us, 135 with 32; 65536 x 1024: 97 us, 88 with 32;
// 125 and 83 since).
// With 80 registers fewer fit: 16384 x 3584 took 107 us, 80 with 64.
constexpr int kBwdWarps = 32;
constexpr int kRingRoom = 216 * 1024;   // backward: shared memory of an SM for rows on their way

// Sum over the block, the same in every thread, in a fixed order: lanes by butterfly, warps in
// sequence.  `red` has room for one float per warp; consecutive calls alternate between two
// such rows, so one barrier each is enough.
template <bool ALWAYS>   // a barrier even for a single warp
__device__ __forceinline__ float block_sum(float x, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    const int warps = blockDim.x >> 5;
    if (warps == 1) {
        if (ALWAYS) __syncthreads();
        return x;
    }
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    // 16 warps at most: four 16-byte reads, absent warps read as the zeros stored at the start
    const float4* r = reinterpret_cast<const float4*>(red);
    const float4 a = r[0], b = r[1], c = r[2], d = r[3];
    return (((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w))) +
           (((c.x + c.y) + (c.z + c.w)) + ((d.x + d.y) + (d.z + d.w)));
}

// 1 / sqrt(sum / cols + eps) to about half an ulp: the mean in two floats, then one Newton step with
// its residual 1 - v y^2 in two floats.  The rounding of each step alone would move a few more
// 8-bit codes across a rounding boundary.
__device__ __forceinline__ float inverse_rms(float sum, float cols, float eps) {
    const float inv = 1.f / cols, inv_lo = fmaf(-inv, cols, 1.f) * inv;   // 1 / cols
    const float q = sum * inv, q_lo = fmaf(sum, inv, -q) + sum * inv_lo;
    const float v = q + eps, b = v - q, v_lo = (q - (v - b)) + (eps - b) + q_lo;
    const float y = rsqrtf(v);
    const float h = y * y, h_lo = fmaf(y, y, -h);
    const float res = fmaf(-v, h, 1.f) - fmaf(v, h_lo, v_lo * h);
    return isfinite(res) ? fmaf(0.5f * y, res, y) : y;   // sum infinite or NaN
}

// S segments per warp.
template <bool BF16, bool VEC, int S>
__global__ void __launch_bounds__(kMaxThreads) k_rmsnorm_forward(const NormArgs a) {
    __shared__ __align__(16) float red[16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    pdl_trigger();
    if (threadIdx.x < 16) red[threadIdx.x] = 0.f;
    __syncthreads();
    pdl_wait();
    const uint32_t row = blockIdx.x;
    float h[S][8];
    float sum = 0.f;
    constexpr int P = VEC && S > 1 ? 2 : 1;   // segments whose loads are in flight together
#pragma unroll
    for (int k0 = 0; k0 < S; k0 += P) {
        Raw<BF16, VEC> x[P], r[P];
        auto load = [&](auto full) {
#pragma unroll
            for (int k = 0; k < P; ++k) {
                const int c0 = (warp + (k0 + k) * warps) * kSeg;
                x[k].template load<full.value>(row_ptr(a.x, row), c0, a.cols, lane);
                if (a.residual.p) r[k].template load<full.value>(row_ptr(a.residual, row), c0, a.cols, lane);
            }
        };
        if (VEC && (warp + (k0 + P - 1) * warps + 1) * kSeg <= a.cols)
            load(std::true_type{});
        else
            load(std::false_type{});
#pragma unroll
        for (int k = 0; k < P; ++k) {
            const int c0 = (warp + (k0 + k) * warps) * kSeg;
            float(&v)[8] = h[k0 + k];
            x[k].get(v);
            if (a.residual.p) {
                float b[8];
                r[k].get(b);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += b[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += v[j] * v[j];
            if (a.h.p && c0 < a.cols) seg_store<BF16, VEC>(row_ptr(a.h, row), c0, a.cols, lane, v);
        }
    }
    const float rstd = inverse_rms(block_sum<false>(sum, red), (float)a.cols, a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    if (!a.y.p && !a.saved.codes) return;
#pragma unroll
    for (int k = 0; k < S; ++k) {
        const int c0 = (warp + k * warps) * kSeg;
        if (c0 >= a.cols) break;
        float w[8], y[8];
        seg_load<false, VEC>(a.weight, c0, a.cols, lane, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            h[k][j] *= rstd;
            y[j] = h[k][j] * w[j];
        }
        if (a.y.p) seg_store<BF16, VEC>(row_ptr(a.y, row), c0, a.cols, lane, y);
        if (a.saved.codes) {
            if (a.saved_weighted)
                seg_quant<VEC>(a.saved, row, c0, a.cols, lane, y);
            else
                seg_quant<VEC>(a.saved, row, c0, a.cols, lane, h[k]);
        }
    }
}

// Where one row's operands lie: in HBM, or in a slot of the ring.
struct RowAt {
    const void *dy, *h, *dres;
    const uint8_t *codes, *scales;
};
// A thread's operands of segments warp + k0 warps, warp + (k0 + 1) warps, ... of a row, as loaded.
template <bool BF16, bool VEC, int N>
struct RowIn {
    Raw<BF16, VEC> dy[N], dres[N];
    union Xhat {
        Raw<BF16, VEC> h;
        Raw8<VEC> q;
        __device__ Xhat() {}
    } x[N];
    __device__ __forceinline__ void load(const NormBwdArgs& a, const RowAt& at, int k0, int warp, int warps, int lane,
                                         bool with_dres) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int c0 = (warp + (k0 + k) * warps) * kSeg;
            dy[k].load(at.dy, c0, a.cols, lane);
            if (a.saved.codes)
                x[k].q.load(at.codes, at.scales, c0, a.cols, lane);
            else
                x[k].h.load(at.h, c0, a.cols, lane);
            if (with_dres) dres[k].load(at.dres, c0, a.cols, lane);
        }
    }
    // Segment k's dy and normalised input.
    __device__ __forceinline__ void get(const NormBwdArgs& a, float rstd, int k, float (&d)[8], float (&n)[8]) const {
        dy[k].get(d);
        if (a.saved.codes) {
            x[k].q.get(a.saved.format, n);
        } else {
            x[k].h.get(n);
#pragma unroll
            for (int j = 0; j < 8; ++j) n[j] *= rstd;
        }
    }
};

// Shared memory of the ring: rows as they lie in HBM, in whole 16-byte pieces.  A row that is not
// aligned keeps its offset within its first piece; every piece copied holds some of the row.
struct RingShape {
    int dy, x, scales, dres, slot;   // room of one row's parts, and of a slot
    int depth;                       // slots; 0: the rows are read directly
};
constexpr int kRingMost = 4;

// The gradients.  Blocks stride over the rows; each keeps its threads' columns of dweight in
// registers and leaves one row of partial sums, which k_dweight adds up in block order.
// RING (rows that fit): the next rows are on their way into shared memory by
// bulk copies while one is reduced, so that HBM stays busy across the reduction's barrier
// with registers for one row only.
template <bool BF16, bool VEC, int S, bool RING>
__global__ void __launch_bounds__(kMaxThreads, S == 1 ? 2 : 1)
    k_rmsnorm_backward(const NormBwdArgs a, const RingShape ring) {
    extern __shared__ __align__(128) uint8_t slots[];
    __shared__ __align__(16) float red[2][16];
    __shared__ uint64_t full[kRingMost];
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    pdl_trigger();
    if (threadIdx.x < 32) red[threadIdx.x >> 4][threadIdx.x & 15] = 0.f;
    if (RING && threadIdx.x == 0) {
        for (int s = 0; s < ring.depth; ++s) mbar_init(full + s, 1);
        abort_word = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    const uint32_t first = blockIdx.x, stride = gridDim.x, rows = (uint32_t)a.rows;   // below 2^31
    constexpr int kSize = BF16 ? 2 : 4;
    auto offset = [](const void* p) { return VEC ? 0 : (int)(reinterpret_cast<uintptr_t>(p) & 15); };
    auto pieces = [&](const void* p) { return (offset(p) + a.cols * kSize + 15) & ~15; };
    auto fetch = [&](uint32_t row, int s) {   // one thread
        uint8_t* to = slots + s * ring.slot;
        const char *y = row_ptr(a.dy, row), *h = row_ptr(a.h, row),
                   *r = row_ptr(a.dres, row);
        const int ny = pieces(y), nx = a.saved.codes ? ring.x : pieces(h), nr = a.dres.p ? pieces(r) : 0;
        mbar_arrive_expect_tx(full + s, ny + nx + ring.scales + nr);
        bulk_load(to, y - offset(y), ny, full + s);
        if (a.saved.codes) {
            bulk_load(to + ring.dy, a.saved.codes + (uint64_t)row * a.saved.ldq, nx, full + s);
            bulk_load(to + ring.dy + ring.x, a.saved.scales + (uint64_t)row * a.saved.lds, ring.scales, full + s);
        } else {
            bulk_load(to + ring.dy, h - offset(h), nx, full + s);
        }
        if (nr) bulk_load(to + ring.dy + ring.x + ring.scales, r - offset(r), nr, full + s);
    };
    if (RING && threadIdx.x == 0)
        for (int s = 0; s < ring.depth && first + s * stride < rows; ++s) fetch(first + s * stride, s);

    // KEEP: the row's operands stay in registers between the sum and dx.  Else, where they would not
    // fit, they are read again, one segment at a time (4096 x 16383 bf16: 348 us, 698 kept; 1024 x
    // 32768 fp32: 191, 244 kept; but 4096 x 16384 bf16: 136 kept, 240 read again).
    constexpr bool KEEP = S <= 2 || (VEC && (BF16 || S == 4));
    constexpr int N = KEEP ? S : 1;   // segments in registers
    float dw[S][8];
#pragma unroll
    for (int k = 0; k < S; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[k][j] = 0.f;
    // one segment per warp leaves registers for its weights (16384 x 3584 from h: 77 us, 83 without)
    float wk[8];
    if constexpr (S == 1) seg_load<false, VEC>(a.weight, warp * kSeg, a.cols, lane, wk);
    int slot = 0, phase = 0, turn = 0;
    for (uint32_t row = first; row < rows; row += stride, turn ^= 1) {
        const float rstd = a.rstd[row];
        RowAt at{row_ptr(a.dy, row), row_ptr(a.h, row), row_ptr(a.dres, row),
                 a.saved.codes + (uint64_t)row * a.saved.ldq, a.saved.scales + (uint64_t)row * a.saved.lds};
        if (RING) {
            // a wait that runs out raises the flag and the status word; later waits then return at once
            mbar_wait(full + slot, phase, abort_flag, a.status, kStatusTimeoutProducer);
            const uint8_t* p = slots + slot * ring.slot;
            const uint8_t *x = p + ring.dy, *r = x + ring.x + ring.scales;
            at = RowAt{p + offset(at.dy), x + offset(at.h), r + offset(at.dres), x, x + ring.x};
        }
        RowIn<BF16, VEC, N> in;
        float n[N][8], d[N][8];
        float sum = 0.f;
#pragma unroll
        for (int k0 = 0; k0 < S; k0 += N) {
            in.load(a, at, k0, warp, warps, lane, KEEP && a.dres.p);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                in.get(a, rstd, k, d[k], n[k]);
                if constexpr (S > 1) seg_load<false, VEC>(a.weight, (warp + (k0 + k) * warps) * kSeg, a.cols, lane, wk);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dw[k0 + k][j] += d[k][j] * n[k][j];
                    d[k][j] *= wk[j];
                    sum += d[k][j] * n[k][j];
                }
            }
        }
        const float mean = block_sum<true>(sum, red[turn]) / (float)a.cols;
        // every thread has read the slot once block_sum's barrier, or with !KEEP the one below, is passed
        auto refill = [&] {
            if (threadIdx.x == 0 && row + ring.depth * stride < rows) fetch(row + ring.depth * stride, slot);
            if (++slot == ring.depth) slot = 0, phase ^= 1;
        };
        if (RING && KEEP) refill();
        if (a.dx.p) {
#pragma unroll
            for (int k0 = 0; k0 < S; k0 += N) {
                if (!KEEP) in.load(a, at, k0, warp, warps, lane, a.dres.p);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const int c0 = (warp + (k0 + k) * warps) * kSeg;
                    if (c0 >= a.cols) break;
                    if constexpr (!KEEP) {
                        in.get(a, rstd, k, d[k], n[k]);
                        seg_load<false, VEC>(a.weight, c0, a.cols, lane, wk);
#pragma unroll
                        for (int j = 0; j < 8; ++j) d[k][j] *= wk[j];
                    }
                    float r[8];
                    if (a.dres.p) {
                        in.dres[k].get(r);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) r[j] = 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) r[j] += rstd * (d[k][j] - n[k][j] * mean);
                    seg_store<BF16, VEC>(row_ptr(a.dx, row), c0, a.cols, lane, r);
                }
            }
        }
        if (RING && !KEEP) {
            __syncthreads();
            refill();
        }
    }
    if (RING && threadIdx.x == 0 && *abort_flag) {   // give copies still in flight time to land
        const unsigned long long t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
    }
    if (!a.partial) return;
    float* out = a.partial + (long long)blockIdx.x * a.cols;
#pragma unroll
    for (int k = 0; k < S; ++k) {
        const int c0 = (warp + k * warps) * kSeg;
        if (c0 < a.cols) seg_store<false, VEC ? kShifted : kByValue>(out, c0, a.cols, lane, dw[k]);
    }
}

// dweight (+)= sum of the blocks' partial rows: warp w of a block takes rows w, w + 32, ... of 32
// columns, then the warps' sums are added in order.
__global__ void __launch_bounds__(1024) k_dweight(const float* partial, int blocks, int cols, float* dweight,
                                                  int accumulate) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    pdl_trigger();
    pdl_wait();
    float s = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int b = warp; b < blocks; b += 32) s += partial[(long long)b * cols + c];
    }
    part[warp][lane] = s;
    __syncthreads();
    s = part[lane][warp];   // warp w: column w of the 32
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int col = blockIdx.x * 32 + warp;
    if (lane == 0 && col < cols) dweight[col] = accumulate ? dweight[col] + s : s;
}

// Segments per warp (1, 2, 4 or 8, at least `least` where the row has two warps' worth) and
// warps per block for rows of `cols` values.
void norm_shape(int cols, int least, int* warps, int* segs) {
    const int n = (cols + kSeg - 1) / kSeg;   // <= 128
    int s = n <= 16 ? 1 : n <= 32 ? 2 : n <= 64 ? 4 : 8;
    if (n >= 2 * least && s < least) s = least;
    *segs = s;
    *warps = (n + s - 1) / s;
}

typedef void (*BackwardKernel)(NormBwdArgs, RingShape);
template <int S>
BackwardKernel pick_backward(bool bf16, bool vec, bool ring) {
    if (!vec) {
        if (!ring) return bf16 ? k_rmsnorm_backward<true, false, S, false> : k_rmsnorm_backward<false, false, S, false>;
        return bf16 ? k_rmsnorm_backward<true, false, S, true> : k_rmsnorm_backward<false, false, S, true>;
    }
    if (!ring) return bf16 ? k_rmsnorm_backward<true, true, S, false> : k_rmsnorm_backward<false, true, S, false>;
    return bf16 ? k_rmsnorm_backward<true, true, S, true> : k_rmsnorm_backward<false, true, S, true>;
}
BackwardKernel pick_backward(bool bf16, bool vec, int segs, bool ring) {
    return segs == 1   ? pick_backward<1>(bf16, vec, ring)
           : segs == 2 ? pick_backward<2>(bf16, vec, ring)
           : segs == 4 ? pick_backward<4>(bf16, vec, ring)
                       : pick_backward<8>(bf16, vec, ring);
}
cudaError_t for_each_ring_kernel() {
    cudaError_t e = cudaSuccess;
    for (int segs = 1; segs <= 8; segs *= 2)
        for (int i = 0; i < 4 && e == cudaSuccess; ++i)
            e = cudaFuncSetAttribute(pick_backward(i & 1, i >> 1, segs, true), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kRingRoom);
    return e;
}

}  // namespace

cudaError_t launch_rmsnorm_forward(const NormArgs& a, bool bf16, bool vec, cudaStream_t s) {
    typedef void (*K)(NormArgs);
    static const K k[4][4] = {{k_rmsnorm_forward<false, false, 1>, k_rmsnorm_forward<false, true, 1>,
                               k_rmsnorm_forward<true, false, 1>, k_rmsnorm_forward<true, true, 1>},
                              {k_rmsnorm_forward<false, false, 2>, k_rmsnorm_forward<false, true, 2>,
                               k_rmsnorm_forward<true, false, 2>, k_rmsnorm_forward<true, true, 2>},
                              {k_rmsnorm_forward<false, false, 4>, k_rmsnorm_forward<false, true, 4>,
                               k_rmsnorm_forward<true, false, 4>, k_rmsnorm_forward<true, true, 4>},
                              {k_rmsnorm_forward<false, false, 8>, k_rmsnorm_forward<false, true, 8>,
                               k_rmsnorm_forward<true, false, 8>, k_rmsnorm_forward<true, true, 8>}};
    int warps, segs;
    norm_shape(a.cols, kFwdSegs, &warps, &segs);
    return launch_pdl(k[segs == 8 ? 3 : segs >> 1][(bf16 ? 2 : 0) + (vec ? 1 : 0)], dim3((unsigned)a.rows),
                      dim3(32 * warps), 0, s, a);
}

int rmsnorm_backward_blocks(long long rows, int cols, int sm_count) {
    int warps, segs;
    norm_shape(cols, kBwdSegs, &warps, &segs);
    long long b = (long long)sm_count * std::max(kBwdWarps / warps, 1);
    if (b > kNormPartialFloats / cols) b = kNormPartialFloats / cols;
    return (int)(b < rows ? b : rows);
}

cudaError_t rmsnorm_prepare() { return for_each_ring_kernel(); }

cudaError_t launch_rmsnorm_backward(const NormBwdArgs& a, bool bf16, bool vec, int sm_count, cudaStream_t s) {
    int warps, segs;
    norm_shape(a.cols, kBwdSegs, &warps, &segs);
    const int blocks = rmsnorm_backward_blocks(a.rows, a.cols, sm_count);
    cudaError_t e = cudaSuccess;
    if (blocks > 0) {
        RingShape r{};
        auto up16 = [](int n) { return (n + 15) / 16 * 16; };
        const int esz = bf16 ? 2 : 4;
        r.dy = up16(a.cols * esz) + (vec ? 0 : 16);
        r.x = a.saved.codes ? up16(a.cols) : r.dy;
        r.scales = a.saved.codes ? up16((a.cols + kActGroup - 1) / kActGroup) : 0;
        r.dres = a.dres.p ? r.dy : 0;
        r.slot = r.dy + r.x + r.scales + r.dres;
        // the blocks of an SM share its shared memory; rows of which two fit a block's share use the ring
        const int room = kRingRoom / std::max(kBwdWarps / warps, 1) - 1024;
        r.depth = std::min(room / r.slot, kRingMost);
        if (r.depth < 2) r.depth = 0;
        e = launch_pdl(pick_backward(bf16, vec, segs, r.depth > 0), dim3(blocks), dim3(32 * warps),
                       (size_t)r.depth * r.slot, s, a, r);
    }
    if (e == cudaSuccess && a.dweight)
        e = launch_pdl(k_dweight, dim3((a.cols + 31) / 32), dim3(1024), 0, s, (const float*)a.partial, blocks, a.cols,
                       a.dweight, a.accumulate);
    return e;
}

}  // namespace muon
