// The root-mean-square norm with the residual's addition, forward and backward.
//
// One block per row; warp w of the block holds segments w, w + W, ... of the row (256
// values each, eight per lane) in registers, so every value crosses HBM once each way.
#include "act8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kMaxThreads = 512;   // 128 registers per thread: up to eight segments per warp

template <bool BF16>
__device__ __forceinline__ void* row_ptr(const Mat& m, long long row) {
    return static_cast<char*>(m.p) + row * m.ld * (BF16 ? 2 : 4);
}

// Sum over the block, the same in every thread.  Fixed order: lanes by butterfly, warps in
// sequence.  `red` has room for one float per warp; two barriers allow its reuse.
__device__ __forceinline__ float block_sum(float x, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return x;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    float t = 0.f;
    for (int w = 0; w < warps; ++w) t += red[w];
    __syncthreads();
    return t;
}

// S segments per warp.
template <bool BF16, bool VEC, int S>
__global__ void __launch_bounds__(kMaxThreads) k_rmsnorm_forward(const NormArgs a) {
    __shared__ float red[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    pdl_trigger();
    pdl_wait();
    const long long row = blockIdx.x;
    float h[S][8];
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < S; ++k) {
        const int c0 = (warp + k * warps) * kSeg;
        seg_load<BF16, VEC>(row_ptr<BF16>(a.x, row), c0, a.cols, lane, h[k]);
        if (a.residual.p) {
            float r[8];
            seg_load<BF16, VEC>(row_ptr<BF16>(a.residual, row), c0, a.cols, lane, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[k][j] += r[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += h[k][j] * h[k][j];
        if (a.h.p && c0 < a.cols) seg_store<BF16, VEC>(row_ptr<BF16>(a.h, row), c0, a.cols, lane, h[k]);
    }
    const float rstd = 1.f / sqrtf(block_sum(sum, red) / (float)a.cols + a.eps);
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
        if (a.y.p) seg_store<BF16, VEC>(row_ptr<BF16>(a.y, row), c0, a.cols, lane, y);
        if (a.saved.codes) {
            if (a.saved_weighted)
                seg_quant<VEC>(a.saved, row, c0, a.cols, lane, y);
            else
                seg_quant<VEC>(a.saved, row, c0, a.cols, lane, h[k]);
        }
    }
}

// Blocks stride over the rows; each keeps its threads' columns of dweight in registers and
// leaves one row of partial sums, which k_dweight adds up in block order.
template <bool BF16, bool VEC, int S>
__global__ void __launch_bounds__(kMaxThreads) k_rmsnorm_backward(const NormBwdArgs a) {
    __shared__ float red[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    pdl_trigger();
    pdl_wait();
    float dw[S][8];
#pragma unroll
    for (int k = 0; k < S; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[k][j] = 0.f;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float rstd = a.rstd[row];
        float n[S][8], d[S][8];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < S; ++k) {
            const int c0 = (warp + k * warps) * kSeg;
            float w[8];
            seg_load<BF16, VEC>(row_ptr<BF16>(a.dy, row), c0, a.cols, lane, d[k]);
            if (a.saved.codes) {
                seg_dequant<VEC>(a.saved, row, c0, a.cols, lane, n[k]);
            } else {
                seg_load<BF16, VEC>(row_ptr<BF16>(a.h, row), c0, a.cols, lane, n[k]);
#pragma unroll
                for (int j = 0; j < 8; ++j) n[k][j] *= rstd;
            }
            seg_load<false, VEC>(a.weight, c0, a.cols, lane, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[k][j] += d[k][j] * n[k][j];
                d[k][j] *= w[j];
                sum += d[k][j] * n[k][j];
            }
        }
        if (!a.dx.p) continue;
        const float mean = block_sum(sum, red) / (float)a.cols;
#pragma unroll
        for (int k = 0; k < S; ++k) {
            const int c0 = (warp + k * warps) * kSeg;
            if (c0 >= a.cols) break;
            float r[8];
            if (a.dres.p) {
                seg_load<BF16, VEC>(row_ptr<BF16>(a.dres, row), c0, a.cols, lane, r);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) r[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] += rstd * (d[k][j] - n[k][j] * mean);
            seg_store<BF16, VEC>(row_ptr<BF16>(a.dx, row), c0, a.cols, lane, r);
        }
    }
    if (!a.partial) return;
    float* out = a.partial + (long long)blockIdx.x * a.cols;
#pragma unroll
    for (int k = 0; k < S; ++k) {
        const int c0 = (warp + k * warps) * kSeg;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = c0 + seg_col<VEC>(lane, j);
            if (c < a.cols) out[c] = dw[k][j];
        }
    }
}

// dweight (+)= sum of the blocks' partial rows, in block order.
__global__ void __launch_bounds__(256) k_dweight(const float* partial, int blocks, int cols, float* dweight,
                                                 int accumulate) {
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    pdl_trigger();
    pdl_wait();
    float s = 0.f;
    if (c < cols)
        for (int b = warp; b < blocks; b += 8) s += partial[(long long)b * cols + c];
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < cols) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += part[w][lane];
        dweight[c] = accumulate ? dweight[c] + t : t;
    }
}

// Warps per block and segments per warp for rows of `cols` values.
void norm_shape(int cols, int* warps, int* segs) {
    const int n = (cols + kSeg - 1) / kSeg;   // <= 128
    *segs = n <= 16 ? 1 : n <= 32 ? 2 : n <= 64 ? 4 : 8;
    *warps = (n + *segs - 1) / *segs;
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
    norm_shape(a.cols, &warps, &segs);
    return launch_pdl(k[segs == 8 ? 3 : segs >> 1][(bf16 ? 2 : 0) + (vec ? 1 : 0)], dim3((unsigned)a.rows), dim3(32 * warps), 0, s, a);
}

int rmsnorm_backward_blocks(long long rows, int cols, int sm_count) {
    int warps, segs;
    norm_shape(cols, &warps, &segs);
    long long b = (long long)sm_count * (64 / warps);
    if (b > kNormPartialFloats / cols) b = kNormPartialFloats / cols;
    return (int)(b < rows ? b : rows);
}

cudaError_t launch_rmsnorm_backward(const NormBwdArgs& a, bool bf16, bool vec, int sm_count, cudaStream_t s) {
    typedef void (*K)(NormBwdArgs);
    static const K k[4][4] = {{k_rmsnorm_backward<false, false, 1>, k_rmsnorm_backward<false, true, 1>,
                               k_rmsnorm_backward<true, false, 1>, k_rmsnorm_backward<true, true, 1>},
                              {k_rmsnorm_backward<false, false, 2>, k_rmsnorm_backward<false, true, 2>,
                               k_rmsnorm_backward<true, false, 2>, k_rmsnorm_backward<true, true, 2>},
                              {k_rmsnorm_backward<false, false, 4>, k_rmsnorm_backward<false, true, 4>,
                               k_rmsnorm_backward<true, false, 4>, k_rmsnorm_backward<true, true, 4>},
                              {k_rmsnorm_backward<false, false, 8>, k_rmsnorm_backward<false, true, 8>,
                               k_rmsnorm_backward<true, false, 8>, k_rmsnorm_backward<true, true, 8>}};
    int warps, segs;
    norm_shape(a.cols, &warps, &segs);
    const int blocks = rmsnorm_backward_blocks(a.rows, a.cols, sm_count);
    cudaError_t e = cudaSuccess;
    if (blocks > 0)
        e = launch_pdl(k[segs == 8 ? 3 : segs >> 1][(bf16 ? 2 : 0) + (vec ? 1 : 0)], dim3(blocks), dim3(32 * warps), 0, s, a);
    if (e == cudaSuccess && a.dweight)
        e = launch_pdl(k_dweight, dim3((a.cols + 31) / 32), dim3(256), 0, s, (const float*)a.partial, blocks, a.cols,
                       a.dweight, a.accumulate);
    return e;
}

}  // namespace muon
