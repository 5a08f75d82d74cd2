// Products of tokens with weights, one weight or one per expert over its own range of tokens:
// y = x W^T, and the gradient of its input, dx = dy W.
#include <algorithm>

#include "act8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kTile = 64, kStep = 16;

__device__ __forceinline__ void expert_range(const ProductArgs& a, int g, int* begin, int* end) {   // tokens < 2^31
    *begin = a.offsets ? min(max(a.offsets[g], 0), (int)a.tokens) : 0;
    *end = a.offsets ? min(max(a.offsets[g + 1], *begin), (int)a.tokens) : (int)a.tokens;
}

// A block computes 64 x 64 tiles on the CUDA cores.
__global__ void __launch_bounds__(256) k_product(const ProductArgs a) {
    __shared__ float xs[kStep][kTile + 1], ws[kStep][kTile + 1];
    __shared__ int unit[4];
    const int k = a.transposed ? a.m : a.n, out = a.transposed ? a.n : a.m, cols = (out + kTile - 1) / kTile;
    pdl_trigger();
    pdl_wait();
    for (long long u = blockIdx.x;; u += gridDim.x) {
        __syncthreads();
        if (threadIdx.x == 0) {
            long long left = u;
            unit[0] = -1;
            for (int g = 0; g < a.groups; ++g) {
                int b, e;
                expert_range(a, g, &b, &e);
                const long long tiles = (long long)((e - b + kTile - 1) / kTile) * cols;
                if (left < tiles) {
                    unit[0] = g, unit[1] = b + (int)(left / cols) * kTile, unit[2] = (int)(left % cols) * kTile, unit[3] = e;
                    break;
                }
                left -= tiles;
            }
        }
        __syncthreads();
        if (unit[0] < 0) return;
        const int t0 = unit[1], c0 = unit[2], end = unit[3];
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x);
        const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(a.weight) + (long long)unit[0] * a.m * a.n;
        float acc[4][4] = {};
        const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
        for (int k0 = 0; k0 < k; k0 += kStep) {
            for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
                const int r = i / kStep, kk = i % kStep;
                xs[kk][r] = t0 + r < end && k0 + kk < k ? __bfloat162float(x[(t0 + r) * a.ldx + k0 + kk]) : 0.f;
                if (!a.transposed)
                    ws[kk][r] = c0 + r < out && k0 + kk < k ? __bfloat162float(w[(long long)(c0 + r) * k + k0 + kk]) : 0.f;
            }
            if (a.transposed)
                for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
                    const int kk = i / kTile, r = i % kTile;
                    ws[kk][r] = c0 + r < out && k0 + kk < k ? __bfloat162float(w[(long long)(k0 + kk) * out + c0 + r]) : 0.f;
                }
            __syncthreads();
#pragma unroll
            for (int kk = 0; kk < kStep; ++kk)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[kk][ty * 4 + i], ws[kk][tx + 16 * j], acc[i][j]);
            __syncthreads();
        }
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y);
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int t = t0 + ty * 4 + i, c = c0 + tx + 16 * j;
                if (t < end && c < out) y[t * a.ldy + c] = __float2bfloat16_rn(acc[i][j]);
            }
    }
}

}  // namespace

cudaError_t launch_product(const ProductArgs& a, int sm_count, cudaStream_t s) {
    return launch_pdl(k_product, dim3(4 * sm_count), dim3(256), 0, s, a);
}

}  // namespace muon
