// Weight gradient from activations held in 8 bits: grad (+)= dy^T x diag(col_scale), one
// weight or one per expert over its own range of tokens.
#include <cuda_bf16.h>

#include "act8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kTileMN = 64, kStepK = 16;

// 64 x 64 outputs per block, four by four per thread, 16 tokens per step through shared
// memory in fp32.
template <bool BF16>
__global__ void __launch_bounds__(256) k_wgrad_simple(const WgradArgs a) {
    __shared__ float sy[kStepK][kTileMN], sx[kStepK][kTileMN];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const long long tiles_n = (a.n + kTileMN - 1) / kTileMN;
    const int m0 = (int)(blockIdx.x / tiles_n) * kTileMN, n0 = (int)(blockIdx.x % tiles_n) * kTileMN;
    const int g = blockIdx.y;
    pdl_trigger();
    pdl_wait();
    long long begin = 0, end = a.tokens;
    if (a.offsets) {
        begin = min(max((long long)a.offsets[g], 0ll), a.tokens);
        end = min(max((long long)a.offsets[g + 1], 0ll), a.tokens);
    }
    float acc[4][4] = {};
    for (long long t0 = begin; t0 < end; t0 += kStepK) {
        for (int i = tid; i < kStepK * kTileMN; i += 256) {
            const int k = i / kTileMN, c = i % kTileMN;
            const long long t = t0 + k;
            float y = 0.f, x = 0.f;
            if (t < end && m0 + c < a.m) y = load_one<true>(a.dy, t * a.lddy + m0 + c);
            if (t < end && n0 + c < a.n)
                x = act_number2(a.x.codes[t * a.x.ldq + n0 + c], a.x.format).x *
                    act_scale(a.x.scales[t * a.x.lds + ((n0 + c) >> 5)]);
            sy[k][c] = y;
            sx[k][c] = x;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kStepK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += sy[k][ty + 16 * i] * sx[k][tx + 16 * j];
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = m0 + ty + 16 * i, c = n0 + tx + 16 * j;
            if (r >= a.m || c >= a.n) continue;
            const long long e = ((long long)g * a.m + r) * a.n + c;
            float v = acc[i][j];
            if (a.col_scale) v *= a.col_scale[c];
            if (a.accumulate) v += load_one<BF16>(a.grad, e);
            store_one<BF16>(a.grad, e, v);
        }
}

}  // namespace

cudaError_t launch_wgrad(const WgradArgs& a, bool bf16_grad, cudaStream_t s) {
    const long long tiles = (long long)((a.m + kTileMN - 1) / kTileMN) * ((a.n + kTileMN - 1) / kTileMN);
    return launch_pdl(bf16_grad ? k_wgrad_simple<true> : k_wgrad_simple<false>, dim3((unsigned)tiles, a.groups),
                      dim3(256), 0, s, a);
}

}  // namespace muon
