// Parameter blocks and launch entry points of the layer-side operators: activations in
// 8 bits, the RMS norm, SwiGLU and the weight gradient.  Host entry points in acts.cu,
// kernels in act_elementwise.cu, rmsnorm.cu and wgrad.cu.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace muon {

constexpr int kActGroup = 32;   // values that share one scale
constexpr int kNormMaxCols = 32768;

enum ActFormat : int { kE4M3 = 0, kInt8 = 1 };

// An activation in 8 bits (muon_act8); codes null: not wanted.
struct Act8 {
    uint8_t* codes;
    uint8_t* scales;
    uint32_t ldq, lds;
    int format;
};

// One rows x cols tensor of fp32 or bf16, row pitch in bytes; p null: not wanted.  Rows and pitches
// are 32-bit numbers, so the address of a row is one multiplication with a 64-bit result.
struct Mat {
    void* p;
    uint32_t pitch;
};

struct PackArgs {
    Mat x;      // pack: input; unpack: output
    Act8 q;
    uint32_t rows;
    int cols;
};

struct SwigluArgs {
    Mat gate, up, a;     // backward: dgate, dup, da
    Act8 gate8, up8, a8;
    uint32_t rows;
    int cols;
};

struct NormArgs {
    Mat x, residual, h, y;
    const float* weight;
    float* rstd;
    Act8 saved;
    int saved_weighted;
    long long rows;
    int cols;
    float eps;
};

struct NormBwdArgs {
    Mat dy, h, dres, dx;
    const float* weight;
    const float* rstd;
    Act8 saved;          // codes null: xhat = rstd h
    float* partial;      // per block, cols sums of dy xhat; null: dweight not wanted
    float* dweight;
    int accumulate;
    int* status;
    long long rows;
    int cols;
};

struct WgradArgs {
    const void* dy;      // tokens x m bf16
    long long lddy;
    Act8 x;
    long long tokens;
    int m, n;
    const int* offsets;  // groups + 1, or null
    int groups;          // >= 1
    const float* col_scale;
    void* grad;
    int accumulate;
    int* status;
    float* partial;      // kMaxParts + kMaxPairs tiles of 256 x 256 sums
    int* counters;       // kMaxParts * 4 words, zero between calls
};
constexpr int kMaxParts = 240;   // parts of split tiles
constexpr int kMaxPairs = 76;    // CTA pairs, one tile of bf16 gradients' running sums each

// bf16: the dtype of the Mat operands; vec: every one of them (and ld) 16-byte aligned.
cudaError_t launch_act_pack(const PackArgs& a, bool bf16, bool vec, cudaStream_t s);
cudaError_t launch_act_unpack(const PackArgs& a, bool bf16, bool vec, cudaStream_t s);
cudaError_t launch_swiglu_forward(const SwigluArgs& a, bool bf16, bool vec, cudaStream_t s);
cudaError_t launch_swiglu_backward(const SwigluArgs& a, bool bf16, bool vec, cudaStream_t s);
cudaError_t launch_rmsnorm_forward(const NormArgs& a, bool bf16, bool vec, cudaStream_t s);
cudaError_t rmsnorm_prepare();   // once per device, before the first backward launch
// Blocks of the backward kernel for these sizes (its partial sums: blocks x cols floats).
int rmsnorm_backward_blocks(long long rows, int cols, int sm_count);
constexpr long long kNormPartialFloats = 8ll << 20;   // bound on blocks x cols
constexpr long long kPartialFloats = (kMaxParts + kMaxPairs) * 65536ll;   // of a grad plan, for either reduction
static_assert(kPartialFloats >= kNormPartialFloats, "one region serves both");
cudaError_t launch_rmsnorm_backward(const NormBwdArgs& a, bool bf16, bool vec, int sm_count, cudaStream_t s);
cudaError_t wgrad_prepare();   // once per device, before the first launch
cudaError_t launch_wgrad(const WgradArgs& a, bool bf16_grad, int sm_count, cudaStream_t s);

}  // namespace muon
