// Parameter blocks and launch entry points of the layer-side operators: activations in
// 8 bits, the RMS norm, SwiGLU, the weight gradient and the other two products of a weight, and
// tokens in their experts' order.  Host entry points in acts.cu, kernels in act_elementwise.cu,
// rmsnorm.cu, wgrad.cu, product.cu and experts.cu; lists of gradients in grads.h.
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
    int* counters;       // kCounters words, zero between calls
};
constexpr int kMaxParts = 240;   // parts of split tiles
constexpr int kCounters = 1280;  // of parts that have arrived: 4 per part of a split tile, or 16 per CTA pair
constexpr int kMaxPairs = 76;    // CTA pairs, one tile of bf16 gradients' running sums each

// The experts' order of tokens.
struct OrderArgs {
    const int* ids;      // n of them, tokens x choices
    long long n;
    int experts;
    int* offsets;        // experts + 1
    int* slots;          // n
};

// Rows moved between the tokens' order and the experts'.
struct MoveArgs {
    Mat x;               // the tokens' side
    Mat y;               // the experts' side
    Mat dy;              // combine backward: its gradient, or null
    const int* slots;    // tokens x choices
    const float* weights;   // tokens x choices, or null: ones
    float* dweights;     // combine backward, or null
    uint32_t tokens, rows;  // rows of y
    int choices, cols;
};

struct ProductArgs {
    const void* x;       // tokens x k bf16, row pitch ldx elements
    long long ldx;
    const void* weight;  // groups x m x n bf16, dense
    void* y;             // tokens x out bf16, row pitch ldy
    long long ldy;
    int first;           // of these tokens among those that offsets counts
    long long tokens;
    int m, n;
    bool transposed;     // y = x W (k = m, out = n), else y = x W^T (k = n, out = m)
    const int* offsets;  // groups + 1, or null
    int groups;          // >= 1
    int* status;
    float* partial;      // kJoinFloats
    int* counters;
    void* aligned;       // room for rows that are not
    long long room;      // its bytes, a multiple of 256
};
constexpr long long kJoinFloats = 2 * kMaxPairs * 8 * 8192ll;   // two parts of a tile per CTA pair

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
// Rows that the products copy take what their parts leave of that region, and, at its end, what the plan has for them
// alone: a plan that is not asked for less has room for 2^28 bytes in all.
constexpr long long kSharedRoom = (kPartialFloats - kJoinFloats) * 4, kAlignedBytes = (1ll << 28) - kSharedRoom;
constexpr long long kMostAligned = 1ll << 34;   // 16-byte pieces of it are counted in 31 bits
static_assert(kSharedRoom > 0 && kSharedRoom % 256 == 0 && kAlignedBytes > 0, "the room's place");
cudaError_t launch_rmsnorm_backward(const NormBwdArgs& a, bool bf16, bool vec, int sm_count, cudaStream_t s);
cudaError_t wgrad_prepare();   // once per device, before the first launch
cudaError_t launch_expert_order(const OrderArgs& a, cudaStream_t s);
cudaError_t launch_expert_dispatch(const MoveArgs& a, bool bf16, bool vec, cudaStream_t s);
cudaError_t launch_expert_combine(const MoveArgs& a, bool bf16, bool vec, cudaStream_t s);
cudaError_t launch_expert_combine_backward(const MoveArgs& a, bool bf16, bool vec, cudaStream_t s);
cudaError_t product_prepare();   // once per device, before the first launch
bool product_fits(const ProductArgs& a);   // where rows have to be copied, the room holds the least pieces
cudaError_t launch_product(const ProductArgs& a, int sm_count, cudaStream_t s);
cudaError_t launch_wgrad(const WgradArgs& a, bool bf16_grad, int sm_count, cudaStream_t s);

}  // namespace muon
