// Activations to 8 bits and back, and SwiGLU with its inputs held in 8 bits.
//
// All four kernels read and write each value once (HBM-bound): one warp takes one segment
// of 256 values of a row at a time.
#include "act8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;

// Segments of this warp: row and first column of each, in steps of the launch's warps
// without a division per step.
struct SegWalk {
    long long row, drow;
    int seg, dseg, segs;
    __device__ __forceinline__ SegWalk(int cols) {
        segs = (cols + kSeg - 1) / kSeg;
        const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
        const long long n = (long long)gridDim.x * (kThreads / 32);
        row = w / segs, seg = (int)(w - row * segs);
        drow = n / segs, dseg = (int)(n - drow * segs);
    }
    __device__ __forceinline__ void next() {
        row += drow, seg += dseg;
        if (seg >= segs) seg -= segs, ++row;
    }
};

template <bool BF16>
__device__ __forceinline__ void* row_ptr(const Mat& m, long long row) {
    return static_cast<char*>(m.p) + row * m.ld * (BF16 ? 2 : 4);
}

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) k_act_pack(const PackArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (SegWalk w(a.cols); w.row < a.rows; w.next()) {
        float v[8];
        seg_load<BF16, VEC>(row_ptr<BF16>(a.x, w.row), w.seg * kSeg, a.cols, lane, v);
        seg_quant<VEC>(a.q, w.row, w.seg * kSeg, a.cols, lane, v);
    }
}

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) k_act_unpack(const PackArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (SegWalk w(a.cols); w.row < a.rows; w.next()) {
        float v[8];
        seg_dequant<VEC>(a.q, w.row, w.seg * kSeg, a.cols, lane, v);
        seg_store<BF16, VEC>(row_ptr<BF16>(a.x, w.row), w.seg * kSeg, a.cols, lane, v);
    }
}

__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) k_swiglu_forward(const SwigluArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (SegWalk w(a.cols); w.row < a.rows; w.next()) {
        const int c0 = w.seg * kSeg;
        float g[8], u[8], o[8];
        seg_load<BF16, VEC>(row_ptr<BF16>(a.gate, w.row), c0, a.cols, lane, g);
        seg_load<BF16, VEC>(row_ptr<BF16>(a.up, w.row), c0, a.cols, lane, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = g[j] * sigmoid(g[j]) * u[j];
        if (a.a.p) seg_store<BF16, VEC>(row_ptr<BF16>(a.a, w.row), c0, a.cols, lane, o);
        if (a.gate8.codes) seg_quant<VEC>(a.gate8, w.row, c0, a.cols, lane, g);
        if (a.up8.codes) seg_quant<VEC>(a.up8, w.row, c0, a.cols, lane, u);
        if (a.a8.codes) seg_quant<VEC>(a.a8, w.row, c0, a.cols, lane, o);
    }
}

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) k_swiglu_backward(const SwigluArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (SegWalk w(a.cols); w.row < a.rows; w.next()) {
        const int c0 = w.seg * kSeg;
        float g[8], u[8], d[8], o[8];
        seg_load<BF16, VEC>(row_ptr<BF16>(a.a, w.row), c0, a.cols, lane, d);
        seg_dequant<VEC>(a.gate8, w.row, c0, a.cols, lane, g);
        seg_dequant<VEC>(a.up8, w.row, c0, a.cols, lane, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = sigmoid(g[j]);
            const float silu = g[j] * s;
            o[j] = silu * u[j];
            g[j] = d[j] * u[j] * (s + silu * (1.f - s));   // dgate
            u[j] = d[j] * silu;                            // dup
        }
        seg_store<BF16, VEC>(row_ptr<BF16>(a.gate, w.row), c0, a.cols, lane, g);
        seg_store<BF16, VEC>(row_ptr<BF16>(a.up, w.row), c0, a.cols, lane, u);
        if (a.a8.codes) seg_quant<VEC>(a.a8, w.row, c0, a.cols, lane, o);
    }
}

// Blocks for all segments, at most `most` (the kernels stride over what is left).
unsigned seg_blocks(long long rows, int cols, long long most) {
    const long long segs = rows * ((cols + kSeg - 1) / kSeg);
    const long long b = (segs + kThreads / 32 - 1) / (kThreads / 32);
    return (unsigned)(b < most ? b : most);
}

template <typename Args>
cudaError_t launch(void (*const (&k)[4])(Args), const Args& a, bool bf16, bool vec, cudaStream_t s) {
    return launch_pdl(k[(bf16 ? 2 : 0) + (vec ? 1 : 0)], dim3(seg_blocks(a.rows, a.cols, 1 << 20)), dim3(kThreads), 0,
                      s, a);
}

}  // namespace

cudaError_t launch_act_pack(const PackArgs& a, bool bf16, bool vec, cudaStream_t s) {
    static void (*const k[4])(PackArgs) = {k_act_pack<false, false>, k_act_pack<false, true>, k_act_pack<true, false>,
                                           k_act_pack<true, true>};
    return launch(k, a, bf16, vec, s);
}
cudaError_t launch_act_unpack(const PackArgs& a, bool bf16, bool vec, cudaStream_t s) {
    static void (*const k[4])(PackArgs) = {k_act_unpack<false, false>, k_act_unpack<false, true>,
                                           k_act_unpack<true, false>, k_act_unpack<true, true>};
    return launch(k, a, bf16, vec, s);
}
cudaError_t launch_swiglu_forward(const SwigluArgs& a, bool bf16, bool vec, cudaStream_t s) {
    static void (*const k[4])(SwigluArgs) = {k_swiglu_forward<false, false>, k_swiglu_forward<false, true>,
                                             k_swiglu_forward<true, false>, k_swiglu_forward<true, true>};
    return launch(k, a, bf16, vec, s);
}
cudaError_t launch_swiglu_backward(const SwigluArgs& a, bool bf16, bool vec, cudaStream_t s) {
    static void (*const k[4])(SwigluArgs) = {k_swiglu_backward<false, false>, k_swiglu_backward<false, true>,
                                             k_swiglu_backward<true, false>, k_swiglu_backward<true, true>};
    return launch(k, a, bf16, vec, s);
}

}  // namespace muon
