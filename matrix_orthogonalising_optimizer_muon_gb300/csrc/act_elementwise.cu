// Activations to 8 bits and back, and SwiGLU with its inputs held in 8 bits.
//
// All four kernels read and write each value once (HBM-bound).  A warp takes units of kUnroll
// neighbouring segments of 256 values of a row, all loads before the first store.
#include "act8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 152 * 16;   // two full SMs' worth of warps on each SM
// Segments in flight per warp (SwiGLU forward, 8192 x 18944 bf16: 222 us; 250 with one, 277 with
// four, whose registers leave too few warps).
constexpr int kUnroll = 2;

// Units of this warp: row and first column of each, in steps of the launch's warps without a
// division per step.
struct Walk {
    long long row, drow;
    int col, dcol, width;
    __device__ __forceinline__ Walk(int cols) {
        const int units = (cols + kUnroll * kSeg - 1) / (kUnroll * kSeg);
        const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
        const long long n = (long long)gridDim.x * (kThreads / 32);
        row = w / units, col = (int)(w - row * units) * (kUnroll * kSeg);
        drow = n / units, dcol = (int)(n - drow * units) * (kUnroll * kSeg);
        width = units * (kUnroll * kSeg);
    }
    __device__ __forceinline__ void next() {
        row += drow, col += dcol;
        if (col >= width) col -= width, ++row;
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
    for (Walk w(a.cols); w.row < a.rows; w.next()) {
        const void* x = row_ptr<BF16>(a.x, w.row);
        Raw<BF16, VEC> raw[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) raw[k].load(x, w.col + k * kSeg, a.cols, lane);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            float v[8];
            raw[k].get(v);
            seg_quant<VEC>(a.q, w.row, w.col + k * kSeg, a.cols, lane, v);
        }
    }
}

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) k_act_unpack(const PackArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (Walk w(a.cols); w.row < a.rows; w.next()) {
        void* y = row_ptr<BF16>(a.x, w.row);
        Raw8<VEC> raw[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) raw[k].load(a.q, w.row, w.col + k * kSeg, a.cols, lane);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            float v[8];
            raw[k].get(a.q.format, v);
            seg_store<BF16, VEC>(y, w.col + k * kSeg, a.cols, lane, v);
        }
    }
}

// 1 / (1 + e^-z); the quotient by the approximate reciprocal (1 ulp; 0 where e^-z overflows).
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + expf(-z)); }

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) k_swiglu_forward(const SwigluArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (Walk w(a.cols); w.row < a.rows; w.next()) {
        const void *gate = row_ptr<BF16>(a.gate, w.row), *up = row_ptr<BF16>(a.up, w.row);
        Raw<BF16, VEC> gr[kUnroll], ur[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            gr[k].load(gate, w.col + k * kSeg, a.cols, lane);
            ur[k].load(up, w.col + k * kSeg, a.cols, lane);
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int c0 = w.col + k * kSeg;
            float g[8], u[8], o[8];
            gr[k].get(g);
            ur[k].get(u);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = g[j] * sigmoid(g[j]) * u[j];
            if (a.a.p) seg_store<BF16, VEC>(row_ptr<BF16>(a.a, w.row), c0, a.cols, lane, o);
            if (a.gate8.codes) seg_quant<VEC>(a.gate8, w.row, c0, a.cols, lane, g);
            if (a.up8.codes) seg_quant<VEC>(a.up8, w.row, c0, a.cols, lane, u);
            if (a.a8.codes) seg_quant<VEC>(a.a8, w.row, c0, a.cols, lane, o);
        }
    }
}

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) k_swiglu_backward(const SwigluArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (Walk w(a.cols); w.row < a.rows; w.next()) {
        const void* da = row_ptr<BF16>(a.a, w.row);
        Raw<BF16, VEC> dr[kUnroll];
        Raw8<VEC> gr[kUnroll], ur[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            dr[k].load(da, w.col + k * kSeg, a.cols, lane);
            gr[k].load(a.gate8, w.row, w.col + k * kSeg, a.cols, lane);
            ur[k].load(a.up8, w.row, w.col + k * kSeg, a.cols, lane);
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int c0 = w.col + k * kSeg;
            float g[8], u[8], d[8], o[8];
            dr[k].get(d);
            gr[k].get(a.gate8.format, g);
            ur[k].get(a.up8.format, u);
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
}

// Blocks for all units, at most kBlocks (the kernels stride over what is left).
unsigned blocks_for(long long rows, int cols) {
    const long long units = rows * ((cols + kUnroll * kSeg - 1) / (kUnroll * kSeg));
    const long long b = (units + kThreads / 32 - 1) / (kThreads / 32);
    return (unsigned)(b < kBlocks ? b : kBlocks);
}

template <typename Args>
cudaError_t launch(void (*const (&k)[4])(Args), const Args& a, bool bf16, bool vec, cudaStream_t s) {
    return launch_pdl(k[(bf16 ? 2 : 0) + (vec ? 1 : 0)], dim3(blocks_for(a.rows, a.cols)), dim3(kThreads), 0,
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
