// Activations to 8 bits and back, and SwiGLU with its inputs held in 8 bits.
//
// All four kernels read and write each value once (HBM-bound).  A warp takes units of kUnroll
// neighbouring segments of 256 values of a row, all loads before the first store.  HBM bounds
// them once units that lie inside the row skip the per-lane masks (with masks the loads wait on one
// another's branches: forward 207 us, backward 278).  Measured at 8192 x 18944 bf16: forward 200 us
// (6.25 TB/s, 94 % of the measured copy rate), backward 225 us (6.3 TB/s, 94 %), pack 69 us (102 %),
// unpack 71 us (99 %).  Rows that are not aligned are loaded and stored in shifted
// pieces, bound by instruction issue (18945 columns: 295, 337, 85 and 96 us).
#include "act8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
// Blocks that fit an SM (by registers); about four times as many are launched, which evens out the
// SMs' ends.  8192 x 18944 bf16: SwiGLU forward 202 us with four (216 with five, whose 48 registers
// spill), backward 219 us with five (221 with six, 224 with four).  Packing: 71 us with eight, 77 with
// six.  The shifted kernels need more registers: 18945 columns, unpacking 96 us with six (106 with
// eight), SwiGLU backward 337 us with four (376 with five).
constexpr int kFit = 8, kFitForward = 4, kFitBackward = 5;
constexpr int kSms = 152;
using Walk = RowWalk<kThreads>;
template <bool VEC>
constexpr int kMode = VEC ? kAligned : kShifted;

template <bool BF16, bool VEC, bool FULL>
__device__ __forceinline__ void unit_act_pack(const PackArgs& a, const Walk& w, int lane) {
    const void* x = row_ptr(a.x, w.row);
    Raw<BF16, kMode<VEC>> raw[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) raw[k].template load<FULL>(x, w.col + k * kSeg, a.cols, lane);
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        if (!FULL && w.col + k * kSeg >= a.cols) break;
        float v[8];
        raw[k].get(v);
        seg_quant<true, FULL>(a.q, w.row, w.col + k * kSeg, a.cols, lane, v);
    }
}
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads, VEC ? kFit : 6) k_act_pack(const PackArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (Walk w(a.cols); w.row < a.rows; w.next()) {
        if (w.col + Walk::kWidth <= a.cols)
            unit_act_pack<BF16, VEC, true>(a, w, lane);
        else
            unit_act_pack<BF16, VEC, false>(a, w, lane);
    }
}

template <bool BF16, bool VEC, bool FULL>
__device__ __forceinline__ void unit_act_unpack(const PackArgs& a, const Walk& w, int lane) {
    void* y = row_ptr(a.x, w.row);
    Raw8<true> raw[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) raw[k].template load<FULL>(a.q, w.row, w.col + k * kSeg, a.cols, lane);
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        if (!FULL && w.col + k * kSeg >= a.cols) break;
        float v[8];
        raw[k].get(a.q.format, v);
        seg_store<BF16, kMode<VEC>, FULL>(y, w.col + k * kSeg, a.cols, lane, v);
    }
}
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads, VEC ? kFit : 6) k_act_unpack(const PackArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (Walk w(a.cols); w.row < a.rows; w.next()) {
        if (w.col + Walk::kWidth <= a.cols)
            unit_act_unpack<BF16, VEC, true>(a, w, lane);
        else
            unit_act_unpack<BF16, VEC, false>(a, w, lane);
    }
}

// e^x for |x| <= 88; SCALED, for -110 <= x <= -80, as 2^64 e^x times 2^-64, so that a result below the normal
// range is rounded once.  e^x = 2^t 2^d with t = x log2 e rounded and 2^d by the first two terms of its
// series: d is what the product's rounding left (an fma gives it exactly, as in Dekker, "A floating-point
// technique for extending the available precision") and x times the rest of log2 e beyond one float, which
// alone is 11 ulp at 87.  Within 5 u, u = 2^-24, by the documented error of the base-2 exponential (expf
// and a division: 217 us forward, 304 backward).
template <bool SCALED>
__device__ __forceinline__ float exponential(float x) {
    constexpr double log2e = 1.4426950408889634;
    constexpr float hi = (float)log2e, lo = (float)(log2e - hi);
    const float t = x * hi, d = fmaf(x, lo, fmaf(x, hi, -t));
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(SCALED ? t + 64.f : t));   // t + 64: exact
    e = fmaf(e, d * 0.693147181f, e);
    return SCALED ? e * 5.42101086e-20f : e;
}
// 1 / (1 + e^-z), within 10 u for z >= -80.  Below, where the reciprocal would leave the normal range,
// e^z itself, for which the eight values of a lane are looked over once (a choice for each of them: forward
// 209 us, backward 231, against 200 and 226).
__device__ __forceinline__ void sigmoid(const float (&z)[8], float (&s)[8]) {
    const float least = fminf(fminf(fminf(z[0], z[1]), fminf(z[2], z[3])), fminf(fminf(z[4], z[5]), fminf(z[6], z[7])));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float e = exponential<false>(-fminf(z[j], 80.f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s[j]) : "f"(1.f + e));
    }
    if (least < -80.f) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (z[j] < -80.f) s[j] = exponential<true>(fmaxf(z[j], -110.f));
    }
}

template <bool BF16, bool VEC, bool FULL>
__device__ __forceinline__ void unit_swiglu_forward(const SwigluArgs& a, const Walk& w, int lane) {
    const void *gate = row_ptr(a.gate, w.row), *up = row_ptr(a.up, w.row);
    Raw<BF16, kMode<VEC>> gr[kUnroll], ur[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        gr[k].template load<FULL>(gate, w.col + k * kSeg, a.cols, lane);
        ur[k].template load<FULL>(up, w.col + k * kSeg, a.cols, lane);
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        const int c0 = w.col + k * kSeg;
        if (!FULL && c0 >= a.cols) break;
        float g[8], u[8], o[8];
        gr[k].get(g);
        ur[k].get(u);
        sigmoid(g, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = g[j] * o[j] * u[j];
        if (a.a.p) seg_store<BF16, kMode<VEC>, FULL>(row_ptr(a.a, w.row), c0, a.cols, lane, o);
        if (a.gate8.codes) seg_quant<true, FULL>(a.gate8, w.row, c0, a.cols, lane, g);
        if (a.up8.codes) seg_quant<true, FULL>(a.up8, w.row, c0, a.cols, lane, u);
        if (a.a8.codes) seg_quant<true, FULL>(a.a8, w.row, c0, a.cols, lane, o);
    }
}
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads, kFitForward) k_swiglu_forward(const SwigluArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (Walk w(a.cols); w.row < a.rows; w.next()) {
        if (w.col + Walk::kWidth <= a.cols)
            unit_swiglu_forward<BF16, VEC, true>(a, w, lane);
        else
            unit_swiglu_forward<BF16, VEC, false>(a, w, lane);
    }
}

template <bool BF16, bool VEC, bool FULL>
__device__ __forceinline__ void unit_swiglu_backward(const SwigluArgs& a, const Walk& w, int lane) {
    const void* da = row_ptr(a.a, w.row);
    Raw<BF16, kMode<VEC>> dr[kUnroll];
    Raw8<true> gr[kUnroll], ur[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        dr[k].template load<FULL>(da, w.col + k * kSeg, a.cols, lane);
        gr[k].template load<FULL>(a.gate8, w.row, w.col + k * kSeg, a.cols, lane);
        ur[k].template load<FULL>(a.up8, w.row, w.col + k * kSeg, a.cols, lane);
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        const int c0 = w.col + k * kSeg;
        if (!FULL && c0 >= a.cols) break;
        float g[8], u[8], d[8], o[8];
        dr[k].get(d);
        gr[k].get(a.gate8.format, g);
        ur[k].get(a.up8.format, u);
        sigmoid(g, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = o[j];
            const float silu = g[j] * s;
            o[j] = silu * u[j];
            g[j] = d[j] * u[j] * (s + silu * (1.f - s));   // dgate
            u[j] = d[j] * silu;                            // dup
        }
        seg_store<BF16, kMode<VEC>, FULL>(row_ptr(a.gate, w.row), c0, a.cols, lane, g);
        seg_store<BF16, kMode<VEC>, FULL>(row_ptr(a.up, w.row), c0, a.cols, lane, u);
        if (a.a8.codes) seg_quant<true, FULL>(a.a8, w.row, c0, a.cols, lane, o);
    }
}
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads, BF16 && VEC ? kFitBackward : 4) k_swiglu_backward(const SwigluArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (Walk w(a.cols); w.row < a.rows; w.next()) {
        if (w.col + Walk::kWidth <= a.cols)
            unit_swiglu_backward<BF16, VEC, true>(a, w, lane);
        else
            unit_swiglu_backward<BF16, VEC, false>(a, w, lane);
    }
}

// Blocks for all units, at most four times what fits (the kernels stride over what is left).
unsigned blocks_for(long long rows, int cols, int fit) {
    constexpr int width = Walk::kWidth;
    const long long units = rows * ((cols + width - 1) / width);
    const long long b = (units + kThreads / 32 - 1) / (kThreads / 32);
    return (unsigned)(b < 4 * fit * kSms ? b : 4 * fit * kSms);
}

template <typename Args>
cudaError_t launch(void (*const (&k)[4])(Args), const Args& a, int fit, bool bf16, bool vec, cudaStream_t s) {
    return launch_pdl(k[(bf16 ? 2 : 0) + (vec ? 1 : 0)], dim3(blocks_for(a.rows, a.cols, fit)), dim3(kThreads), 0,
                      s, a);
}

}  // namespace

cudaError_t launch_act_pack(const PackArgs& a, bool bf16, bool vec, cudaStream_t s) {
    static void (*const k[4])(PackArgs) = {k_act_pack<false, false>, k_act_pack<false, true>, k_act_pack<true, false>,
                                           k_act_pack<true, true>};
    return launch(k, a, kFit, bf16, vec, s);
}
cudaError_t launch_act_unpack(const PackArgs& a, bool bf16, bool vec, cudaStream_t s) {
    static void (*const k[4])(PackArgs) = {k_act_unpack<false, false>, k_act_unpack<false, true>,
                                           k_act_unpack<true, false>, k_act_unpack<true, true>};
    return launch(k, a, kFit, bf16, vec, s);
}
cudaError_t launch_swiglu_forward(const SwigluArgs& a, bool bf16, bool vec, cudaStream_t s) {
    static void (*const k[4])(SwigluArgs) = {k_swiglu_forward<false, false>, k_swiglu_forward<false, true>,
                                             k_swiglu_forward<true, false>, k_swiglu_forward<true, true>};
    return launch(k, a, kFitForward, bf16, vec, s);
}
cudaError_t launch_swiglu_backward(const SwigluArgs& a, bool bf16, bool vec, cudaStream_t s) {
    static void (*const k[4])(SwigluArgs) = {k_swiglu_backward<false, false>, k_swiglu_backward<false, true>,
                                             k_swiglu_backward<true, false>, k_swiglu_backward<true, true>};
    return launch(k, a, kFitBackward, bf16, vec, s);
}

}  // namespace muon
