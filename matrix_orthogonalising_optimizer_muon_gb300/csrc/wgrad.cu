// Weight gradient from activations held in 8 bits: grad (+)= dy^T x diag(col_scale), one
// weight or one per expert over its own range of tokens.
//
// The product contracts over tokens, so both operands are read as they are stored, tokens x
// columns, as MN-major tcgen05 operands: A = dy (bf16), B = x.  x arrives as one byte per
// value; eight warps turn codes and scales into bf16 in shared memory.  A code times a power
// of two has at most 8 significant bits and lies in bf16's normal range, so this loses
// nothing, and the product costs bf16 tensor time while x costs a byte per value of traffic.
//
// A cluster of two CTAs computes 256 x 256 tiles (tcgen05.mma.cta_group::2, M = N = 256,
// fp32 accumulators in TMEM, double-buffered), persistent over the tiles.  Per CTA, 14 warps:
//   0      TMA of x: per step of 64 tokens its 128 columns' codes (8 KB) and scales (1 KB)
//   1      MMA issue (one thread of the even CTA) and TMEM allocation
//   2      TMA of dy: its 128 columns (16 KB per step)
//   3-10   conversion of x into a 16 KB bf16 operand per step
//   11-14  epilogue: column scale, addition to grad, stores
// Two rings: x as it arrives (full_r by TMA, empty_r by the conversion), and the operands (dy
// and converted x; ready, on the even CTA, by both CTAs' conversion warps and dy's TMA bytes,
// empty, on both, by the MMAs), so the MMA thread has one wait and one commit per step.
#include <cuda.h>
#include <cuda_bf16.h>

#include "act8.cuh"
#include "kernels.h"
#include "plan.h"
#include "ptx.cuh"

namespace muon {
namespace {

#ifndef W_NB
#define W_NB 5
#define W_NR 5
#define W_CW 10
#define W_CG 5
#endif
constexpr int kWgStepT = 64;            // tokens per step
constexpr int kRingM = W_NB;            // steps of MMA operands
constexpr int kRingR = W_NR;            // steps of x as it arrives
constexpr int kConvWarps = W_CW;
constexpr int kConvGroups = W_CG;       // steps in conversion at a time
constexpr int kGroupWarps = kConvWarps / kConvGroups;
constexpr int kRows = kWgStepT / kGroupWarps;   // token rows per conversion warp and step
constexpr int kConvFirst = 3;           // first conversion warp
constexpr int kEpiFirst = kConvFirst + kConvWarps;
constexpr int kWgEpiWarps = 4;
constexpr int kWgThreads = 32 * (kEpiFirst + kWgEpiWarps);
constexpr int kBandM = 8;               // tiles along m whose columns of dy are in flight together
// A ring slot is always converted by the same warps, which so see every phase of its barriers.
static_assert(kRingR % kConvGroups == 0 && kRingM % kConvGroups == 0 && kRows % 8 == 0, "ring sizes");

struct WgCfg {
    static constexpr int A_BYTES = 128 * kWgStepT * 2;      // 128 columns of dy, or of x in bf16
    static constexpr int RAW_BYTES = 128 * kWgStepT;
    static constexpr int SCALE_BYTES = 16 * kWgStepT;
    static constexpr int R_BYTES = RAW_BYTES + SCALE_BYTES;
    static constexpr int CHUNK_BYTES = 64 * kWgStepT * 2;   // 64 columns of an MN-major operand
    static constexpr int SLOT_BYTES = 2 * A_BYTES;          // dy, then x
    static constexpr int R_OFFSET = kRingM * SLOT_BYTES;
    static constexpr int OUT_OFFSET = R_OFFSET + kRingR * R_BYTES;
    static constexpr int OUT_LD = 36;                       // one 32 x 32 block of floats, rows padded by 16 bytes
    static constexpr int OUT_WARP = 32 * OUT_LD * 4;
    static constexpr int BAR_OFFSET = OUT_OFFSET + kWgEpiWarps * OUT_WARP;
    static constexpr int SMEM_BYTES = BAR_OFFSET + 512 + 1024;
};
static_assert(WgCfg::SMEM_BYTES <= 232448, "weight-gradient kernel exceeds the shared memory of one CTA");

struct WgradLaunch {
    CUtensorMap map_y, map_x, map_s;
    WgradArgs a;
    int tiles_m, tiles_n, units;   // units: tiles of all groups
    int chain;                     // tokens one accumulator takes
    int wide;                      // rows of grad are aligned to four elements
};

struct Unit {
    int m0, n0;
    long long begin, end;   // tokens
    int group;
};

__device__ __forceinline__ Unit decode_unit(const WgradLaunch& L, int u) {
    const int per = L.tiles_m * L.tiles_n;
    Unit r;
    r.group = u / per;
    int t = u - r.group * per;
    // bands of kBandM tiles along m, within a band along n: the tiles that run together share
    // both operands' columns in L2
    const int band = t / (kBandM * L.tiles_n);
    t -= band * kBandM * L.tiles_n;
    const int wide = min(kBandM, L.tiles_m - band * kBandM);
    r.m0 = (band * kBandM + t % wide) * 256;
    r.n0 = t / wide * 256;
    r.begin = 0, r.end = L.a.tokens;
    if (L.a.offsets) {
        r.begin = min(max((long long)L.a.offsets[r.group], 0ll), L.a.tokens);
        r.end = min(max((long long)L.a.offsets[r.group + 1], r.begin), L.a.tokens);
    }
    return r;
}
__device__ __forceinline__ int unit_steps(const Unit& u) { return (int)((u.end - u.begin + kWgStepT - 1) / kWgStepT); }

__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf2_sub(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Four codes times the power of two s2 (twice the same bf16) as two pairs of bf16: bytes 0 and
// 2 of w in x, bytes 1 and 3 in y.  So the operand's columns are permuted within every four,
// which the epilogue undoes for free; pairing
// neighbours would cost a byte permutation per pair on the ALU, the busiest pipe here.
//  e4m3: the seven magnitude bits placed at bits 4-10 of a bf16 read as code * 2^-120 (the
//        exponent biases differ by 120; a subnormal code lands as a bf16 subnormal).
//  int8: with x = q & 127 the bf16 0x4300 + x is 128 + x exactly, and 128 or 256 less is q.
// A group that was not finite has codes 0 and the scale byte 255, a bf16 infinity: NaN.
template <int FMT>
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t w, uint32_t s2) {
    if (FMT == kE4M3) {
        const uint32_t e = ((w << 8) & 0x80008000u) | ((w << 4) & 0x07f007f0u);
        const uint32_t o = (w & 0x80008000u) | ((w >> 4) & 0x07f007f0u);
        return make_uint2(bf2_mul(bf2_mul(e, 0x7b807b80u), s2), bf2_mul(bf2_mul(o, 0x7b807b80u), s2));   // 2^120
    }
    const uint32_t h = w >> 8;
    const uint32_t e = bf2_sub((w & 0x007f007fu) | 0x43004300u, (w & 0x00800080u) | 0x43004300u);
    const uint32_t o = bf2_sub((h & 0x007f007fu) | 0x43004300u, (h & 0x00800080u) | 0x43004300u);
    return make_uint2(bf2_mul(e, s2), bf2_mul(o, s2));
}

// Four neighbouring elements, aligned to their size.
template <bool BF16>
__device__ __forceinline__ float4 load_four(const void* p, long long e) {
    if (!BF16) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + e);
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + e);
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}
template <bool BF16>
__device__ __forceinline__ void store_four(void* p, long long e, const float4& v) {
    if (BF16)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + e) = make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
    else
        *reinterpret_cast<float4*>(static_cast<float*>(p) + e) = v;
}

__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t x) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}

// TMA_Y: dy's rows are 16-byte aligned and come by TMA; else, and for the last step of an
// expert's tokens, whose following rows are other experts', the conversion warps load them.
template <int FMT, bool TMA_Y, bool BF16>
__global__ void __launch_bounds__(kWgThreads) k_wgrad(const __grid_constant__ WgradLaunch L) {
    using Cfg = WgCfg;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full_r = reinterpret_cast<uint64_t*>(smem + Cfg::BAR_OFFSET);
    uint64_t* empty_r = full_r + kRingR;
    uint64_t* ready = empty_r + kRingR;
    uint64_t* empty = ready + kRingM;
    uint64_t* tfull = empty + kRingM;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t q = cluster_ctarank() & 1u;
    const bool leader = q == 0;
    const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kRingR; ++s) {
            mbar_init(full_r + s, 1);
            mbar_init(empty_r + s, kGroupWarps);
        }
        for (int s = 0; s < kRingM; ++s) {
            mbar_init(ready + s, 1 + 2 * kGroupWarps);
            mbar_init(empty + s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull + a, 1);
            mbar_init(tempty + a, 2 * kWgEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        if (TMA_Y) tma_prefetch_desc(&L.map_y);
        tma_prefetch_desc(&L.map_x);
        tma_prefetch_desc(&L.map_s);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();   // barriers of both CTAs initialised before any remote signal
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_trigger();
    pdl_wait();

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA of x
            uint32_t it = 0;
            bool ok = true;
            for (int u = first; ok && u < L.units; u += stride) {
                const Unit w = decode_unit(L, u);
                const int steps = unit_steps(w);
                const int xn = w.n0 + 128 * (int)q;
                for (int k = 0; k < steps; ++k, ++it) {
                    const uint32_t s = it % kRingR;
                    if (!mbar_wait_idle(empty_r + s, (it / kRingR & 1u) ^ 1u, abort_flag, L.a.status,
                                        kStatusTimeoutProducer, false)) {
                        ok = false;
                        break;
                    }
                    uint8_t* sr = smem + Cfg::R_OFFSET + s * Cfg::R_BYTES;
                    const int t0 = (int)(w.begin + (long long)k * kWgStepT);
                    mbar_arrive_expect_tx(full_r + s, Cfg::R_BYTES);
                    tma_load_2d(sr, &L.map_x, full_r + s, xn, t0);
                    tma_load_2d(sr + Cfg::RAW_BYTES, &L.map_s, full_r + s, (xn >> 5) & ~15, t0);
                }
            }
            if (!ok) {   // let the copies already issued land before the CTA exits
                const uint32_t from = it > (uint32_t)kRingR ? it - kRingR : 0u;
                const unsigned long long t0 = globaltimer_ns();
                for (uint32_t j = from; j < it; ++j)
                    while (!mbar_try_wait(full_r + j % kRingR, j / kRingR & 1u) &&
                           globaltimer_ns() - t0 < kWaitTimeoutNs) {
                    }
            }
        }
    } else if (warp == 2) {
        if (lane == 0) {
            // ---------------- TMA of dy, completion on the even CTA's barrier
            uint32_t slot = 0, ph = 1;
            bool ok = true;
            for (int u = first; ok && u < L.units; u += stride) {
                const Unit w = decode_unit(L, u);
                const int steps = unit_steps(w);
                const int ym = w.m0 + 128 * (int)q;
                for (int k = 0; k < steps; ++k) {
                    if (!mbar_wait_idle(empty + slot, ph, abort_flag, L.a.status, kStatusTimeoutProducer, false)) {
                        ok = false;
                        break;
                    }
                    const long long t0 = w.begin + (long long)k * kWgStepT;
                    if (!TMA_Y || t0 + kWgStepT > w.end) {   // filled by the conversion warps
                        if (leader) mbar_arrive(ready + slot);
                    } else {
                        uint8_t* sa = smem + slot * Cfg::SLOT_BYTES;
                        const uint32_t fb = mapa_shared(smem_u32(ready + slot), 0);
                        if (leader) mbar_arrive_expect_tx(ready + slot, 2 * Cfg::A_BYTES);
                        tma_load_2d_pair(sa, &L.map_y, fb, ym, (int)t0);
                        tma_load_2d_pair(sa + Cfg::CHUNK_BYTES, &L.map_y, fb, ym + 64, (int)t0);
                    }
                    if (++slot == kRingM) slot = 0, ph ^= 1u;
                }
            }
            if (!ok) {   // copies already issued signal the even CTA; give them time to land
                const unsigned long long t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 2000000ull) {
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            // ---------------- MMA issue.  The tensor cores queue few instructions, so what this thread
            // does between two steps' MMAs is time they may idle: the next step's barrier is tested
            // before the step's last MMA is issued.
            uint32_t slot = 0, ph = 0;
            int local = 0;
            bool ok = true, next = false;
            constexpr uint32_t idesc = idesc_make(true, 256, 256, true, true);
            constexpr uint64_t kSlot = Cfg::SLOT_BYTES >> 4, kStep = 16 * 128 >> 4;   // of the address field
            const uint64_t ad0 = sdesc_sw128(smem_u32(smem), Cfg::CHUNK_BYTES, 1024);
            const uint64_t bd0 = sdesc_sw128(smem_u32(smem) + Cfg::A_BYTES, Cfg::CHUNK_BYTES, 1024);
            for (int u = first; ok && u < L.units; u += stride) {
                const Unit w = decode_unit(L, u);
                const int steps = unit_steps(w), chain = L.chain / kWgStepT;
                const int last = ((int)(w.end - w.begin - 1) & (kWgStepT - 1)) / 16 + 1;   // MMAs of the last step
                for (int k0 = 0; ok && k0 < steps; k0 += chain, ++local) {
                    const uint32_t acc = local & 1;
                    if (!mbar_wait_idle(tempty + acc, (local >> 1 & 1u) ^ 1u, abort_flag, L.a.status,
                                        kStatusTimeoutMma, true)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem_base + acc * 256;
                    const int k1 = min(steps, k0 + chain);
                    for (int k = k0; k < k1; ++k) {
                        if (!next && !mbar_wait(ready + slot, ph, abort_flag, L.a.status, kStatusTimeoutMma)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t ad = ad0 + slot * kSlot, bd = bd0 + slot * kSlot;
                        uint64_t* done = empty + slot;
                        const int n = k == steps - 1 ? last : 4;
                        mma_f16kind_pair(d, ad, bd, idesc, k != k0);
                        for (int kk = 1; kk < n - 1; ++kk) mma_f16kind_pair(d, ad + kk * kStep, bd + kk * kStep, idesc, 1);
                        if (++slot == kRingM) slot = 0, ph ^= 1u;
                        next = mbar_test_wait(ready + slot, ph);
                        if (n > 1) mma_f16kind_pair(d, ad + (n - 1) * kStep, bd + (n - 1) * kStep, idesc, 1);
                        mma_commit_pair(done, 0x3);
                    }
                    if (ok) mma_commit_pair(tfull + acc, 0x3);
                }
            }
            mma_commit_pair(drain, 0x1);
            const unsigned long long t0 = globaltimer_ns();
            while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
            }
        }
    } else if (warp < kEpiFirst) {
        // ---------------- conversion: warp cw of the kGroupWarps that take every kConvGroups-th step
        const int cw = (warp - kConvFirst) % kGroupWarps;
        const uint32_t cg = (warp - kConvFirst) / kGroupWarps;
        const uint32_t ready_lead = mapa_shared(smem_u32(ready), 0);
        uint32_t it = 0;
        bool ok = true;
        // A pass of a warp takes eight token rows: lane l the row p of l / 8, or p ^ 5 for the upper
        // four of its eight lanes, and 16 codes (16-byte piece l & 3) of either 64-column half.
        // Rows p and p ^ 5 differ in bits 0 and 2: under the 128-byte swizzle of both buffers the
        // eight lanes of a memory phase then touch all bank groups, in the loads (bit 2) and in the
        // stores of the even, then the odd 16-byte pieces of the operand row (bit 0).
        const int prow = (lane >> 3) ^ (lane & 4 ? 5 : 0), pc = lane & 3;
        const int row0 = cw * kRows + prow;
        const uint32_t src0 = row0 * 128 + ((pc ^ prow) << 4);             // half 0; half 1: ^ 64
        const uint32_t dst0 = row0 * 128 + (((2 * pc) ^ prow) << 4);       // its second piece: ^ 16
        const uint32_t sel = 0x0404u + 0x1010u * (pc >> 1);                // its scale byte in bytes 1 and 3
        for (int u = first; ok && u < L.units; u += stride) {
            const Unit w = decode_unit(L, u);
            const int steps = unit_steps(w);
            const int off = ((w.n0 + 128 * (int)q) >> 5) & 15;   // the CTA's four of the 16 loaded scales
            for (int k = 0; k < steps; ++k, ++it) {
                const int left = (int)min((long long)kWgStepT, w.end - w.begin - (long long)k * kWgStepT);
                const bool plain = !TMA_Y || left < kWgStepT;
                if (it % kConvGroups != cg) continue;
                const uint32_t r = it % kRingR, b = it % kRingM;
                const uint8_t* sr = smem + Cfg::R_OFFSET + r * Cfg::R_BYTES;
                const uint32_t sa = smem_u32(smem + b * Cfg::SLOT_BYTES), sb = sa + Cfg::A_BYTES;
                if (!mbar_wait_idle(full_r + r, it / kRingR & 1u, abort_flag, L.a.status, kStatusTimeoutProducer,
                                    false)) {
                    ok = false;
                    break;
                }
                uint4 raw[kRows / 4];
                uint32_t sc[kRows / 8];
#pragma unroll
                for (int i = 0; i < kRows / 8; ++i) {
                    raw[2 * i] = *reinterpret_cast<const uint4*>(sr + i * 1024 + src0);
                    raw[2 * i + 1] = *reinterpret_cast<const uint4*>(sr + i * 1024 + (src0 ^ 64));
                    sc[i] = *reinterpret_cast<const uint32_t*>(sr + Cfg::RAW_BYTES + (row0 + 8 * i) * 16 + off);
                }
                if (left < kWgStepT) {
#pragma unroll
                    for (int i = 0; i < kRows / 8; ++i)
                        if (row0 + 8 * i >= left) raw[2 * i] = raw[2 * i + 1] = make_uint4(0, 0, 0, 0), sc[i] = 0;
                }
                if (!mbar_wait_idle(empty + b, (it / kRingM & 1u) ^ 1u, abort_flag, L.a.status,
                                    kStatusTimeoutProducer, false)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int i = 0; i < kRows / 4; ++i) {
                    const uint32_t s2 = __byte_perm(sc[i >> 1], 0, sel + (i & 1) * 0x2020u) >> 1;
                    const uint2 a = codes_to_bf16<FMT>(raw[i].x, s2), d = codes_to_bf16<FMT>(raw[i].y, s2);
                    const uint2 e = codes_to_bf16<FMT>(raw[i].z, s2), f = codes_to_bf16<FMT>(raw[i].w, s2);
                    const uint32_t to = sb + (i & 1) * Cfg::CHUNK_BYTES + (i >> 1) * 1024;
                    sts128(to + dst0, make_uint4(a.x, a.y, d.x, d.y));
                    sts128(to + (dst0 ^ 16), make_uint4(e.x, e.y, f.x, f.y));
                }
                if (plain) {   // dy: the warp's token rows, columns 2 lane, 2 lane + 1 of both halves
                    const int ym = w.m0 + 128 * (int)q + 2 * lane;
#pragma unroll 16
                    for (int i = 0; i < 2 * kRows; ++i) {
                        const int t = cw * kRows + (i >> 1), col = ym + 64 * (i & 1);
                        const uint16_t* p = static_cast<const uint16_t*>(L.a.dy) +
                                            (w.begin + (long long)k * kWgStepT + t) * L.a.lddy + col;
                        const uint32_t y0 = t < left && col < L.a.m ? p[0] : 0;
                        const uint32_t y1 = t < left && col + 1 < L.a.m ? p[1] : 0;
                        sts32(sa + (i & 1) * Cfg::CHUNK_BYTES + t * 128 + (((lane >> 2) ^ (t & 7)) << 4) + (lane & 3) * 4,
                              y0 | y1 << 16);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // writes visible to the MMAs
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(empty_r + r);
                    // Release at CTA scope on either barrier: the MMAs read this warp's writes in its own
                    // CTA's shared memory, where the fence above has put them.  A release at cluster scope
                    // waits about 1000 cycles for the warp's other traffic (370 against 260 us at
                    // 8192 tokens, 3584 x 3584).
                    if (leader)
                        mbar_arrive(ready + b);
                    else
                        mbar_arrive_remote_cta(ready_lead + b * 8);
                }
            }
        }
    } else {
        // ---------------- epilogue: TMEM lane quarter = warp % 4.  Each 32 x 32 block goes through
        // shared memory, so that a warp reads and writes grad in 128-byte row pieces: four rows at a
        // time, four columns per lane, where the rows are aligned, else one row, a column per lane.
        const int wq = warp & 3;
        const uint32_t tempty_lead = mapa_shared(smem_u32(tempty), 0);
        float* blk = reinterpret_cast<float*>(smem + Cfg::OUT_OFFSET + (warp - kEpiFirst) * Cfg::OUT_WARP);
        const int rl = lane >> 3, cl = 4 * (lane & 7);
        int local = 0;
        bool ok = true;
        for (int u = first; ok && u < L.units; u += stride) {
            const Unit w = decode_unit(L, u);
            const int chains = (int)((w.end - w.begin + L.chain - 1) / L.chain);
            const int r0 = w.m0 + 128 * (int)q + 32 * wq;
            const int rows = min(32, L.a.m - r0);
            const long long gbase = ((long long)w.group * L.a.m + r0) * L.a.n;
            if (chains == 0 && L.a.accumulate) continue;
            for (int ch = 0; ch < max(chains, 1); ++ch) {
                const bool any = chains > 0;
                const bool add = L.a.accumulate || ch > 0;   // a later chain of tokens adds to what this warp wrote
                const uint32_t acc = local & 1;
                if (any && !mbar_wait_idle(tfull + acc, local >> 1 & 1u, abort_flag, L.a.status,
                                           kStatusTimeoutEpilogue, true)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tbase = tmem_base + acc * 256 + (static_cast<uint32_t>(wq * 32) << 16);
                for (int c0 = 0; c0 < 256 && w.n0 + c0 < L.a.n && rows > 0; c0 += 32) {
                    const bool wide = L.wide && w.n0 + c0 + 32 <= L.a.n;
                    float4 g[8];
                    if (wide) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int r = 4 * i + rl;
                            g[i] = add && r < rows ? load_four<BF16>(L.a.grad, gbase + (long long)r * L.a.n + w.n0 + c0 + cl)
                                                   : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                    }
                    if (any) {
                        uint32_t v[32];
                        tmem_ld32(tbase + c0, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; j += 4)   // undoes the operand's column order
                            *reinterpret_cast<uint4*>(blk + lane * Cfg::OUT_LD + j) =
                                make_uint4(v[j], v[j + 2], v[j + 1], v[j + 3]);
                        __syncwarp();
                    }
                    if (wide) {
                        float4 cs = make_float4(1.f, 1.f, 1.f, 1.f);
                        if (L.a.col_scale) {
                            const float* p = L.a.col_scale + w.n0 + c0 + cl;
                            cs = make_float4(p[0], p[1], p[2], p[3]);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int r = 4 * i + rl;
                            if (any) {
                                const float4 v = *reinterpret_cast<const float4*>(blk + r * Cfg::OUT_LD + cl);
                                g[i].x = fmaf(v.x, cs.x, g[i].x), g[i].y = fmaf(v.y, cs.y, g[i].y);
                                g[i].z = fmaf(v.z, cs.z, g[i].z), g[i].w = fmaf(v.w, cs.w, g[i].w);
                            }
                            if (r < rows)
                                store_four<BF16>(L.a.grad, gbase + (long long)r * L.a.n + w.n0 + c0 + cl, g[i]);
                        }
                    } else if (w.n0 + c0 + lane < L.a.n) {
                        const int col = w.n0 + c0 + lane;
                        const float cs = L.a.col_scale ? L.a.col_scale[col] : 1.f;
                        for (int rb = 0; rb < rows; rb += 8) {
                            float v[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                v[i] = add && rb + i < rows ? load_one<BF16>(L.a.grad, gbase + (long long)(rb + i) * L.a.n + col)
                                                            : 0.f;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                if (any) v[i] = fmaf(blk[(rb + i) * Cfg::OUT_LD + lane], cs, v[i]);
                                if (rb + i < rows) store_one<BF16>(L.a.grad, gbase + (long long)(rb + i) * L.a.n + col, v[i]);
                            }
                        }
                    }
                    __syncwarp();
                }
                if (any) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (leader)
                            mbar_arrive(tempty + acc);
                        else
                            mbar_arrive_remote(tempty_lead + acc * 8);
                    }
                    ++local;
                }
            }
        }
    }

    tc_fence_before();
    cluster_sync();   // every MMA of the pair done, both TMEMs drained
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

// Row-major tokens x cols tensor, boxes of box_cols x 64 tokens.
bool map_2d(CUtensorMap* map, const void* base, bool bytes, uint64_t cols, uint64_t rows, uint64_t pitch,
            uint32_t box_cols, bool swizzle) {
    muon_impl::EncodeTiledFn fn = muon_impl::encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {pitch};
    cuuint32_t box[2] = {box_cols, (cuuint32_t)kWgStepT};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

typedef void (*WgradKernel)(WgradLaunch);
WgradKernel pick(int fmt, bool tma_y, bool bf16) {
    static const WgradKernel k[2][2][2] = {
        {{k_wgrad<kE4M3, false, false>, k_wgrad<kE4M3, false, true>}, {k_wgrad<kE4M3, true, false>, k_wgrad<kE4M3, true, true>}},
        {{k_wgrad<kInt8, false, false>, k_wgrad<kInt8, false, true>}, {k_wgrad<kInt8, true, false>, k_wgrad<kInt8, true, true>}}};
    return k[fmt][tma_y][bf16];
}

}  // namespace

cudaError_t wgrad_prepare() {
    for (int i = 0; i < 8; ++i) {
        const cudaError_t e = cudaFuncSetAttribute(pick(i & 1, i >> 1 & 1, i >> 2 & 1),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, WgCfg::SMEM_BYTES);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_wgrad(const WgradArgs& a, bool bf16_grad, int sm_count, cudaStream_t s) {
    if (a.tokens == 0) {   // nothing to contract
        const size_t bytes = (size_t)a.groups * a.m * a.n * (bf16_grad ? 2 : 4);
        return a.accumulate ? cudaSuccess : cudaMemsetAsync(a.grad, 0, bytes, s);
    }
    WgradLaunch L;
    L.a = a;
    L.tiles_m = (a.m + 255) / 256;
    L.tiles_n = (a.n + 255) / 256;
    const long long units = (long long)a.groups * L.tiles_m * L.tiles_n;
    if (units >= (1ll << 31)) return cudaErrorInvalidValue;
    L.units = (int)units;
    // The tensor cores' adds truncate: the sum of one accumulator drifts by about 1.1e-5 of
    // itself over 16384 tokens of random data, in proportion to their number.  An fp32 gradient
    // keeps that below 6e-6 by adding up partial sums of 8192 tokens in the epilogue.
    L.chain = bf16_grad ? 1 << 30 : 8192;
    L.wide = a.n % 4 == 0 && (reinterpret_cast<uintptr_t>(a.grad) & (bf16_grad ? 7 : 15)) == 0;
    // TMA needs 16-byte aligned rows; x has them by its format
    const bool tma_y = ((reinterpret_cast<uintptr_t>(a.dy) | (uintptr_t)(a.lddy * 2)) & 15) == 0;
    if ((tma_y && !map_2d(&L.map_y, a.dy, false, a.m, a.tokens, a.lddy * 2, 64, true)) ||
        !map_2d(&L.map_x, a.x.codes, true, a.n, a.tokens, a.x.ldq, 128, true) ||
        !map_2d(&L.map_s, a.x.scales, true, (a.n + kActGroup - 1) / kActGroup, a.tokens, a.x.lds, 16, false))
        return cudaErrorInvalidValue;
    const unsigned pairs = (unsigned)std::min<long long>(units, sm_count / 2);
    return launch_pdl_cluster(pick(a.x.format, tma_y, bf16_grad), dim3(2 * pairs), dim3(kWgThreads), WgCfg::SMEM_BYTES,
                              s, 2u, L);
}

}  // namespace muon
