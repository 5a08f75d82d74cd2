// Device side of the 8-bit activation format, in units of one warp's segment: 256
// neighbouring values of a row, eight per lane.
//
// Two layouts of a segment over the lanes, chosen per launch:
//  VEC   lane l holds values 8 l .. 8 l + 7: one 16-byte load (bf16) or two (fp32) per
//        lane; four lanes share a scale group.  Needs 16-byte aligned rows.
//  else  lane l holds values 32 j + l, j = 0 .. 7: element loads, coalesced whatever the
//        alignment; value j of all lanes is one scale group.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "acts.h"

namespace muon {

constexpr int kSeg = 256;

template <bool VEC>
__device__ __forceinline__ int seg_col(int lane, int j) {
    return VEC ? 8 * lane + j : 32 * j + lane;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ char* row_ptr(const Mat& m, uint32_t row) {
    return static_cast<char*>(m.p) + (uint64_t)row * m.pitch;
}
template <bool BF16>
__device__ __forceinline__ float load_one(const void* p, long long i) {
    return BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store_one(void* p, long long i, float v) {
    if (BF16)
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<float*>(p)[i] = v;
}

// A lane's eight values of a segment as loaded: bf16 in pairs (VEC), else fp32.  Loading and
// widening are apart so that several segments' loads can be in flight in few registers.
template <bool BF16, bool VEC>
struct Raw {
    static constexpr bool kPairs = BF16 && VEC;
    uint32_t r[kPairs ? 4 : 8];

    // Columns c0 .. c0 + 255 of the row at p; zero at and beyond `cols`.  FULL: none is.
    template <bool FULL = false>
    __device__ __forceinline__ void load(const void* p, int c0, int cols, int lane) {
        if (VEC && (FULL || c0 + 8 * lane + 8 <= cols)) {
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + (long long)(c0 + 8 * lane) * (BF16 ? 2 : 4));
            const uint4 a = q[0];
            r[0] = a.x, r[1] = a.y, r[2] = a.z, r[3] = a.w;
            if constexpr (!kPairs) {
                const uint4 b = q[1];
                r[4] = b.x, r[5] = b.y, r[6] = b.z, r[7] = b.w;
            }
        } else if constexpr (kPairs) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = c0 + 8 * lane + 2 * j;
                const uint16_t* q = static_cast<const uint16_t*>(p) + c;
                r[j] = (c < cols ? q[0] : 0u) | (c + 1 < cols ? (uint32_t)q[1] << 16 : 0u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = c0 + seg_col<VEC>(lane, j);
                r[j] = c < cols ? __float_as_uint(load_one<BF16>(p, c)) : 0u;
            }
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if constexpr (kPairs)
                v[j] = j & 1 ? bf16_hi(r[j >> 1]) : bf16_lo(r[j >> 1]);
            else
                v[j] = __uint_as_float(r[j]);
    }
};

// The segment's values of row pointer p, columns c0 .. c0 + 255; zero at and beyond `cols`.
template <bool BF16, bool VEC>
__device__ __forceinline__ void seg_load(const void* p, int c0, int cols, int lane, float (&v)[8]) {
    Raw<BF16, VEC> raw;
    raw.load(p, c0, cols, lane);
    raw.get(v);
}

template <bool BF16, bool VEC, bool FULL = false>
__device__ __forceinline__ void seg_store(void* p, int c0, int cols, int lane, const float (&v)[8]) {
    if (VEC && (FULL || c0 + 8 * lane + 8 <= cols)) {
        const long long e = c0 + 8 * lane;
        if (BF16) {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + e) =
                make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
        } else {
            float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + e);
            f[0] = make_float4(v[0], v[1], v[2], v[3]);
            f[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = c0 + seg_col<VEC>(lane, j);
            if (c < cols) store_one<BF16>(p, c, v[j]);
        }
    }
}

// Scale byte of a group whose largest magnitude has the bits `a` (sign cleared): the
// smallest biased exponent with a <= L 2^e, L = 448 = 1.75 2^8 or 127 = 1.984375 2^6.
// Adding 2^23 - 1 - mantissa(L) carries into the exponent exactly when the mantissa of a
// exceeds that of L.  An infinity or NaN gives 255.
template <int FMT>
__device__ __forceinline__ uint32_t act_scale_byte(uint32_t a) {
    const int e = FMT == kE4M3 ? (int)((a + 0x1fffffu) >> 23) - 8 : (int)((a + 0x01ffffu) >> 23) - 6;
    const int top = FMT == kE4M3 ? 127 + 119 : 127 + 121;
    return a >= 0x7f800000u ? 255u : (uint32_t)min(max(e, 127 - 110), top);
}
// 2^-e of a scale byte (17 .. 248); zero for a group that is not finite, so its codes are zero.
__device__ __forceinline__ float act_inverse(uint32_t byte) {
    return byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
}
// 2^e of a scale byte, NaN for 255 (byte 0 stands for the subnormal 2^-127).
__device__ __forceinline__ float act_scale(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7fc00000u : byte == 0u ? 0x00400000u : byte << 23);
}

// Two values already divided by their scale -> two codes (low byte first).
template <int FMT>
__device__ __forceinline__ uint32_t act_code2(float a, float b) {
    if (FMT == kE4M3) {
        uint16_t r;   // round to nearest even, saturating at 448; b goes to the low byte
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
        return r;
    }
    // groups clamped at the largest scale may exceed 127; 1.5 * 2^23 rounds to a whole number in
    // the low bits, ties to even
    const uint32_t x = __float_as_uint(fminf(fmaxf(a, -127.f), 127.f) + 12582912.f);
    const uint32_t y = __float_as_uint(fminf(fmaxf(b, -127.f), 127.f) + 12582912.f);
    return __byte_perm(x, y, 0x7740) & 0xffffu;
}
// Four codes (low byte first) -> their numbers.
template <int FMT>
__device__ __forceinline__ void act_number4(uint32_t w, float* v) {
    if (FMT == kE4M3) {
        uint32_t h[2];
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[0]) : "h"((uint16_t)(w & 0xffff)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[1]) : "h"((uint16_t)(w >> 16)));
        const float2 a = __half22float2(*reinterpret_cast<__half2*>(h));
        const float2 b = __half22float2(*reinterpret_cast<__half2*>(h + 1));
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
        return;
    }
    const uint32_t u = w ^ 0x80808080u;   // code + 128, then 2^23 + that, as the bits of a float
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 | j)) - 8388736.f;
}

// Writes the segment in 8 bits at row `row`.  Values beyond `cols` must be zero; lanes of
// a partly filled last group take part with those zeros.
template <int FMT, bool VEC, bool FULL>
__device__ __forceinline__ void seg_quant(const Act8& q, uint32_t row, int c0, int cols, int lane,
                                          const float (&v)[8]) {
    uint8_t* codes = q.codes + (uint64_t)row * q.ldq + c0;
    uint8_t* scales = q.scales + (uint64_t)row * q.lds + (c0 >> 5);
    uint32_t m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = __float_as_uint(v[j]) & 0x7fffffffu;
    if (VEC) {
        uint32_t a = __vimax3_u32(__vimax3_u32(m[0], m[1], m[2]), __vimax3_u32(m[3], m[4], m[5]), max(m[6], m[7]));
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
        const uint32_t byte = act_scale_byte<FMT>(a);
        const float inv = act_inverse(byte);
        uint32_t lo = act_code2<FMT>(v[0] * inv, v[1] * inv) | act_code2<FMT>(v[2] * inv, v[3] * inv) << 16;
        uint32_t hi = act_code2<FMT>(v[4] * inv, v[5] * inv) | act_code2<FMT>(v[6] * inv, v[7] * inv) << 16;
        if (byte == 255u) lo = hi = 0;   // a group that is not finite
        // row pitches are multiples of 16: the eight bytes lie within the row's padding
        if (FULL || c0 + 8 * lane < cols) {
            *reinterpret_cast<uint2*>(codes + 8 * lane) = make_uint2(lo, hi);
            if ((lane & 3) == 0) scales[lane >> 2] = (uint8_t)byte;
        }
    } else {
        uint32_t mine = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t byte = act_scale_byte<FMT>(__reduce_max_sync(0xffffffffu, m[j]));
            if (lane == j) mine = byte;
            const uint32_t code = byte == 255u ? 0u : act_code2<FMT>(v[j] * act_inverse(byte), 0.f);
            if (c0 + 32 * j + lane < cols) codes[32 * j + lane] = (uint8_t)code;
        }
        if (lane < 8 && c0 + 32 * lane < cols) scales[lane] = (uint8_t)mine;
    }
}
// The same, the format chosen at run time (uniform over the launch).
template <bool VEC, bool FULL = false>
__device__ __forceinline__ void seg_quant(const Act8& q, uint32_t row, int c0, int cols, int lane,
                                          const float (&v)[8]) {
    if (q.format == kE4M3)
        seg_quant<kE4M3, VEC, FULL>(q, row, c0, cols, lane, v);
    else
        seg_quant<kInt8, VEC, FULL>(q, row, c0, cols, lane, v);
}

// A lane's share of a segment in 8 bits as loaded: eight codes and their scale byte (VEC), else
// eight codes, each with its group's byte above it.
template <bool VEC>
struct Raw8 {
    uint32_t r[VEC ? 3 : 8];

    // The segment of row `row`; reads as zero at and beyond `cols`.  FULL: none is.
    template <bool FULL = false>
    __device__ __forceinline__ void load(const Act8& q, uint32_t row, int c0, int cols, int lane) {
        load<FULL>(q.codes + (uint64_t)row * q.ldq, q.scales + (uint64_t)row * q.lds, c0, cols, lane);
    }
    template <bool FULL = false>
    __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, int c0, int cols, int lane) {
        codes += c0, scales += c0 >> 5;
        if constexpr (VEC) {
            r[0] = r[1] = r[2] = 0;
            if (FULL || c0 + 8 * lane < cols) {   // the row's padding completes the eight bytes
                const uint2 w = *reinterpret_cast<const uint2*>(codes + 8 * lane);
                r[0] = w.x, r[1] = w.y, r[2] = scales[lane >> 2];
                const int left = cols - c0 - 8 * lane;
                if (left < 8) {   // padding: whatever it holds
                    r[0] &= left >= 4 ? 0xffffffffu : (1u << 8 * left) - 1u;
                    r[1] &= left <= 4 ? 0u : (1u << 8 * (left - 4)) - 1u;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = 32 * j + lane;
                r[j] = c0 + c < cols ? codes[c] | (uint32_t)scales[j] << 8 : 0u;
            }
        }
    }
    template <int FMT>
    __device__ __forceinline__ void get(float (&v)[8]) const {
        if constexpr (VEC) {
            const float s = act_scale(r[2]);
            act_number4<FMT>(r[0], v);
            act_number4<FMT>(r[1], v + 4);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= s;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t w = r[j];
                float n[4];
                act_number4<FMT>(w & 0xffu, n);
                v[j] = n[0] * act_scale(w >> 8);
            }
        }
    }
    __device__ __forceinline__ void get(int format, float (&v)[8]) const {
        if (format == kE4M3)
            get<kE4M3>(v);
        else
            get<kInt8>(v);
    }
};

}  // namespace muon
