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

// The segment's values of row pointer p (already at the row), columns c0 .. c0 + 255;
// zero at and beyond `cols`.
template <bool BF16, bool VEC>
__device__ __forceinline__ void seg_load(const void* p, int c0, int cols, int lane, float (&v)[8]) {
    if (VEC && c0 + 8 * lane + 8 <= cols) {
        const long long e = c0 + 8 * lane;
        if (BF16) {
            const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + e);
            v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
            v[4] = bf16_lo(w.z), v[5] = bf16_hi(w.z), v[6] = bf16_lo(w.w), v[7] = bf16_hi(w.w);
        } else {
            const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + e);
            const float4 a = f[0], b = f[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = c0 + seg_col<VEC>(lane, j);
        v[j] = c < cols ? load_one<BF16>(p, c) : 0.f;
    }
}

template <bool BF16, bool VEC>
__device__ __forceinline__ void seg_store(void* p, int c0, int cols, int lane, const float (&v)[8]) {
    if (VEC && c0 + 8 * lane + 8 <= cols) {
        const long long e = c0 + 8 * lane;
        if (BF16) {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + e) =
                make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
        } else {
            float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + e);
            f[0] = make_float4(v[0], v[1], v[2], v[3]);
            f[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = c0 + seg_col<VEC>(lane, j);
        if (c < cols) store_one<BF16>(p, c, v[j]);
    }
}

// Scale byte of a group whose largest magnitude has the bits `a` (sign cleared): the
// smallest biased exponent with a <= L 2^e, L = 448 = 1.75 2^8 or 127 = 1.984375 2^6.
// Adding 2^23 - 1 - mantissa(L) carries into the exponent exactly when the mantissa of a
// exceeds that of L.  An infinity or NaN gives 255.
__device__ __forceinline__ uint32_t act_scale_byte(uint32_t a, int format) {
    const int e = format == kE4M3 ? (int)((a + 0x1fffffu) >> 23) - 8 : (int)((a + 0x01ffffu) >> 23) - 6;
    const int top = format == kE4M3 ? 127 + 119 : 127 + 121;
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
__device__ __forceinline__ uint32_t act_code2(float a, float b, int format) {
    if (format == kE4M3) {
        uint16_t r;   // round to nearest even, saturating at 448; b goes to the low byte
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
        return r;
    }
    // groups clamped at the largest scale may exceed 127
    const int x = __float2int_rn(fminf(fmaxf(a, -127.f), 127.f)), y = __float2int_rn(fminf(fmaxf(b, -127.f), 127.f));
    return (uint32_t)(x & 0xff) | ((uint32_t)(y & 0xff) << 8);
}
// Two codes (low byte first) -> their numbers.
__device__ __forceinline__ float2 act_number2(uint32_t q, int format) {
    if (format == kE4M3) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)q));
        return __half22float2(*reinterpret_cast<__half2*>(&h));
    }
    return make_float2((float)(int8_t)(q & 0xff), (float)(int8_t)((q >> 8) & 0xff));
}

// Writes the segment in 8 bits at row `row`.  Values beyond `cols` must be zero; lanes of
// a partly filled last group take part with those zeros.
template <bool VEC>
__device__ __forceinline__ void seg_quant(const Act8& q, long long row, int c0, int cols, int lane,
                                          const float (&v)[8]) {
    uint8_t* codes = q.codes + row * q.ldq + c0;
    uint8_t* scales = q.scales + row * q.lds + (c0 >> 5);
    uint32_t m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = __float_as_uint(v[j]) & 0x7fffffffu;
    if (VEC) {
        uint32_t a = max(max(max(m[0], m[1]), max(m[2], m[3])), max(max(m[4], m[5]), max(m[6], m[7])));
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
        const uint32_t byte = act_scale_byte(a, q.format);
        const float inv = act_inverse(byte);
        float w[8];
        // inv = 0 marks a group that is not finite: its codes are zero (0 * inf would be NaN)
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = inv == 0.f ? 0.f : v[j] * inv;
        const uint32_t lo = act_code2(w[0], w[1], q.format) | act_code2(w[2], w[3], q.format) << 16;
        const uint32_t hi = act_code2(w[4], w[5], q.format) | act_code2(w[6], w[7], q.format) << 16;
        // row pitches are multiples of 16: the eight bytes lie within the row's padding
        if (c0 + 8 * lane < cols) {
            *reinterpret_cast<uint2*>(codes + 8 * lane) = make_uint2(lo, hi);
            if ((lane & 3) == 0) scales[lane >> 2] = (uint8_t)byte;
        }
    } else {
        uint32_t mine = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t byte = act_scale_byte(__reduce_max_sync(0xffffffffu, m[j]), q.format);
            if (lane == j) mine = byte;
            const float inv = act_inverse(byte);
            const float w = inv == 0.f ? 0.f : v[j] * inv;
            if (c0 + 32 * j + lane < cols) codes[32 * j + lane] = (uint8_t)act_code2(w, 0.f, q.format);
        }
        if (lane < 8 && c0 + 32 * lane < cols) scales[lane] = (uint8_t)mine;
    }
}

// Reads the segment of row `row` back; zero at and beyond `cols`.
template <bool VEC>
__device__ __forceinline__ void seg_dequant(const Act8& q, long long row, int c0, int cols, int lane, float (&v)[8]) {
    const uint8_t* codes = q.codes + row * q.ldq + c0;
    const uint8_t* scales = q.scales + row * q.lds + (c0 >> 5);
    if (VEC) {
        uint2 w = make_uint2(0, 0);
        float s = 0.f;
        if (c0 + 8 * lane < cols) {   // the row's padding completes the eight bytes
            w = *reinterpret_cast<const uint2*>(codes + 8 * lane);
            s = act_scale(scales[lane >> 2]);
        }
        const float2 a = act_number2(w.x & 0xffff, q.format), b = act_number2(w.x >> 16, q.format);
        const float2 c = act_number2(w.y & 0xffff, q.format), d = act_number2(w.y >> 16, q.format);
        v[0] = a.x * s, v[1] = a.y * s, v[2] = b.x * s, v[3] = b.y * s;
        v[4] = c.x * s, v[5] = c.y * s, v[6] = d.x * s, v[7] = d.y * s;
        if (c0 + 8 * lane + 8 > cols) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + 8 * lane + j >= cols) v[j] = 0.f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = 32 * j + lane;
            v[j] = c0 + c < cols ? act_number2(codes[c], q.format).x * act_scale(scales[j]) : 0.f;
        }
    }
}

}  // namespace muon
