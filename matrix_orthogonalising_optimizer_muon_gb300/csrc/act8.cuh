// Device side of the 8-bit activation format, in units of one warp's segment: 256
// neighbouring values of a row, eight per lane.
//
// How a segment lies over the lanes and is moved, chosen per launch:
//  kAligned  lane l holds values 8 l .. 8 l + 7: one 16-byte load (bf16) or two (fp32) per lane; four
//            lanes share a scale group.  Needs 16-byte aligned rows.
//  kShifted  the same on rows that are not aligned: the lanes load and store the aligned pieces that
//            hold their values and shift them into place.  The elementwise kernels use it.
//  kByValue  lane l holds values 32 j + l, j = 0 .. 7: element loads, coalesced whatever the alignment;
//            value j of all lanes is one scale group.  The norms use it: their rows' loads and stores are
//            a smaller part beside the barrier (forward 127 us, 151 shifted, at 16384 x 3585 bf16), while
//            SwiGLU and packing gain (8192 x 18945: 369, 457, 155, 126 us by value, 295, 337, 85, 96
//            shifted).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "acts.h"

namespace muon {

constexpr int kSeg = 256;
enum { kByValue = 0, kAligned = 1, kShifted = 2 };   // the first two convert from `rows are aligned`

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

// Words moved down by `shift` bytes (0 to 15, whole values); the last four are left undefined.
template <bool BF16, int N>
__device__ __forceinline__ void words_down(uint32_t (&w)[N], int shift) {
#pragma unroll
    for (int i = 0; i + 2 < N; ++i) w[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i + 1 < N; ++i) w[i] = shift & 4 ? w[i + 1] : w[i];
    if (BF16) {
#pragma unroll
        for (int i = 0; i + 1 < N; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (shift & 2) * 8);
    }
}

// A lane's eight values of a segment as loaded: bf16 in pairs (not by value), else fp32.  Loading and
// widening are apart so that several segments' loads can be in flight in few registers.
template <bool BF16, int MODE>
struct Raw {
    static constexpr bool VEC = MODE == kAligned, kPairs = BF16 && MODE != kByValue;
    static constexpr int kWords = kPairs ? 4 : 8, kSize = BF16 ? 2 : 4;
    uint32_t r[kWords];

    // Columns c0 .. c0 + 255 of the row at p; zero at and beyond `cols`.  FULL: none is.
    template <bool FULL = false>
    __device__ __forceinline__ void load(const void* p, int c0, int cols, int lane) {
        if constexpr (MODE == kByValue) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = c0 + seg_col<false>(lane, j);
                r[j] = c < cols ? __float_as_uint(load_one<BF16>(p, c)) : 0u;
            }
        } else {
            load_pieces<FULL>(p, c0, cols, lane);
        }
    }
    template <bool FULL>
    __device__ __forceinline__ void load_pieces(const void* p, int c0, int cols, int lane) {
        if (!VEC && !FULL && c0 + kSeg <= cols) return load_pieces<true>(p, c0, cols, lane);
        const int left = cols - c0 - 8 * lane;
        const char* at = static_cast<const char*>(p) + (long long)(c0 + 8 * lane) * kSize;
        if (VEC && (FULL || left >= 8)) {
            const uint4* q = reinterpret_cast<const uint4*>(at);
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 a = q[i];
                r[4 * i] = a.x, r[4 * i + 1] = a.y, r[4 * i + 2] = a.z, r[4 * i + 3] = a.w;
            }
        } else if (FULL || left > 0) {
            // the aligned pieces that hold the values; the last one again where there are fewer
            constexpr int kPieces = kWords / 4 + (VEC ? 0 : 1);
            const int shift = VEC ? 0 : (int)(reinterpret_cast<uintptr_t>(at) & 15);
            const int last = (shift + (FULL ? 8 : min(left, 8)) * kSize - 1) & ~15;
            uint32_t w[4 * kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const uint4 a = *reinterpret_cast<const uint4*>(at - shift + min(16 * i, last));
                w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
            }
            if (!VEC) words_down<BF16>(w, shift);
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                r[i] = w[i];
                if (!FULL && BF16) r[i] &= left > 2 * i + 1 ? 0xffffffffu : left > 2 * i ? 0xffffu : 0u;
                if (!FULL && !BF16 && left <= i) r[i] = 0u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) r[i] = 0u;
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

// Stores the segment's values below `cols`.  Every lane of the warp takes part.  Shifted: a lane stores
// the aligned piece (fp32: two) that begins in the lane below it, with the values that reach into it
// from there; the segment's ragged ends go value by value.
template <bool BF16, int MODE, bool FULL = false>
__device__ __forceinline__ void seg_store(void* p, int c0, int cols, int lane, const float (&v)[8]) {
    if constexpr (MODE == kByValue) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = c0 + seg_col<false>(lane, j);
            if (c < cols) store_one<BF16>(p, c, v[j]);
        }
        return;
    }
    if (MODE == kShifted && !FULL && c0 + kSeg <= cols) return seg_store<BF16, MODE, true>(p, c0, cols, lane, v);
    constexpr int kWords = BF16 ? 4 : 8, kSize = BF16 ? 2 : 4;
    uint32_t own[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) own[i] = BF16 ? bf16_pair(v[2 * i], v[2 * i + 1]) : __float_as_uint(v[i]);
    const int c = c0 + 8 * lane;
    char* at = static_cast<char*>(p) + (long long)c * kSize;
    auto one = [&](char* to, uint32_t word, int j) {
        if (BF16)
            *reinterpret_cast<uint16_t*>(to + 2 * j) = (uint16_t)(j & 1 ? word >> 16 : word);
        else
            *reinterpret_cast<uint32_t*>(to + 4 * j) = word;
    };
    if (MODE == kAligned) {
        if (FULL || c + 8 <= cols) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                reinterpret_cast<uint4*>(at)[i] = make_uint4(own[4 * i], own[4 * i + 1], own[4 * i + 2], own[4 * i + 3]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < cols) one(at, own[BF16 ? j >> 1 : j], j);
        }
        return;
    }
    const int shift = (int)(reinterpret_cast<uintptr_t>(p) & 15);   // of every lane's values
    const int back = shift / kSize;   // values of the lane below in this lane's pieces
    uint32_t w[kWords + 4];           // the lane below's last 16 bytes, then this one's
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(0xffffffffu, own[kWords - 4 + i], 1);
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[4 + i] = own[i];
    // the pieces begin 16 - shift bytes into w; for 0 they are this lane's own
    words_down<BF16>(w, shift ? 16 - shift : 0);
    if (shift == 0) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = own[i];
    }
    const bool whole = (lane > 0 || shift == 0) && (FULL || c - back + 8 <= cols);
    if (whole) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i)
            reinterpret_cast<uint4*>(at - shift)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    // the values outside those pieces: lane 0's first 8 - back and lane 31's last, one per lane
    const int from = lane < 8 - back ? 0 : 31;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        const uint32_t x = __shfl_sync(0xffffffffu, own[i], from);
        if ((BF16 ? lane >> 1 : lane) == i) word = x;
    }
    const int e = c0 + 8 * from + lane;
    if (lane < 8 && shift != 0 && (FULL || e < cols))
        one(static_cast<char*>(p) + (long long)(e - lane) * kSize, word, lane);
    if (!FULL && !whole && (lane > 0 || shift == 0)) {   // the piece that holds the row's end
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c - back + j < cols) one(at - shift, w[BF16 ? j >> 1 : j], j);
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
        const int left = cols - c0 - 8 * lane;
        if (FULL || left >= 8) {
            *reinterpret_cast<uint2*>(codes + 8 * lane) = make_uint2(lo, hi);
        } else {   // the row's end: what follows may be another's
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < left) codes[8 * lane + j] = (uint8_t)((j < 4 ? lo : hi) >> 8 * (j & 3));
        }
        if ((FULL || left > 0) && (lane & 3) == 0) scales[lane >> 2] = (uint8_t)byte;
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
