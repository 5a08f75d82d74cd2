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
// fp32 accumulators in TMEM, double-buffered), persistent over the tiles.  Per CTA, 15 warps:
//   0      TMA of x: per step of 64 tokens its 128 columns' codes (8 KB) and scales (1 KB)
//   1      MMA issue (the even CTA's) and TMEM allocation
//   2      TMA of dy: its 128 columns (16 KB per step)
//   3-10   conversion of x into a 16 KB bf16 operand per step, four steps at a time
//   11-14  epilogue: column scale, addition to grad, stores
// Two rings: x as it arrives (full_r by TMA, empty_r by the conversion), and the operands (dy
// and converted x; ready, on the even CTA, by both CTAs' conversion warps, the odd one's through
// copies of 16 bytes, and dy's TMA bytes, empty, on both, by the MMAs), so the MMA warp has one
// wait and one commit per step.
//
// What bounds it: shared memory.  A step moves 82 KB through each SM's 128 bytes a cycle (MMA
// operands 32 KB, dy in 16 KB, codes in and out 18 KB, converted x 16 KB), 640 cycles where its
// MMAs take 512.  Under the profiler at 8192 tokens x 3584 x 3584 the tensor pipe is busy 70 % of
// the cycles with work and the shared-memory pipe 95 %, a part of it for the chains' sums (kChain).
// Measured: 159 us there (1320 TFLOP/s; 196 tiles are 2.6 turns of the 76 pairs), 1500 us at 16384 x
// 18944 x 3584 with fp32 or bf16 gradients (1480 TFLOP/s, 78 % of the measured burst rate of a library
// product, under the power cap).  256 x 256 is the largest tile whose accumulators fit TMEM twice, so
// that an epilogue overlaps the next tile.  Weights of few tokens are bound by the epilogue: 32 experts
// of 1024 x 2048 with 64 tokens each take 42 us, 21 of them HBM's for the gradients.
#include <cuda.h>
#include <cuda_bf16.h>

#include "act8.cuh"
#include "kernels.h"
#include "plan.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kWgStepT = 64;            // tokens per step
constexpr int kRingM = 4;               // steps of MMA operands
constexpr int kRingR = 8;               // steps of x as it arrives
// Steps in conversion at a time: the way from a landed step to its arrival at the MMA warp takes a
// warp about 2000 cycles, four times a step's MMAs (183 us with two groups, 148 with four).
constexpr int kConvGroups = 4;
constexpr int kConvFirst = 3;           // first conversion warp
constexpr int kWgEpiWarps = 4;
// Warps by whether dy comes by TMA or is copied by the conversion warps, which are then twice as many
// (8192 x 3585 x 3584: 298 us; 434 with eight; 335-365 since bf16 gradients add up chains: with 80
// registers a thread their epilogue spills).
template <bool TMA_Y>
struct Roles {
    static constexpr int kConvWarps = TMA_Y ? 8 : 16;
    static constexpr int kGroupWarps = kConvWarps / kConvGroups;
    static constexpr int kRows = kWgStepT / kGroupWarps;   // token rows per conversion warp and step
    static constexpr int kEpiFirst = kConvFirst + kConvWarps;
    static constexpr int kThreads = 32 * (kEpiFirst + kWgEpiWarps);
    static_assert(kRows % 8 == 0, "whole passes");
};
// Tokens that one accumulator takes.  The tensor cores' adds truncate, so its sum drifts in proportion to
// them: by 1.1e-5 of itself over 16384 tokens of random data, by 1.3 % over 2^21 tokens of one sign.  The
// epilogue adds up the chains' sums in fp32 instead: fp32 gradients in place, bf16 ones in the workspace.
// That leaves 8.4e-7 (an fp32 product on the CUDA cores: 6.9e-7) and costs an fp32 gradient 7 % (16384 x
// 18944 x 3584: 1437 -> 1541 us; chains of 4096 tokens: 2e-6, 1470 us), a bf16 one 10 % (there 1348 ->
// 1513 us, 8192 x 3584 x 3584 134 -> 147, back to back).
constexpr uint32_t kChain = 2048;
constexpr int kBandM = 8;               // tiles along m whose columns of dy are in flight together
constexpr int kSortGroups = 256;        // experts that are dealt out by their number of tokens
constexpr int kTurnTable = 96;          // turns decoded at the start
// A ring slot is always converted by the same warps, which so see every phase of its barriers.
static_assert(kRingR % kConvGroups == 0 && kRingM % kConvGroups == 0, "ring sizes");

struct WgCfg {
    static constexpr int A_BYTES = 128 * kWgStepT * 2;      // 128 columns of dy, or of x in bf16
    static constexpr int RAW_BYTES = 128 * kWgStepT;
    static constexpr int SCALE_BYTES = 16 * kWgStepT;
    static constexpr int R_BYTES = RAW_BYTES + SCALE_BYTES;
    static constexpr int CHUNK_BYTES = 64 * kWgStepT * 2;   // 64 columns of an MN-major operand
    static constexpr int SLOT_BYTES = 2 * A_BYTES;          // dy, then x
    static constexpr int R_OFFSET = kRingM * SLOT_BYTES;
    static constexpr int OUT_OFFSET = R_OFFSET + kRingR * R_BYTES;
    static constexpr int OUT_LD = 144;                      // row of a 32 x 32 block of floats, padded by 16 bytes
    static constexpr int OUT_WARP = 32 * OUT_LD;
    static constexpr int BAR_OFFSET = OUT_OFFSET + kWgEpiWarps * OUT_WARP;
    static constexpr int SIGNAL_OFFSET = BAR_OFFSET + 512;   // 16 bytes per conversion warp
    static constexpr int EXPERTS_OFFSET = SIGNAL_OFFSET + 256;
    static constexpr int TABLE_OFFSET = EXPERTS_OFFSET + kSortGroups * 10;
    static constexpr int SMEM_BYTES = TABLE_OFFSET + kTurnTable * 32 + 1024;
};
static_assert(WgCfg::SMEM_BYTES <= 232448, "weight-gradient kernel exceeds the shared memory of one CTA");

// Division of whole numbers below 2^31 by a divisor known at launch: with 2^(32 + s) / d rounded
// up to the 33 bits 2^32 + m, n / d = (n + floor(n m / 2^32)) / 2^s (Granlund and Montgomery,
// "Division by invariant integers using multiplication").  A tile's decoding is a chain of them.
struct Divisor {
    uint32_t d, m;
    int s;
    __host__ void set(uint32_t divisor) {
        d = divisor;
        s = 0;
        while ((1ull << s) < d) ++s;
        m = (uint32_t)(((((1ull << s) - d) << 32) / d) + 1);
    }
    __device__ __forceinline__ int div(int n) const {
        return (int)(((unsigned long long)(uint32_t)n + __umulhi((uint32_t)n, m)) >> s);
    }
};

struct WgradLaunch {
    CUtensorMap map_y, map_x, map_s;
    WgradArgs a;
    int tiles_m, tiles_n;
    Divisor tiles, band, wide_band, last_band, part;   // by tiles of a weight, of a band, bands' widths, parts
    int units;                     // whole tiles of all groups, then parts of split tiles
    int whole, parts;              // units below `whole` are tiles, the others one of `parts` of a tile
    int wide;                      // rows of grad are aligned to four elements
    int sectors;                   // rows of a bf16 grad are aligned to 32 bytes
};

// Experts by decreasing number of tokens, built by every CTA when there are several (at most
// kSortGroups, else in their own order): dealt out in turns, equal tiles then meet in the same
// turn, and the last turns are the short ones.
struct Experts {
    int begin[kSortGroups], end[kSortGroups];
    uint16_t order[kSortGroups];
};

struct __align__(16) Unit {
    int m0, n0;
    int begin, end;             // tokens
    int group, tile, part, pad; // part < 0: the whole tile
};

__device__ __forceinline__ void expert_range(const WgradArgs& a, int g, int* begin, int* end) {   // tokens < 2^31
    *begin = min(max(a.offsets[g], 0), (int)a.tokens);
    *end = min(max(a.offsets[g + 1], *begin), (int)a.tokens);
}

__device__ __forceinline__ Unit decode_unit(const WgradLaunch& L, const Experts* ex, int u) {
    Unit r;
    r.part = -1;
    if (u >= L.whole) {
        const int v = u - L.whole, t = L.part.div(v);
        u = L.whole + t;
        r.part = v - t * L.parts;
    }
    r.tile = u;
    r.group = L.tiles.div(u);
    int t = u - r.group * (int)L.tiles.d;
    // bands of kBandM tiles along m, within a band along n: the tiles that run together share
    // both operands' columns in L2
    const int band = L.band.div(t);
    t -= band * (int)L.band.d;
    const bool full = (band + 1) * kBandM <= L.tiles_m;
    const int col = full ? L.wide_band.div(t) : L.last_band.div(t);
    r.m0 = (band * kBandM + t - col * (full ? kBandM : (int)L.last_band.d)) * 256;
    r.n0 = col * 256;
    r.begin = 0, r.end = (int)L.a.tokens;
    if (L.a.offsets) {
        if (L.a.groups <= kSortGroups) {
            r.group = ex->order[r.group];
            r.begin = ex->begin[r.group], r.end = ex->end[r.group];
        } else {
            expert_range(L.a, r.group, &r.begin, &r.end);
        }
    } else if (r.part >= 0) {
        const long long steps = (L.a.tokens + kWgStepT - 1) / kWgStepT;
        r.begin = (int)(steps * r.part / L.parts * kWgStepT);
        r.end = (int)min(steps * (r.part + 1) / L.parts * kWgStepT, L.a.tokens);
    }
    return r;
}
// The units of this CTA pair, one per turn.  Experts are dealt out by length: every other turn
// runs backwards, so that no pair gets the longest of each.  The first kTurnTable turns are decoded
// once, by all threads at the kernel's start: decoded by each role at each tile, they cost a tile
// of few tokens more than its product (about 1000 cycles, one after another).
struct Turns {
    int pair, pairs, count;
    bool snake;
    __device__ __forceinline__ explicit Turns(const WgradLaunch& L)
        : pair(blockIdx.x >> 1), pairs(gridDim.x >> 1), snake(L.a.offsets != nullptr) {
        count = L.units / pairs;
        count += unit(count) < L.units;
    }
    __device__ __forceinline__ int unit(int turn) const {
        return turn * pairs + (snake && (turn & 1) ? pairs - 1 - pair : pair);
    }
    __device__ __forceinline__ Unit get(const WgradLaunch& L, const Experts* ex, uint32_t table, int turn) const {
        if (turn >= kTurnTable) return decode_unit(L, ex, unit(turn));
        Unit u;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.m0), "=r"(u.n0), "=r"(u.begin), "=r"(u.end)
                     : "r"(table + turn * 32));
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.group), "=r"(u.tile), "=r"(u.part), "=r"(u.pad)
                     : "r"(table + turn * 32 + 16));
        return u;
    }
};

__device__ __forceinline__ int unit_steps(const Unit& u) {
    return (int)((uint32_t)(u.end - u.begin + kWgStepT - 1) / kWgStepT);
}

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
__device__ __forceinline__ float4 load_four(const char* p) {
    if (!BF16) return *reinterpret_cast<const float4*>(p);
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}
template <bool BF16>
__device__ __forceinline__ void store_four(char* p, const float* v) {
    if (BF16)
        *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
    else
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
// Adds to fp32 in global memory, without an answer.
__device__ __forceinline__ void red_four(void* p, const float* v) {
    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3])
                 : "memory");
}
__device__ __forceinline__ void red_one(void* p, float v) {
    asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(p), "f"(v) : "memory");
}
// A lane's 32 sums of a block of a part, 32 rows of 256 floats: as OutTile holds them.
template <bool WIDE>
__device__ __forceinline__ void part_load(const float* p, float (&f)[32]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (WIDE) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(p + i * 1024));
            f[4 * i] = x.x, f[4 * i + 1] = x.y, f[4 * i + 2] = x.z, f[4 * i + 3] = x.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[4 * i + j] = __ldcg(p + (4 * i + j) * 256);
        }
}
// The same, added to f: 16 at a time, which the epilogue of copied dy has registers for.
template <bool WIDE>
__device__ __forceinline__ void part_add(const float* p, float (&f)[32]) {
#pragma unroll
    for (int h = 0; h < 8; h += 4) {
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* q = p + (h + i) * 1024;
            x[i] = WIDE ? __ldcg(reinterpret_cast<const float4*>(q))
                        : make_float4(__ldcg(q), __ldcg(q + 256), __ldcg(q + 512), __ldcg(q + 768));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float* v = f + 4 * (h + i);
            v[0] += x[i].x, v[1] += x[i].y, v[2] += x[i].z, v[3] += x[i].w;
        }
    }
}
template <bool WIDE>
__device__ __forceinline__ void part_store(float* p, const float (&f)[32], bool more) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (WIDE) {
            if (more)
                red_four(p + i * 1024, f + 4 * i);
            else
                store_four<false>(reinterpret_cast<char*>(p + i * 1024), f + 4 * i);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (more)
                    red_one(p + (4 * i + j) * 256, f[4 * i + j]);
                else
                    p[(4 * i + j) * 256] = f[4 * i + j];
            }
        }
}

// One lane's share of a warp's 32 rows of a tile of grad, in blocks of 32 columns: 32 sums per
// block, as four columns (cl .. + 3) of eight rows (rl, rl + 4, ...) where the rows of grad are
// aligned to four elements (WIDE), else as one column (lane) of all rows; either way a warp
// touches 128-byte row pieces.  Addresses advance by additions: with one warp per scheduler
// here, a multiplication and a comparison per store cost 80 cycles each.
template <bool BF16, bool WIDE>
struct OutTile {
    static constexpr int kSize = BF16 ? 2 : 4;
    char* p;
    const float* scale;
    long long step;      // bytes from a row of this lane to its next
    int rows, cols;      // rows, and columns from this lane's first on, that exist
    bool add;
    __device__ __forceinline__ OutTile(const WgradLaunch& L, const Unit& w, int r0, int lane) : add(L.a.accumulate) {
        const int row = r0 + (WIDE ? lane >> 3 : 0), col = w.n0 + (WIDE ? 4 * (lane & 7) : lane);
        p = static_cast<char*>(L.a.grad) + (((long long)w.group * L.a.m + row) * L.a.n + col) * kSize;
        scale = L.a.col_scale ? L.a.col_scale + col : nullptr;
        step = (WIDE ? 4ll : 1ll) * L.a.n * kSize;
        rows = WIDE ? min(max((L.a.m - row + 3) / 4, 0), 8) : min(max(L.a.m - row, 0), 32);
        cols = L.a.n - col;
    }

    // f: the sums of the block at column c0 of the tile; times the column scale, and added to what
    // is there when the call accumulates or `more`.  fp32 is added by reductions in L2: the only
    // thread that writes an element issues them in program order, so the bits do not vary, and
    // no value travels to the SM and back (16384 x 18944 x 3584: 1614 -> 1541 us).
    __device__ __forceinline__ void put(float (&f)[32], int c0, bool more) const {
        if (c0 >= cols) return;
        more = more || add;
        char* to = p + c0 * kSize;
        if (WIDE) {   // n % 4 == 0: the four columns exist together
            if (scale) {
                const float s[4] = {scale[c0], scale[c0 + 1], scale[c0 + 2], scale[c0 + 3]};
#pragma unroll
                for (int i = 0; i < 32; ++i) f[i] *= s[i & 3];
            }
            if (more) {
                if (BF16) {   // half of the loads before their stores
#pragma unroll
                    for (int h = 0; h < 8; h += 4) {
                        float4 g[4];
                        char* from = to;
#pragma unroll
                        for (int i = 0; i < 4; ++i, from += step)
                            if (h + i < rows) g[i] = load_four<BF16>(from);
#pragma unroll
                        for (int i = 0; i < 4; ++i, to += step) {
                            float* v = f + 4 * (h + i);
                            v[0] += g[i].x, v[1] += g[i].y, v[2] += g[i].z, v[3] += g[i].w;
                            if (h + i < rows) store_four<BF16>(to, v);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i, to += step)
                        if (i < rows) red_four(to, f + 4 * i);
                }
                return;
            }
            if (rows == 8) {
#pragma unroll
                for (int i = 0; i < 8; ++i, to += step) store_four<BF16>(to, f + 4 * i);
                return;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i, to += step)
                if (i < rows) store_four<BF16>(to, f + 4 * i);
            return;
        }
        const float s = scale ? scale[c0] : 1.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i] *= s;
        if (more) {
            if (BF16) {
#pragma unroll
                for (int h = 0; h < 32; h += 8) {
                    float g[8];
                    char* from = to;
#pragma unroll
                    for (int i = 0; i < 8; ++i, from += step) g[i] = h + i < rows ? load_one<BF16>(from, 0) : 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i, to += step)
                        if (h + i < rows) store_one<BF16>(to, 0, f[h + i] + g[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i, to += step)
                    if (i < rows) red_one(to, f[i]);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i, to += step)
            if (i < rows) store_one<BF16>(to, 0, f[i]);
    }
};

__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t x) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}

// Eight token rows of dy (row .. row + 7 of the step at t0; zero from `left` on), columns m0 ..
// m0 + 127, into the swizzled operand when its rows are not 16-byte aligned: a lane makes 16
// bytes from the two aligned 16-byte pieces that hold them, two rows per pass.  Every piece
// loaded holds an element of the row; columns at and beyond m get whatever lies there and
// reach rows of the product that are not stored.
__device__ __forceinline__ void copy_rows(const WgradArgs& a, long long t0, int left, int m0, int row, uint32_t dst,
                                          int lane) {
    const int j = lane & 15, col = m0 + 8 * j;
    uint32_t v[4][8];
    int d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = row + 2 * i + (lane >> 4);
        const uintptr_t line = reinterpret_cast<uintptr_t>(a.dy) + (uintptr_t)((t0 + t) * a.lddy) * 2;
        const uintptr_t at = line + (uintptr_t)col * 2;
        d[i] = (int)(at & 15);
        const uint4* p = reinterpret_cast<const uint4*>(at & ~(uintptr_t)15);
        const bool live = t < left && col < a.m;
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (live) x = *p;
        if (live && d[i] && reinterpret_cast<uintptr_t>(p + 1) < line + (uintptr_t)a.m * 2) y = p[1];
        v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
        v[i][4] = y.x, v[i][5] = y.y, v[i][6] = y.z, v[i][7] = y.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = row + 2 * i + (lane >> 4);
#pragma unroll
        for (int k = 0; k < 6; ++k) v[i][k] = d[i] & 8 ? v[i][k + 2] : v[i][k];
#pragma unroll
        for (int k = 0; k < 5; ++k) v[i][k] = d[i] & 4 ? v[i][k + 1] : v[i][k];
        const int sh = 8 * (d[i] & 2);
        sts128(dst + (j >> 3) * WgCfg::CHUNK_BYTES + t * 128 + (((j & 7) ^ (t & 7)) << 4),
               make_uint4(__funnelshift_r(v[i][0], v[i][1], sh), __funnelshift_r(v[i][1], v[i][2], sh),
                          __funnelshift_r(v[i][2], v[i][3], sh), __funnelshift_r(v[i][3], v[i][4], sh)));
    }
}

struct EpilogueArgs {
    const Experts* ex;
    Turns turns;
    uint32_t table;
    uint32_t tmem_base, tempty_lead, blk;   // blk: this warp's staging block in shared memory
    uint64_t* tfull;
    volatile int* abort_flag;
    int q, wq, lane;
};

// Hands accumulator `acc` back to the MMA warp once this warp's last load from it is complete.  The
// arrival orders no memory: behind a release it would wait for the stores of grad.
__device__ __forceinline__ void release_tmem(const EpilogueArgs& e, uint32_t acc) {
    tc_fence_before();
    __syncwarp();
    if (e.lane == 0) mbar_arrive_remote_relaxed(e.tempty_lead + acc * 8);
}

// 32 aligned bytes: a whole sector from one lane.
__device__ __forceinline__ void store_sector(void* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// A bf16 tile that is only written, whole, to rows of 32-byte aligned sectors: each lane stores its
// TMEM lane's row, 32 columns at a time, without a detour through shared memory (32 experts of
// 1024 x 2048: 83 -> 73 us; the same through shared memory and TMA stores 78 us).
__device__ __forceinline__ void store_rows(const WgradLaunch& L, const Unit& w, const EpilogueArgs& e, uint32_t tbase,
                                           uint32_t acc) {
    const int row = w.m0 + 128 * e.q + 32 * e.wq + e.lane;
    char* to = static_cast<char*>(L.a.grad) + (((long long)w.group * L.a.m + row) * L.a.n + w.n0) * 2;
    const float* scale = L.a.col_scale ? L.a.col_scale + w.n0 : nullptr;
    uint32_t v[2][32];
    tmem_ld32(tbase, v[0]);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        tmem_ld_wait();
        if (c < 7)
            tmem_ld32(tbase + 32 * (c + 1), v[(c + 1) & 1]);
        else
            release_tmem(e, acc);
        uint32_t o[16];
#pragma unroll
        for (int j = 0; j < 32; j += 4) {   // undoes the operand's column order
            float f[4] = {__uint_as_float(v[c & 1][j]), __uint_as_float(v[c & 1][j + 2]), __uint_as_float(v[c & 1][j + 1]),
                          __uint_as_float(v[c & 1][j + 3])};
            if (scale) {
#pragma unroll
                for (int k = 0; k < 4; ++k) f[k] *= scale[32 * c + j + k];
            }
            o[j / 2] = bf16_pair(f[0], f[1]), o[j / 2 + 1] = bf16_pair(f[2], f[3]);
        }
        store_sector(to + 64 * c, o);
        store_sector(to + 64 * c + 32, o + 8);
    }
}

// One epilogue warp: TMEM lane quarter wq, 32 rows of the tile, each 32 x 32 block through
// shared memory into the layout of OutTile.
template <bool BF16, bool WIDE, bool DIRECT>
__device__ __forceinline__ void epilogue(const WgradLaunch& L, const EpilogueArgs& e) {
    const int rl = e.lane >> 3, cl = 4 * (e.lane & 7);
    int local = 0;
    bool ok = true;
    for (int turn = 0; ok && turn < e.turns.count; ++turn) {
        const Unit w = e.turns.get(L, e.ex, e.table, turn);
        const int chains = (int)(((uint32_t)(w.end - w.begin) + kChain - 1) / kChain);
        const int r0 = w.m0 + 128 * e.q + 32 * e.wq;
        if (chains == 0) {   // an expert without tokens
            const OutTile<BF16, WIDE> out(L, w, r0, e.lane);
            for (int c0 = 0; c0 < 256 && !L.a.accumulate; c0 += 32) {
                float f[32] = {};
                out.put(f, c0, false);
            }
            continue;
        }
        // a part's sums go to the workspace, this warp's 32 x 256 of them as row-major rows; so do those of
        // a bf16 tile until its last chain, to the pair's own tile there, which each warp uses again
        const long long mine = 4 * e.q + e.wq, at = WIDE ? rl * 256 + cl : e.lane;
        float* part = nullptr;
        if (w.part >= 0) part = L.a.partial + ((w.tile - L.whole) * 8ll + mine) * L.parts * 8192 + at;
        float* run = nullptr;
        if (BF16 && part == nullptr && chains > 1)
            run = L.a.partial + ((kMaxParts + e.turns.pair) * 8ll + mine) * 8192 + at;
        for (int ch = 0; ch < chains; ++ch) {
            const uint32_t acc = local & 1;
            if (!mbar_wait_idle(e.tfull + acc, local >> 1 & 1u, e.abort_flag, L.a.status, kStatusTimeoutEpilogue,
                                true)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t tbase = e.tmem_base + acc * 256 + (static_cast<uint32_t>(e.wq * 32) << 16);
            if (BF16 && WIDE && DIRECT && L.sectors && part == nullptr && run == nullptr && !L.a.accumulate &&
                w.n0 + 256 <= L.a.n && r0 + 32 <= L.a.m) {
                store_rows(L, w, e, tbase, acc);
                ++local;
                continue;
            }
            const OutTile<BF16, WIDE> out(L, w, r0, e.lane);
            for (int c0 = 0; c0 < 256; c0 += 32) {
                uint32_t v[32];
                tmem_ld32(tbase + c0, v);
                tmem_ld_wait();
                if (c0 == 256 - 32) release_tmem(e, acc);
#pragma unroll
                for (int j = 0; j < 32; j += 4)   // undoes the operand's column order
                    sts128(e.blk + e.lane * WgCfg::OUT_LD + j * 4, make_uint4(v[j], v[j + 2], v[j + 1], v[j + 3]));
                __syncwarp();
                float f[32];
                if (WIDE) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 x = lds128(e.blk + (rl + 4 * i) * WgCfg::OUT_LD + cl * 4);
                        f[4 * i] = __uint_as_float(x.x), f[4 * i + 1] = __uint_as_float(x.y);
                        f[4 * i + 2] = __uint_as_float(x.z), f[4 * i + 3] = __uint_as_float(x.w);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(lds32(e.blk + i * WgCfg::OUT_LD + e.lane * 4));
                }
                __syncwarp();
                if (run != nullptr && ch == chains - 1) part_add<WIDE>(run + c0, f);   // this thread's own sums
                float* to = part != nullptr ? part + w.part * 8192 : ch < chains - 1 ? run : nullptr;
                if (to != nullptr)
                    part_store<WIDE>(to + c0, f, ch > 0);
                else
                    out.put(f, c0, !BF16 && ch > 0);   // a later chain of tokens adds to what this warp wrote
            }
            ++local;
        }
        if (part != nullptr && ok) {   // the warp that comes last adds up all parts, in their order
            __threadfence();
            __syncwarp();
            int* count = L.a.counters + ((w.tile - L.whole) * 8 + 4 * e.q + e.wq);
            int seen = 0;
            if (e.lane == 0) seen = atomicAdd(count, 1);
            if (__shfl_sync(0xffffffffu, seen, 0) == L.parts - 1) {
                if (e.lane == 0) *count = 0;   // for the next call
                __threadfence();
                __syncwarp();   // all lanes' reads after lane 0's fence: the shuffle orders no memory
                const OutTile<BF16, WIDE> out(L, w, r0, e.lane);
                for (int c0 = 0; c0 < 256; c0 += 32) {
                    float f[32];
                    part_load<WIDE>(part + c0, f);
                    for (int k = 1; k < L.parts; ++k) {
                        float g[32];
                        part_load<WIDE>(part + k * 8192 + c0, g);
#pragma unroll
                        for (int i = 0; i < 32; ++i) f[i] += g[i];
                    }
                    out.put(f, c0, false);
                }
            }
        }
    }
}

// TMA_Y: dy's rows are 16-byte aligned and come by TMA; else the conversion warps copy them.
template <int FMT, bool TMA_Y, bool BF16>
__global__ void __launch_bounds__(Roles<TMA_Y>::kThreads) k_wgrad(const __grid_constant__ WgradLaunch L) {
    using Cfg = WgCfg;
    using R = Roles<TMA_Y>;
    constexpr int kGroupWarps = R::kGroupWarps, kRows = R::kRows, kEpiFirst = R::kEpiFirst, kWgThreads = R::kThreads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full_r = reinterpret_cast<uint64_t*>(smem + Cfg::BAR_OFFSET);
    uint64_t* empty_r = full_r + kRingR;
    uint64_t* ready = empty_r + kRingR;
    uint64_t* empty = ready + kRingM;
    uint64_t* tail = empty + kRingM;
    uint64_t* tfull = tail + kRingM;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t q = cluster_ctarank() & 1u;
    const bool leader = q == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kRingR; ++s) {
            mbar_init(full_r + s, 1);
            mbar_init(empty_r + s, kGroupWarps);
        }
        for (int s = 0; s < kRingM; ++s) {
            mbar_init(ready + s, 1 + kGroupWarps);
            mbar_init(empty + s, 1);
            mbar_init(tail + s, 1);
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

    Experts* ex = reinterpret_cast<Experts*>(smem + Cfg::EXPERTS_OFFSET);
    if (L.a.offsets && L.a.groups <= kSortGroups) {
        for (int g = threadIdx.x; g < L.a.groups; g += kWgThreads) {
            expert_range(L.a, g, &ex->begin[g], &ex->end[g]);
        }
        __syncthreads();
        for (int g = threadIdx.x; g < L.a.groups; g += kWgThreads) {
            const int n = ex->end[g] - ex->begin[g];
            int rank = 0;
            for (int h = 0; h < L.a.groups; ++h) {
                const int o = ex->end[h] - ex->begin[h];
                rank += o > n || (o == n && h < g);
            }
            ex->order[rank] = (uint16_t)g;
        }
        __syncthreads();
    }
    const Turns turns(L);
    const uint32_t table = smem_u32(smem + Cfg::TABLE_OFFSET);
    for (int t = threadIdx.x; t < min(turns.count, kTurnTable); t += kWgThreads)
        reinterpret_cast<Unit*>(smem + Cfg::TABLE_OFFSET)[t] = decode_unit(L, ex, turns.unit(t));
    __syncthreads();

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA of x
            uint32_t it = 0;
            bool ok = true;
            for (int turn = 0; ok && turn < turns.count; ++turn) {
                const Unit w = turns.get(L, ex, table, turn);
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
                    const int t0 = w.begin + k * kWgStepT;
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
        // The odd CTA has nothing to do here where dy is copied.  It must not wait either: nothing waits for it,
        // so the ring could pass it by two rounds, whose parity it takes for none.
        if (lane == 0 && (TMA_Y || leader)) {
            // ---------------- TMA of dy, completion on the even CTA's barrier
            uint32_t slot = 0, ph = 1;
            bool ok = true;
            for (int turn = 0; ok && turn < turns.count; ++turn) {
                const Unit w = turns.get(L, ex, table, turn);
                const int steps = unit_steps(w);
                const int ym = w.m0 + 128 * (int)q;
                for (int k = 0; k < steps; ++k) {
                    if (!mbar_wait_idle(empty + slot, ph, abort_flag, L.a.status, kStatusTimeoutProducer, true)) {
                        ok = false;
                        break;
                    }
                    const int t0 = w.begin + k * kWgStepT;
                    uint8_t* sa = smem + slot * Cfg::SLOT_BYTES;
                    if (!TMA_Y || w.end - t0 < kWgStepT) {
                        // the conversion warps fill it, or first see it land (tail) and zero the rows that
                        // belong to other experts
                        if (TMA_Y) {
                            mbar_arrive_expect_tx(tail + slot, Cfg::A_BYTES);
                            tma_load_2d(sa, &L.map_y, tail + slot, ym, t0);
                            tma_load_2d(sa + Cfg::CHUNK_BYTES, &L.map_y, tail + slot, ym + 64, t0);
                        }
                        if (leader) mbar_arrive_expect_tx(ready + slot, 16 * kGroupWarps);
                    } else {
                        const uint32_t fb = mapa_shared(smem_u32(ready + slot), 0);
                        if (leader) mbar_arrive_expect_tx(ready + slot, 2 * Cfg::A_BYTES + 16 * kGroupWarps);
                        tma_load_2d_pair(sa, &L.map_y, fb, ym, t0);
                        tma_load_2d_pair(sa + Cfg::CHUNK_BYTES, &L.map_y, fb, ym + 64, t0);
                    }
                    if (++slot == kRingM) slot = 0, ph ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        if (leader) {
            // ---------------- MMA issue.  The tensor cores queue few instructions, so what this warp
            // does between two steps' MMAs is time they may idle: the whole warp runs the loop, so that
            // addresses stay in uniform registers, one elected lane issues, and the next step's barrier
            // is tested before the step's last MMA is issued.
            const bool one = elect_one();
            uint32_t slot = 0, ph = 0;
            int local = 0;
            bool ok = true, next = false;
            constexpr uint32_t idesc = idesc_make(true, 256, 256, true, true);
            constexpr uint32_t kSlot = Cfg::SLOT_BYTES >> 4, kStep = 16 * 128 >> 4;   // of the address field
            const uint64_t ad0 = sdesc_sw128(smem_u32(smem), Cfg::CHUNK_BYTES, 1024);
            const uint64_t bd0 = sdesc_sw128(smem_u32(smem) + Cfg::A_BYTES, Cfg::CHUNK_BYTES, 1024);
            for (int turn = 0; ok && turn < turns.count; ++turn) {
                const Unit w = turns.get(L, ex, table, turn);
                const int steps = unit_steps(w), chain = kChain / kWgStepT;
                const int last = ((w.end - w.begin - 1) & (kWgStepT - 1)) / 16 + 1;   // MMAs of the last step
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
                    const int whole = k1 == steps && last < 4 ? k1 - 1 : k1;
                    for (int k = k0; k < k1; ++k) {
                        if (!next && !mbar_wait_cluster(ready + slot, ph, abort_flag, L.a.status,
                                                        kStatusTimeoutMma)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t ad = ad0 + slot * kSlot, bd = bd0 + slot * kSlot;
                        uint64_t* done = empty + slot;
                        if (++slot == kRingM) slot = 0, ph ^= 1u;
                        if (k < whole) {
                            if (one) {
                                mma_f16kind_pair(d, ad, bd, idesc, k != k0);
                                mma_f16kind_pair(d, ad + kStep, bd + kStep, idesc, 1);
                                mma_f16kind_pair(d, ad + 2 * kStep, bd + 2 * kStep, idesc, 1);
                            }
                            next = mbar_test_wait_cluster(ready + slot, ph);
                            if (one) {
                                mma_f16kind_pair(d, ad + 3 * kStep, bd + 3 * kStep, idesc, 1);
                                mma_commit_pair(done, 0x3);
                            }
                        } else {
                            if (one) {
                                for (int kk = 0; kk < last; ++kk)
                                    mma_f16kind_pair(d, ad + kk * kStep, bd + kk * kStep, idesc, (k - k0) | kk);
                                mma_commit_pair(done, 0x3);
                            }
                            next = false;
                        }
                    }
                    if (ok && one) mma_commit_pair(tfull + acc, 0x3);
                }
            }
            if (one) mma_commit_pair(drain, 0x1);
            const unsigned long long t0 = globaltimer_ns();
            while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
            }
            __syncwarp();
        }
    } else if (warp < kEpiFirst) {
        // ---------------- conversion: warp cw of the kGroupWarps that take every kConvGroups-th step
        const int cw = (warp - kConvFirst) % kGroupWarps;
        const uint32_t cg = (warp - kConvFirst) / kGroupWarps;
        const uint32_t ready_lead = mapa_shared(smem_u32(ready), 0);
        uint32_t it = 0, tail_ph = 0;   // tail_ph: phase bit of each slot's tail barrier
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
        for (int turn = 0; ok && turn < turns.count; ++turn) {
            const Unit w = turns.get(L, ex, table, turn);
            const int steps = unit_steps(w);
            const int off = ((w.n0 + 128 * (int)q) >> 5) & 15;   // the CTA's four of the 16 loaded scales
            for (int k = 0; k < steps; ++k, ++it) {
                const int left = min(kWgStepT, w.end - w.begin - k * kWgStepT);
                if (it % kConvGroups != cg) continue;
                const uint32_t r = it % kRingR, b = it % kRingM;
                const uint32_t sr = smem_u32(smem + Cfg::R_OFFSET + r * Cfg::R_BYTES);
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
                    raw[2 * i] = lds128(sr + i * 1024 + src0);
                    raw[2 * i + 1] = lds128(sr + i * 1024 + (src0 ^ 64));
                    sc[i] = lds32(sr + Cfg::RAW_BYTES + (row0 + 8 * i) * 16 + off);
                }
                if (left < kWgStepT) {
#pragma unroll
                    for (int i = 0; i < kRows / 8; ++i)
                        if (row0 + 8 * i >= left) raw[2 * i] = raw[2 * i + 1] = make_uint4(0, 0, 0, 0), sc[i] = 0;
                }
                if (!mbar_wait_idle(empty + b, (it / kRingM & 1u) ^ 1u, abort_flag, L.a.status,
                                    kStatusTimeoutProducer, true)) {
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
                if (!TMA_Y) {
                    const long long t0 = w.begin + (long long)k * kWgStepT;
                    for (int b0 = 0; b0 < kRows / 2; b0 += 4)
                        copy_rows(L.a, t0, left, w.m0 + 128 * (int)q, cw * kRows + 2 * b0, sa, lane);
                } else if (left < kWgStepT) {
                    // the rows that follow belong to other experts: zero, whatever they hold
                    if (!mbar_wait_idle(tail + b, tail_ph >> b & 1u, abort_flag, L.a.status, kStatusTimeoutProducer,
                                        false)) {
                        ok = false;
                        break;
                    }
                    tail_ph ^= 1u << b;
                    for (int t = max(left, cw * kRows); t < (cw + 1) * kRows; ++t) {
                        sts32(sa + t * 128 + lane * 4, 0);
                        sts32(sa + Cfg::CHUNK_BYTES + t * 128 + lane * 4, 0);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // writes visible to the MMAs
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(empty_r + r);
                    // The even CTA's MMAs read the odd CTA's operand too, so its arrival is a copy of 16
                    // bytes whose completion releases at cluster scope.  A thread that releases at that
                    // scope waits about 1800 cycles (238 against 156 us at 8192 tokens, 3584 x 3584; 369
                    // with one warp that passes the odd CTA's steps on).
                    if (leader)
                        mbar_arrive(ready + b);
                    else   // from and to this warp's 16 bytes, which mean nothing
                        bulk_signal(ready_lead + (Cfg::SIGNAL_OFFSET - Cfg::BAR_OFFSET - 16 * kRingR) +
                                        16 * (warp - kConvFirst),
                                    smem + Cfg::SIGNAL_OFFSET + 16 * (warp - kConvFirst), ready_lead + b * 8);
                }
            }
        }
    } else {
        // ---------------- epilogue
        EpilogueArgs e{ex, turns, table};
        e.tmem_base = tmem_base;
        e.tfull = tfull;
        e.tempty_lead = mapa_shared(smem_u32(tempty), 0);
        e.blk = smem_u32(smem + Cfg::OUT_OFFSET + (warp - kEpiFirst) * Cfg::OUT_WARP);
        e.abort_flag = abort_flag;
        e.q = (int)q, e.wq = warp & 3, e.lane = lane;
        if (L.wide)
            epilogue<BF16, true, TMA_Y>(L, e);
        else
            epilogue<BF16, false, TMA_Y>(L, e);
    }

    if (*abort_flag) {   // copies already issued signal the even CTA; give them time to land
        const unsigned long long t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
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
        {{k_wgrad<kE4M3, false, false>, k_wgrad<kE4M3, false, true>},
         {k_wgrad<kE4M3, true, false>, k_wgrad<kE4M3, true, true>}},
        {{k_wgrad<kInt8, false, false>, k_wgrad<kInt8, false, true>},
         {k_wgrad<kInt8, true, false>, k_wgrad<kInt8, true, true>}}};
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
    const int pairs = std::min(sm_count / 2, kMaxPairs);
    L.whole = (int)units;
    L.parts = 1;
    if (!a.offsets) {
        // The tiles of the last, incomplete turn (all tiles, when they are fewer than the CTA
        // pairs) are split along the tokens into the number of parts that is estimated fastest:
        // 0.3 us per step of 64 tokens, and joining about 5 us for each part.
        const int rest = (int)(units % pairs);
        const long long steps = (a.tokens + kWgStepT - 1) / kWgStepT;
        double best = 0.3 * steps;
        for (int p = 2; rest > 0 && p <= 8 && rest * p <= kMaxParts && p <= steps; ++p) {
            const double t = 0.3 * (double)((rest * p + pairs - 1) / pairs) * (double)((steps + p - 1) / p) + 5.0 * p;
            if (t < best) best = t, L.parts = p;
        }
        if (L.parts > 1) L.whole = (int)units - rest;
    }
    L.units = L.whole + ((int)units - L.whole) * L.parts;
    L.tiles.set(L.tiles_m * L.tiles_n);
    L.band.set(kBandM * L.tiles_n);
    L.wide_band.set(kBandM);
    L.last_band.set(std::max(L.tiles_m % kBandM, 1));
    L.part.set(L.parts);
    L.wide = a.n % 4 == 0 && (reinterpret_cast<uintptr_t>(a.grad) & (bf16_grad ? 7 : 15)) == 0;
    L.sectors = bf16_grad && a.n % 16 == 0 && (reinterpret_cast<uintptr_t>(a.grad) & 31) == 0;
    // TMA needs 16-byte aligned rows; x has them by its format
    const bool tma_y = ((reinterpret_cast<uintptr_t>(a.dy) | (uintptr_t)(a.lddy * 2)) & 15) == 0;
    if ((tma_y && !map_2d(&L.map_y, a.dy, false, a.m, a.tokens, a.lddy * 2, 64, true)) ||
        !map_2d(&L.map_x, a.x.codes, true, a.n, a.tokens, a.x.ldq, 128, true) ||
        !map_2d(&L.map_s, a.x.scales, true, (a.n + kActGroup - 1) / kActGroup, a.tokens, a.x.lds, 16, false))
        return cudaErrorInvalidValue;
    return launch_pdl_cluster(pick(a.x.format, tma_y, bf16_grad), dim3(2 * std::min(L.units, pairs)),
                              dim3(tma_y ? Roles<true>::kThreads : Roles<false>::kThreads), WgCfg::SMEM_BYTES,
                              s, 2u, L);
}

}  // namespace muon
