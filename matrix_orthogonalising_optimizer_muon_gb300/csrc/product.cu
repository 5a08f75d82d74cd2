// Products of tokens with weights, one weight or one per expert over its own range of tokens:
// y = x W^T, and the gradient of its input, dx = dy W.
//
// The weight is the M operand and the tokens are the N operand of the tensor cores: D^T = W x^T.  An
// expert's range ends anywhere, and N follows it in steps of 32 (M comes in 256 alone), so that short
// ranges cost their weights' bytes and little more.  Both operands are read as they are stored: tokens
// K-major; the weight K-major (y = x W^T contracts over its columns) or MN-major (dx = dy W contracts
// over its rows).
//
// A cluster of two CTAs computes tiles of 256 outputs x up to 256 tokens (tcgen05.mma.cta_group::2, fp32
// accumulators in TMEM, double-buffered).  Per CTA: warp 0 issues the TMA loads, warp 1 the MMAs (the
// even CTA's), warps 2-9 are the epilogue, two for each quarter of the TMEM lanes, on alternate blocks of 32
// tokens.  A step is 64 values of the contraction: 16 KB of the weight and up to 16 KB of tokens per CTA, in
// a ring of six (five: 2 % slower).
//
// What bounds it: the way from L2 to the SMs.  A step of a 256 x 256 tile takes 64 KB through it in 0.33 us, 15 TB/s
// over all pairs, about as long as its MMAs at the full clock; requests that bring later steps into L2 make it slower
// (the 32 experts below 65 us, 106 through TMA).  Measured: 8192 x 3584 x 3584 107 us (1970 TFLOP/s, 103 % of the
// measured burst rate of a library product), 16384 x 18944 x 3584 1160-1260 us under the power cap, eight experts of
// 18944 x 3584 over 16384 rows 1365 us.  32 experts of 1024 x 2048 over 16384 ragged rows 59 us: 308 tiles of 256
// outputs, low ones among them, whose steps cost their weight's 32 KB all the same, in five turns, and about 10 us
// around them (launch 2, set-up 0.6, plan 2.5, first loads 1, last epilogue 2).  Few rows are bound by the weights'
// bytes and those 10 us: 32 rows for 32 experts 28 us (HBM 20), eight rows for eight of them 11.5 (HBM 5), one row of
// one weight of 3584 x 3584 10.4 (HBM 3.8).
//
// How the work is dealt out (every CTA derives the same plan from the offsets): tiles in the order experts,
// bands of token tiles, outputs, token tiles, one per CTA pair and turn, so that the tiles in flight share
// operands in L2.  (A contiguous run of tiles per pair balances ragged experts better, but each operand is then
// read again a whole tile later, when L2 has lost it: 102 us against 64 for the 32 experts below.)  The last,
// incomplete turn may be cut along the contraction; its partial sums meet in the workspace, and the part that
// comes last adds them up in their order.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "act8.cuh"
#include "kernels.h"
#include "plan.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kStepK = 64;
constexpr int kRing = 6;
constexpr int kEpiFirst = 2, kEpi = 8;             // epilogue warps
constexpr int kThreads = 32 * (kEpiFirst + kEpi);
constexpr int kBins = 512;                         // experts are searched in at most this many bins
constexpr int kItems = 96;                         // items decoded at the start

struct Cfg {
    static constexpr int A_BYTES = 128 * kStepK * 2;
    static constexpr int CHUNK_BYTES = 64 * kStepK * 2;   // 64 outputs of an MN-major weight
    static constexpr int SLOT_BYTES = 2 * A_BYTES;
    static constexpr int OUT_OFFSET = kRing * SLOT_BYTES;
    static constexpr int OUT_WARP = 2048;                 // 32 outputs x 32 tokens in bf16
    static constexpr int BAR_OFFSET = OUT_OFFSET + kEpi * OUT_WARP;
    static constexpr int PLAN_OFFSET = BAR_OFFSET + 256;
    static constexpr int ITEM_OFFSET = PLAN_OFFSET + 4 * kBins * 4 + 2 * kBins * 2 + 416;
    static constexpr int SMEM_BYTES = ITEM_OFFSET + kItems * 32 + 1024;
};
static_assert(Cfg::SMEM_BYTES <= 232448, "product kernel exceeds the shared memory of one CTA");
static_assert(Cfg::ITEM_OFFSET % 16 == 0, "items are loaded 16 bytes at a time");

// Division of whole numbers below 2^31 by a divisor known at launch, as in wgrad.cu.
struct Divisor {
    uint32_t d, m;
    int s;
    __host__ void set(uint32_t divisor) {
        d = divisor;
        s = 0;
        while ((1ull << s) < d) ++s;
        m = (uint32_t)(((((1ull << s) - d) << 32) / d) + 1);
    }
    __host__ __device__ __forceinline__ int div(int n) const {
        return (int)(((unsigned long long)(uint32_t)n + ((unsigned long long)(uint32_t)n * m >> 32)) >> s);
    }
};

// What every thread knows of the launch's plan.
struct Outline {
    int cap, units, turns, stretches;   // greatest height of a tile, tiles, whole turns, stretches of the last
    int span, least;                    // steps of the last turn's tiles; of a part, the least
    int stride, bins;                   // experts per bin of Plan::tiles
};

struct ProductLaunch {
    CUtensorMap map_w, map_x[4];   // map_x: boxes of 128, 64, 32 and 16 tokens
    ProductArgs a;
    int out, k, steps, tiles_m;    // outputs, contraction, its steps, tiles along the outputs
    int wide;                      // rows of y are aligned to four elements
    int pairs, band;               // CTA pairs; token tiles whose outputs are taken before the next ones'
    Divisor by_tiles, by_band, by_pairs, by_steps;   // by tiles_m, band tiles_m, pairs, steps
    // one weight: the plan
    Outline outline;
    int count, height, start[kMaxPairs + 1];
};

// The launch's plan in shared memory.  Where there is more than one turn, experts are placed by decreasing height
// of their tiles (when they are at most kBins): the turns' tiles are then alike, and the last turn's are the lowest.
struct Plan {
    int tiles[kBins + 4];                     // token tiles before the expert, or the bin of experts, at each place
    int begin[kBins], end[kBins], count[kBins];   // of each expert (at most kBins): tokens and tiles
    uint16_t height[kBins], order[kBins];     // of each expert; the expert at each place
    int start[kMaxPairs + 4];   // begins of the pairs' stretches, in steps from the first tile of the last turn
    int next[12];                // places of the heights while they are dealt out
    int sums[4];                 // token tiles when they are at most 256, 128, 64 tokens high
    unsigned long long all;      // the last of them
    int pad[2];
};
static_assert(sizeof(Plan) == Cfg::ITEM_OFFSET - Cfg::PLAN_OFFSET, "plan's place");

struct __align__(16) Item {
    int m0, t0, end, group;    // first output, first token, end of the expert's tokens
    int k0, k1, n;             // steps, height in tokens (a multiple of 32)
    int part;                  // parts << 16 | part << 8 | first pair; 0: the whole sum
};

__device__ __forceinline__ void expert_range(const ProductArgs& a, int g, int* begin, int* end) {   // tokens < 2^31
    const int last = a.first + (int)a.tokens;
    *begin = a.offsets ? min(max(a.offsets[g], a.first), last) - a.first : 0;
    *end = a.offsets ? max(min(max(a.offsets[g + 1], a.first), last) - a.first, *begin) : (int)a.tokens;
}

// An expert's token tiles: as few as the greatest height allows, of equal height in steps of 32 (the last
// may be lower).
__host__ __device__ __forceinline__ void cut_range(int tokens, int cap, int* count, int* height) {
    const int n = (int)((uint32_t)(tokens + cap - 1) >> (cap == 256 ? 8 : cap == 128 ? 7 : 6));
    // 32 times the quotient rounded down, then up to what holds all tokens: at most twice, for the division's error
#ifdef __CUDA_ARCH__
    int h = (int)(__fdividef((float)tokens, (float)max(n, 1)) * 0.03125f) << 5;
#else
    int h = tokens / (n > 0 ? n : 1) / 32 * 32;
#endif
    if ((long long)h * n < tokens) h += 32;
    if ((long long)h * n < tokens) h += 32;
    *count = n, *height = h;
}

// Tile u of the launch, the whole of its sum.
__device__ __forceinline__ Item decode_unit(const ProductLaunch& L, const Plan& p, const Outline& o, int u) {
    Item it;
    const int v = L.by_tiles.div(u);
    int before = 0, count, height;
    if (o.stride > 1) {
        int lo = 0, hi = o.bins - 1;
        while (lo < hi) {   // the last bin whose tiles begin at or before v
            const int mid = (lo + hi + 1) >> 1;
            if (p.tiles[mid] <= v)
                lo = mid;
            else
                hi = mid - 1;
        }
        before = p.tiles[lo];
        it.group = lo * o.stride;
        for (;; ++it.group, before += count) {
            expert_range(L.a, it.group, &it.t0, &it.end);
            cut_range(it.end - it.t0, o.cap, &count, &height);
            if (before + count > v) break;
        }
    } else {
        int lo = 0;
        if (o.bins > 1) {
            int hi = o.bins - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.tiles[mid] <= v)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            before = p.tiles[lo];
            lo = p.order[lo];
        }
        it.group = lo, it.t0 = p.begin[lo], it.end = p.end[lo], count = p.count[lo], height = p.height[lo];
    }
    uint32_t r = u - before * L.tiles_m;
    int band = 0;
    if (count > L.band) {
        band = L.by_band.div((int)r);
        r -= band * L.band * L.tiles_m;
    }
    const uint32_t wide = min(L.band, count - band * L.band), m = r / wide;
    it.m0 = (int)m * 256, it.t0 += (band * L.band + (int)(r - m * wide)) * height;
    it.k0 = 0, it.k1 = L.steps, it.part = 0;
    it.n = min(height, (it.end - it.t0 + 31) & ~31);   // tokens < 2^31 - 4096
    return it;
}

// Places of the experts by decreasing height, those without tiles last: one warp.
__device__ __forceinline__ void order_experts(Plan& p, int groups, int lane) {
    if (lane < 12) p.next[lane] = 0;
    __syncwarp();
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {   // count the heights, then deal out the places
        for (int g0 = 0; g0 < groups; g0 += 32) {
            const int g = g0 + lane, key = g < groups ? 8 - (p.height[g] >> 5) : 9;
            const unsigned peers = __match_any_sync(0xffffffffu, key);
            const int rank = __popc(peers & ((1u << lane) - 1)), at = p.next[key] + rank;
            __syncwarp();
            if (rank == 0) p.next[key] += __popc(peers);
            __syncwarp();
            if (pass == 1 && g < groups) p.order[at] = (uint16_t)g;
        }
        if (pass == 0) {
            const int n = lane < 12 ? p.next[lane] : 0;
            int sum = n;
#pragma unroll
            for (int d = 1; d < 16; d *= 2) {
                const int x = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += x;
            }
            if (lane < 12) p.next[lane] = sum - n;
            __syncwarp();
        }
    }
}

// How tiles of at most 32 `high` tokens would be dealt out, and the time that takes, in 32 cycles.  A step takes as
// long as its MMAs, and 256 cycles for the weight's 16 KB besides.  The tiles of the last, incomplete turn are cut
// along the contraction into stretches of equal length, one per pair, where that saves more than joining the parts
// takes: about 24 steps' time and, to write and read them, 34 more for 256 tokens, all at the greatest height, though
// the last turn's tiles are the lowest where there are several turns (8 rows for eight of 32 experts, 32
// steps: 11.5 us whole, 12.6 cut; 16 rows of 18944 values, 296 steps: 61 whole, 30 cut).
struct Dealt {
    int units, whole, rest, time;
    bool cut;
    __host__ __device__ __forceinline__ Dealt(const ProductLaunch& L, int tiles, int high) {
        const int step = 8 + high, turn = L.steps * step;   // steps <= 2^14
        units = tiles * L.tiles_m;
        whole = L.by_pairs.div(units);
        rest = units - whole * L.pairs;
        const int joined = L.by_pairs.div(rest * turn) + (24 + 34 * high / 8) * step;
        cut = rest > 0 && joined < turn;
        // beyond 2^31 any height does
        const long long t = (long long)whole * turn + (cut ? joined : rest > 0 ? turn : 0);
        time = t < 0x7fffffff ? (int)t : 0x7fffffff;
    }
};

// n0, n1, n2: token tiles when they are at most 256, 128, 64 tokens high.  The greatest height is the fastest of these.
__host__ __device__ __forceinline__ Outline outline_of(const ProductLaunch& L, int n0, int n1, int n2) {
    Outline o;
    const int groups = L.a.groups;
    o.stride = (groups + kBins - 1) / kBins;
    o.bins = (groups + o.stride - 1) / o.stride;
    Dealt d(L, n2, 2);
    o.cap = 64;
    if (n1 < n2) {   // some expert has more than 64 tokens
        const Dealt e(L, n1, 4);
        if (e.time <= d.time) d = e, o.cap = 128;
    }
    if (n0 < n1) {
        const Dealt e(L, n0, 8);
        if (e.time <= d.time) d = e, o.cap = 256;
    }
    o.units = d.units;
    o.turns = d.whole + (d.rest > 0 && !d.cut);
    o.least = 2 + (o.cap >> 5);
    o.span = d.cut ? d.rest * L.steps : 0;
    o.stretches = d.cut ? (o.span >= o.least * L.pairs ? L.pairs : o.span >= o.least ? o.span / o.least : 1) : 0;
    return o;
}

// Begin of stretch i, in steps from the first tile of the last turn: parts of a tile have at least `edge` steps.
__host__ __device__ __forceinline__ int stretch_start(const ProductLaunch& L, const Outline& o, int i) {
    if (i == o.stretches) return o.span;
    int at = o.stretches == L.pairs ? L.by_pairs.div(o.span * i) : o.span * i / o.stretches;   // below 2^28
    const int edge = o.least < L.steps / 2 ? o.least : L.steps > 3 ? L.steps / 2 : 1;
    const int k = at - L.by_steps.div(at) * L.steps;
    if (k < edge)
        at -= k;
    else if (k > L.steps - edge)
        at += L.steps - k;
    return at;
}

// Fills the plan: all threads of the CTA.
__device__ __forceinline__ Outline make_plan(const ProductLaunch& L, Plan& p, int threads) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, groups = L.a.groups;
    if (!L.a.offsets) {   // one weight: the host knows it
        if (tid <= L.outline.stretches) p.start[tid] = L.start[tid];
        if (tid == 0) {
            p.begin[0] = 0, p.end[0] = (int)L.a.tokens;
            p.count[0] = L.count, p.height[0] = (uint16_t)L.height;
        }
        __syncthreads();
        return L.outline;
    }
    const bool few = groups <= kBins;
    if (tid < 4) p.sums[tid] = 0;
    if (tid == 0) p.all = 0;
    __syncthreads();
    int n0 = 0, n1 = 0, n2 = 0;
    for (int g = tid; g < groups; g += threads) {
        int b, e;
        expert_range(L.a, g, &b, &e);
        if (few) p.begin[g] = b, p.end[g] = e;
        n0 += (e - b + 255) >> 8, n1 += (e - b + 127) >> 7, n2 += (e - b + 63) >> 6;
    }
    // Offsets that decrease may give the experts many times the tokens that there are, and more tiles than can be
    // counted: they get none.
    const unsigned low = __reduce_add_sync(0xffffffffu, n2 & 0xffff), high = __reduce_add_sync(0xffffffffu, n2 >> 16);
    n0 = __reduce_add_sync(0xffffffffu, n0), n1 = __reduce_add_sync(0xffffffffu, n1);
    n2 = __reduce_add_sync(0xffffffffu, n2);
    if (lane == 0 && (low | high)) {
        atomicAdd(p.sums, n0), atomicAdd(p.sums + 1, n1), atomicAdd(p.sums + 2, n2);
        atomicAdd(&p.all, ((unsigned long long)high << 16) + low);
    }
    __syncthreads();
    const bool counted = p.all <= (unsigned long long)(L.a.tokens / 64 + groups);
    const Outline o = outline_of(L, counted ? p.sums[0] : 0, counted ? p.sums[1] : 0, counted ? p.sums[2] : 0);
    if (few) {
        for (int g = tid; g < groups; g += threads) {
            int count, height;
            cut_range(p.end[g] - p.begin[g], o.cap, &count, &height);
            p.count[g] = count, p.height[g] = (uint16_t)height, p.order[g] = (uint16_t)g;
        }
    } else {
        for (int b = tid; b < o.bins; b += threads) {
            int tiles = 0;
            for (int g = b * o.stride; g < min((b + 1) * o.stride, groups); ++g) {
                int begin, end, count, height;
                expert_range(L.a, g, &begin, &end);
                cut_range(end - begin, o.cap, &count, &height);
                tiles += count;
            }
            p.tiles[b] = tiles;
        }
    }
    if (warp == 1)
        for (int i = lane; o.stretches && i <= o.stretches; i += 32) p.start[i] = stretch_start(L, o, i);
    __syncthreads();
    if (o.bins > 1) {
        if (warp == 0) {
            if (few && o.units > L.pairs) {
                order_experts(p, groups, lane);
                __syncwarp();
            }
            int tiles = 0;
            for (int b0 = 0; b0 < o.bins; b0 += 32) {   // tiles of the places before
                const int b = b0 + lane, t = b >= o.bins ? 0 : few ? p.count[p.order[b]] : p.tiles[b];
                int sum = t;
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const int x = __shfl_up_sync(0xffffffffu, sum, d);
                    if (lane >= d) sum += x;
                }
                if (b < o.bins) p.tiles[b] = tiles + sum - t;
                tiles += __shfl_sync(0xffffffffu, sum, 31);
            }
        }
        __syncthreads();
    }
    return o;
}

// What a CTA pair does, one item per turn: whole tiles, every other turn backwards (pairs get high and low
// tiles alike), then its stretch of the last turn.
struct Items {
    int pair, pairs, turns, count;
    __device__ __forceinline__ Items(const ProductLaunch& L, const Plan& p, const Outline& o)
        : pair(blockIdx.x >> 1), pairs(L.pairs), turns(o.turns) {
        if (turns > 0 && unit_of(turns - 1) >= o.units) --turns;
        count = turns;
        if (pair < o.stretches && p.start[pair + 1] > p.start[pair])
            count += L.by_steps.div(p.start[pair + 1] - 1) - L.by_steps.div(p.start[pair]) + 1;
    }
    __device__ __forceinline__ int unit_of(int turn) const {
        return turn * pairs + (turn & 1 ? pairs - 1 - pair : pair);
    }
    __device__ __forceinline__ Item decode(const ProductLaunch& L, const Plan& p, const Outline& o, int turn) const {
        if (turn < turns) return decode_unit(L, p, o, unit_of(turn));
        const int from = p.start[pair], to = p.start[pair + 1];
        const int u = L.by_steps.div(from) + turn - turns, begin = u * L.steps, end = begin + L.steps;
        Item it = decode_unit(L, p, o, o.turns * pairs + u);
        it.k0 = max(from - begin, 0), it.k1 = min(to - begin, L.steps);
        if (it.k0 > 0 || it.k1 < L.steps) {
            int a = pair, z = pair;   // the pairs that have the tile's first and last steps
            while (p.start[a] > begin) --a;
            while (p.start[z + 1] < end) ++z;
            it.part = (z - a + 1) << 16 | (pair - a) << 8 | a;
        }
        return it;
    }
    __device__ __forceinline__ Item get(const ProductLaunch& L, const Plan& p, const Outline& o, uint32_t table,
                                        int turn) const {
        if (turn >= kItems) return decode(L, p, o, turn);
        Item u;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.m0), "=r"(u.t0), "=r"(u.end), "=r"(u.group)
                     : "r"(table + turn * 32));
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.k0), "=r"(u.k1), "=r"(u.n), "=r"(u.part)
                     : "r"(table + turn * 32 + 16));
        return u;
    }
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t x) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}

struct Epilogue {
    uint32_t tmem_base, tempty_lead, blk, table;
    uint64_t* tfull;
    volatile int* abort_flag;
    int q, wq, lane;
    int first;   // this warp's first block of tokens, every other of which are its
};

// Hands accumulator `acc` back to the MMA warp once this warp's last load from it is complete.
__device__ __forceinline__ void release_tmem(const Epilogue& e, uint32_t acc) {
    tc_fence_before();
    __syncwarp();
    if (e.lane == 0) mbar_arrive_remote_relaxed(e.tempty_lead + acc * 8);
}

// Stores a warp's 32 outputs x 32 tokens, f: this lane's output of each token.  Tokens t .. t + 31 below `end`.
// Aligned rows: pairs of tokens in bf16 through shared memory, from which a lane takes four outputs of two
// tokens; else a lane stores its output of each token, a warp 64 bytes of a row at a time.
__device__ __forceinline__ void store_block(const ProductLaunch& L, const Epilogue& e, const float (&f)[32], int c0,
                                            int t, int end) {
    char* y = static_cast<char*>(L.a.y);
    const uint32_t blk = e.blk;
    if (L.wide) {
        __syncwarp();   // the block before has been read
#pragma unroll
        for (int p = 0; p < 16; ++p) sts32(blk + p * 128 + e.lane * 4, bf16_pair(f[2 * p], f[2 * p + 1]));
        __syncwarp();
        const int p0 = e.lane >> 3, c = c0 + 4 * (e.lane & 7);
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = lds128(blk + (p0 + 4 * i) * 128 + (e.lane & 7) * 16);
        char* to = y + ((long long)(t + 2 * p0) * L.a.ldy + c) * 2;
        const long long pitch = L.a.ldy * 2;
        if (c < L.out) {
#pragma unroll
            for (int i = 0; i < 4; ++i, to += 8 * pitch) {
                const int r = t + 2 * (p0 + 4 * i);
                if (r < end)
                    *reinterpret_cast<uint2*>(to) =
                        make_uint2(__byte_perm(x[i].x, x[i].y, 0x5410), __byte_perm(x[i].z, x[i].w, 0x5410));
                if (r + 1 < end)
                    *reinterpret_cast<uint2*>(to + pitch) =
                        make_uint2(__byte_perm(x[i].x, x[i].y, 0x7632), __byte_perm(x[i].z, x[i].w, 0x7632));
            }
        }
    } else {
        const int c = c0 + e.lane;
        char* to = y + ((long long)t * L.a.ldy + c) * 2;
        if (c < L.out) {
#pragma unroll
            for (int j = 0; j < 32; ++j, to += L.a.ldy * 2)
                if (t + j < end) *reinterpret_cast<__nv_bfloat16*>(to) = __float2bfloat16_rn(f[j]);
        }
    }
}

// A lane's 32 sums of a block in the workspace: 16 bytes per lane and access, neighbours side by side.
struct Block {
    float4 x[8];
    __device__ __forceinline__ void load(const float* p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __ldcg(reinterpret_cast<const float4*>(p + i * 128));
    }
    __device__ __forceinline__ void add_to(float (&f)[32]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[4 * i] += x[i].x, f[4 * i + 1] += x[i].y, f[4 * i + 2] += x[i].z, f[4 * i + 3] += x[i].w;
    }
};
__device__ __forceinline__ void part_store(float* p, const uint32_t (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4*>(p + i * 128) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// One epilogue warp: TMEM lane quarter wq, that is 32 outputs of a tile, and every block of tokens or every other.
__device__ __forceinline__ void epilogue(const ProductLaunch& L, const Plan& plan, const Outline& outline,
                                         const Items& items, const Epilogue& e) {
    int local = 0;
    for (int turn = 0; turn < items.count; ++turn, ++local) {
        const Item w = items.get(L, plan, outline, e.table, turn);
        const uint32_t acc = local & 1;
        if (!mbar_wait_idle(e.tfull + acc, local >> 1 & 1u, e.abort_flag, L.a.status, kStatusTimeoutEpilogue, true))
            return;
        tc_fence_after();
        const uint32_t tbase = e.tmem_base + acc * 256 + (static_cast<uint32_t>(e.wq * 32) << 16);
        const int c0 = w.m0 + 128 * e.q + 32 * e.wq;
        const int parts = w.part >> 16, part = w.part >> 8 & 255, first = w.part & 255;
        // a pair has at most two parts of tiles: one that begins inside its tile, one that begins with it (kJoinFloats)
        auto slot = [&](int k) {
            return L.a.partial + ((2 * (first + k) + (k == 0)) * 8ll + 4 * e.q + e.wq) * 8192 + e.lane * 4;
        };
        for (int c = e.first; c < w.n; c += 64) {
            uint32_t v[32];
            tmem_ld32(tbase + c, v);
            tmem_ld_wait();
            if (c + 64 >= w.n) release_tmem(e, acc);
            if (parts) {
                part_store(slot(part) + c * 32, v);
            } else {
                float f[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);
                store_block(L, e, f, c0, w.t0 + c, w.end);
            }
        }
        if (e.first >= w.n) {   // no block of this tile
            release_tmem(e, acc);
        } else if (parts) {
            int* count = L.a.counters + (first * 2 + e.q) * 8 + e.wq + (e.first >> 3);
            int seen = 0;
            __syncwarp();   // the warp's sums before lane 0's release
            if (e.lane == 0)
                asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(seen) : "l"(count) : "memory");
            if (__shfl_sync(0xffffffffu, seen, 0) == parts - 1) {   // the last part: all of them, in their order
                if (e.lane == 0) *count = 0;   // for the next call
                __syncwarp();   // all lanes' reads after lane 0's acquire: the shuffle orders no memory
                for (int c = e.first; c < w.n; c += 64) {
                    Block a;
                    a.load(slot(0) + c * 32);
                    float f[32] = {};
                    for (int k = 0; k < parts; ++k) {
                        const Block b = a;   // the next part is on its way while this one is added
                        if (k + 1 < parts) a.load(slot(k + 1) + c * 32);
                        b.add_to(f);
                    }
                    store_block(L, e, f, c0, w.t0 + c, w.end);
                }
            }
        }
    }
}

// MN: the weight is MN-major (dx = dy W).
template <bool MN>
__global__ void __launch_bounds__(kThreads) k_product(const __grid_constant__ ProductLaunch L) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::BAR_OFFSET);
    uint64_t* empty = full + kRing;
    uint64_t* tfull = empty + kRing;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    Plan& plan = *reinterpret_cast<Plan*>(smem + Cfg::PLAN_OFFSET);
    const uint32_t table = smem_u32(smem + Cfg::ITEM_OFFSET);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t q = cluster_ctarank() & 1u;
    const bool leader = q == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kRing; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull + a, 1);
            mbar_init(tempty + a, 2 * kEpi);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&L.map_w);
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
    const Outline outline = make_plan(L, plan, kThreads);
    const Items items(L, plan, outline);
    for (int t = threadIdx.x; t < min(items.count, kItems); t += kThreads)
        reinterpret_cast<Item*>(smem + Cfg::ITEM_OFFSET)[t] = items.decode(L, plan, outline, t);
    __syncthreads();

    if (warp == 0) {
        // ---------------- TMA, completion on the even CTA's barrier.  The whole warp runs the loop and one elected
        // lane issues (a loop of one lane alone: 64 us against 58 for the 32 experts' product; a second warp
        // for the tokens gains nothing more)
        const bool one = elect_one();
        uint32_t slot = 0, ph = 1;
        bool ok = true;
        for (int turn = 0; ok && turn < items.count; ++turn) {
            const Item w = items.get(L, plan, outline, table, turn);
            const int rows = w.n >> 1, t0 = w.t0 + (int)q * rows, m0 = w.m0 + 128 * (int)q;
            for (int k = w.k0; k < w.k1; ++k) {
                if (!mbar_wait_idle(empty + slot, ph, abort_flag, L.a.status, kStatusTimeoutProducer, true)) {
                    ok = false;
                    break;
                }
                if (one) {
                    uint8_t* to = smem + slot * Cfg::SLOT_BYTES;
                    const uint32_t fb = mapa_shared(smem_u32(full + slot), 0);
                    const int kk = k * kStepK;
                    if (leader) mbar_arrive_expect_tx(full + slot, 2 * (Cfg::A_BYTES + rows * 128));
                    if (MN) {
                        tma_load_3d_pair(to, &L.map_w, fb, m0, kk, w.group);
                        tma_load_3d_pair(to + Cfg::CHUNK_BYTES, &L.map_w, fb, m0 + 64, kk, w.group);
                    } else {
                        tma_load_3d_pair(to, &L.map_w, fb, kk, m0, w.group);
                    }
                    if (rows == 128) {
                        tma_load_2d_pair(to + Cfg::A_BYTES, &L.map_x[0], fb, kk, t0);
                    } else {
                        int at = 0;
#pragma unroll
                        for (int b = 1; b < 4; ++b) {
                            if (rows & (128 >> b)) {
                                tma_load_2d_pair(to + Cfg::A_BYTES + at * 128, &L.map_x[b], fb, kk, t0 + at);
                                at += 128 >> b;
                            }
                        }
                    }
                }
                if (++slot == kRing) slot = 0, ph ^= 1u;
            }
        }
    } else if (warp == 1) {
        if (leader) {
            // ---------------- MMA issue: the whole warp runs the loop, so that addresses stay in uniform
            // registers, one elected lane issues, and the next step's barrier is tested before the step's last
            // MMA is issued
            const bool one = elect_one();
            uint32_t slot = 0, ph = 0;
            int local = 0;
            bool ok = true, next = false;
            constexpr uint32_t kSlot = Cfg::SLOT_BYTES >> 4;             // of the address field
            constexpr uint32_t kA = MN ? 16 * 128 >> 4 : 32 >> 4, kB = 32 >> 4;
            const uint64_t ad0 = sdesc_sw128(smem_u32(smem), MN ? Cfg::CHUNK_BYTES : 16, 1024);
            const uint64_t bd0 = sdesc_sw128(smem_u32(smem) + Cfg::A_BYTES, 16, 1024);
            const int last = ((L.k - 1) & (kStepK - 1)) / 16 + 1;        // MMAs of the contraction's last step
            for (int turn = 0; ok && turn < items.count; ++turn, ++local) {
                const Item w = items.get(L, plan, outline, table, turn);
                const uint32_t idesc = idesc_make(true, 256, w.n, MN, false);
                const uint32_t acc = local & 1;
                if (!mbar_wait_idle(tempty + acc, (local >> 1 & 1u) ^ 1u, abort_flag, L.a.status, kStatusTimeoutMma,
                                    true)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + acc * 256;
                const int whole = w.k1 == L.steps && last < 4 ? w.k1 - 1 : w.k1;
                for (int k = w.k0; k < w.k1; ++k) {
                    if (!next && !mbar_wait_cluster(full + slot, ph, abort_flag, L.a.status, kStatusTimeoutMma)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = ad0 + slot * kSlot, bd = bd0 + slot * kSlot;
                    uint64_t* done = empty + slot;
                    if (++slot == kRing) slot = 0, ph ^= 1u;
                    if (k < whole) {
                        if (one) {
                            mma_f16kind_pair(d, ad, bd, idesc, k != w.k0);
                            mma_f16kind_pair(d, ad + kA, bd + kB, idesc, 1);
                            mma_f16kind_pair(d, ad + 2 * kA, bd + 2 * kB, idesc, 1);
                        }
                        next = mbar_test_wait_cluster(full + slot, ph);
                        if (one) {
                            mma_f16kind_pair(d, ad + 3 * kA, bd + 3 * kB, idesc, 1);
                            mma_commit_pair(done, 0x3);
                        }
                    } else {
                        if (one) {
                            for (int kk = 0; kk < last; ++kk)
                                mma_f16kind_pair(d, ad + kk * kA, bd + kk * kB, idesc, (k - w.k0) | kk);
                            mma_commit_pair(done, 0x3);
                        }
                        next = false;
                    }
                }
                if (ok && one) mma_commit_pair(tfull + acc, 0x3);
            }
            if (one) mma_commit_pair(drain, 0x1);
            const unsigned long long t0 = globaltimer_ns();
            while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
            }
            __syncwarp();
        }
    } else {
        // ---------------- epilogue
        Epilogue e;
        e.tmem_base = tmem_base;
        e.tempty_lead = mapa_shared(smem_u32(tempty), 0);
        e.blk = smem_u32(smem + Cfg::OUT_OFFSET + (warp - kEpiFirst) * Cfg::OUT_WARP);
        e.table = table;
        e.tfull = tfull;
        e.abort_flag = abort_flag;
        e.q = (int)q, e.wq = warp & 3, e.lane = lane;
        e.first = (warp - kEpiFirst) / 4 * 32;
        epilogue(L, plan, outline, items, e);
    }

    __syncwarp();
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

bool map_tokens(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint64_t pitch, uint32_t box_rows) {
    muon_impl::EncodeTiledFn fn = muon_impl::encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {pitch};
    cuuint32_t box[2] = {kStepK, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ------------------------------------------------------------------ rows that TMA cannot read
// TMA takes rows whose addresses are multiples of 16 bytes.  Others are first copied into aligned rows in the
// workspace, chunk by chunk where they do not fit: 8192 x 3584 x 3585 takes 137 us, its aligned neighbour 107 (358 to
// 396 when warps of the product itself copied each operand of each tile through shifts, bound by the latency of that
// way however they were arranged).  The copy is bound by HBM, 5 TB/s read and written.
struct Job {
    const char* src;
    char* dst;
    long long pitch;       // of src, bytes
    uint32_t dst_pitch;    // a multiple of 128
    int bytes;             // of a row
    int pieces;            // 16 bytes each, of all rows
    Divisor by_row;        // pieces of a row
    Divisor by_expert;     // rows of each expert, of which those without tokens are left out; d 0: all rows
};
struct AlignArgs {
    Job job[2];
    int blocks;            // of the first job; the others are the second's
    ProductArgs a;
};

// A lane makes 16 bytes from the two aligned pieces that hold them, of which each holds a value of the row.
constexpr int kAlignThreads = 256, kAlignUnroll = 4;
__global__ void __launch_bounds__(kAlignThreads) k_align_rows(const AlignArgs args) {
    pdl_trigger();
    pdl_wait();
    const bool second = (int)blockIdx.x >= args.blocks;
    const Job& j = args.job[second];
    const int block = second ? blockIdx.x - args.blocks : blockIdx.x;
    const int blocks = second ? gridDim.x - args.blocks : args.blocks;
    constexpr int kBlock = kAlignThreads * kAlignUnroll;
    for (long long p0 = (long long)block * kBlock + threadIdx.x; p0 < j.pieces; p0 += (long long)blocks * kBlock) {
        uint32_t v[kAlignUnroll][8];
        int d[kAlignUnroll];
        char* to[kAlignUnroll];
#pragma unroll
        for (int k = 0; k < kAlignUnroll; ++k) {
            const long long p = p0 + k * kAlignThreads;
            const int row = p < j.pieces ? j.by_row.div((int)p) : 0, at = ((int)p - row * (int)j.by_row.d) * 16;
            bool live = p < j.pieces;
            if (live && j.by_expert.d) {
                int begin, end;
                expert_range(args.a, j.by_expert.div(row), &begin, &end);
                live = begin < end;
            }
            const char* line = j.src + row * j.pitch;
            d[k] = (int)(reinterpret_cast<uintptr_t>(line) & 15);
            const uint4* q = reinterpret_cast<const uint4*>(line + at - d[k]);
            uint4 x = make_uint4(0, 0, 0, 0), y = x;
            if (live) x = q[0];
            if (live && d[k] && reinterpret_cast<const char*>(q + 1) < line + j.bytes) y = q[1];
            v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
            v[k][4] = y.x, v[k][5] = y.y, v[k][6] = y.z, v[k][7] = y.w;
            to[k] = live ? j.dst + (uint64_t)row * j.dst_pitch + at : nullptr;
        }
#pragma unroll
        for (int k = 0; k < kAlignUnroll; ++k) {
            words_down<true>(v[k], d[k]);
            if (to[k]) *reinterpret_cast<uint4*>(to[k]) = make_uint4(v[k][0], v[k][1], v[k][2], v[k][3]);
        }
    }
}

typedef void (*ProductKernel)(ProductLaunch);
ProductKernel pick(bool mn) { return mn ? k_product<true> : k_product<false>; }

// A product whose rows are aligned: of a.groups weights whose rows are `pitch` elements apart, `out` outputs.
cudaError_t launch_aligned(const ProductArgs& a, int out, long long pitch, int sm_count, cudaStream_t s) {
    ProductLaunch L;
    L.a = a;
    L.out = out;
    L.k = a.transposed ? a.m : a.n;
    L.steps = (L.k + kStepK - 1) / kStepK;
    L.tiles_m = (L.out + 255) / 256;
    if ((a.tokens / 64 + a.groups) * L.tiles_m >= (1ll << 31)) return cudaErrorInvalidValue;
    L.pairs = std::min(sm_count / 2, kMaxPairs);
    // A wider band reads the weight fewer times, as long as its tokens stay in L2 (16 tiles of 4096 values: 32 MB):
    // eight experts of 18944 x 3584 1365 us with 16 and 1397 with eight, 8192 x 8192 x 8192 592 and 580.
    L.band = L.k <= 4096 ? 16 : 8;
    L.by_tiles.set(L.tiles_m), L.by_band.set(L.band * L.tiles_m), L.by_pairs.set(L.pairs), L.by_steps.set(L.steps);
    if (!a.offsets) {
        const int t = (int)a.tokens;
        L.outline = outline_of(L, (int)((t + 255ll) >> 8), (int)((t + 127ll) >> 7), (int)((t + 63ll) >> 6));
        cut_range(t, L.outline.cap, &L.count, &L.height);
        for (int i = 0; L.outline.stretches && i <= L.outline.stretches; ++i)
            L.start[i] = stretch_start(L, L.outline, i);
    }
    L.wide = L.out % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.y) | (uintptr_t)(a.ldy * 2)) & 7) == 0;
    // weights: rows of the contraction or of the outputs
    if (!muon_impl::make_map(&L.map_w, const_cast<void*>(a.weight), true, a.transposed ? out : a.n,
                             a.transposed ? a.m : out, a.groups, pitch, 64, a.transposed ? 64 : 128))
        return cudaErrorInvalidValue;
    for (int b = 0; b < 4; ++b)
        if (!map_tokens(&L.map_x[b], a.x, L.k, a.tokens, a.ldx * 2, 128 >> b)) return cudaErrorInvalidValue;
    return launch_pdl_cluster(pick(a.transposed), dim3(2 * L.pairs), dim3(kThreads),
                              Cfg::SMEM_BYTES, s, 2u, L);
}

// Rows begin at multiples of 128 bytes, so that a box's rows are whole lines of L2.
long long aligned_pitch(long long cols) { return muon_impl::round_up(cols, 64); }
// As many units of `size` elements as fit into `room`, of `all`: a multiple of 256 or, where fewer fit, of 64; 0 where
// not even those do.
long long chunk_of(long long all, long long size, long long room) {
    const long long n = room / size;
    return n >= muon_impl::round_up(all, 64) ? all : n >= 256 ? n / 256 * 256 : n / 64 * 64;
}
void set_job(Job* j, const void* src, long long pitch, void* dst, long long dst_pitch, long long rows, int cols) {
    j->src = static_cast<const char*>(src), j->dst = static_cast<char*>(dst), j->pitch = pitch * 2;
    j->dst_pitch = (uint32_t)(dst_pitch * 2), j->bytes = cols * 2;
    j->by_row.set((uint32_t)((cols + 7) / 8));
    j->pieces = (int)(rows * ((cols + 7) / 8));   // within the room
}
static_assert((kSharedRoom + kAlignedBytes) / 2 / 2 >= 1ll << 26, "64 rows of 2^20 elements of each operand: any product fits");

// What is copied, and in which pieces.
struct Pieces {
    bool align_w, align_x;
    long long px, pw;                  // pitches of the copies, elements
    long long tokens, experts, outs;   // of a piece: experts, or the outputs of one that is too large
    long long used;                    // elements of the tokens' copies, behind which the weights' begin
    bool fit;

    explicit Pieces(const ProductArgs& a) {
        const int out = a.transposed ? a.n : a.m, k = a.transposed ? a.m : a.n;
        align_w = a.n % 8 != 0 || (reinterpret_cast<uintptr_t>(a.weight) & 15) != 0;
        align_x = ((reinterpret_cast<uintptr_t>(a.x) | (uintptr_t)(a.ldx * 2)) & 15) != 0;
        px = aligned_pitch(k), pw = aligned_pitch(a.n);
        const long long all = a.room / 2, each = a.m * pw, wish = align_w ? std::min(a.groups * each, all / 2) : 0;
        tokens = align_x ? chunk_of(a.tokens, px, all - wish) : a.tokens;
        used = align_x ? muon_impl::round_up(tokens * px, 128) : 0;
        experts = a.groups, outs = out;
        if (align_w) {
            experts = std::min<long long>((all - used) / each, a.groups);
            if (experts == 0) experts = 1, outs = chunk_of(out, a.transposed ? a.m : pw, all - used);
        }
        fit = tokens > 0 && outs > 0;
    }
};

}  // namespace

cudaError_t product_prepare() {
    for (int i = 0; i < 2; ++i) {
        const cudaError_t e =
            cudaFuncSetAttribute(pick(i), cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

bool product_fits(const ProductArgs& a) { return Pieces(a).fit; }

cudaError_t launch_product(const ProductArgs& a, int sm_count, cudaStream_t s) {
    const int out = a.transposed ? a.n : a.m, k = a.transposed ? a.m : a.n;
    const Pieces p(a);
    const bool align_w = p.align_w, align_x = p.align_x;
    if (!align_w && !align_x) return launch_aligned(a, out, a.n, sm_count, s);
    if (!p.fit) return cudaErrorInvalidValue;
    char* room = static_cast<char*>(a.aligned);
    char* room_w = room + p.used * 2;
    const long long px = p.px, tokens = p.tokens, experts = p.experts, outs = p.outs;
    for (long long g = 0; g < a.groups; g += experts)
        for (long long o = 0; o < out; o += outs)
            for (long long t = 0; t < a.tokens; t += tokens) {
                ProductArgs c = a;
                const int n_out = (int)std::min(outs, out - o);
                c.groups = (int)std::min(experts, a.groups - g);
                c.offsets = a.offsets ? a.offsets + g : nullptr;
                c.first = (int)t, c.tokens = std::min(tokens, a.tokens - t);
                c.x = static_cast<const char*>(a.x) + t * a.ldx * 2;
                c.y = static_cast<char*>(a.y) + (t * a.ldy + o) * 2;
                c.weight = static_cast<const char*>(a.weight) + (g * a.m * a.n + (a.transposed ? o : o * a.n)) * 2;
                long long pitch = a.n;
                AlignArgs r{};
                r.a = c;
                if (align_w) {
                    const int cols = a.transposed ? n_out : a.n, rows = a.transposed ? a.m : n_out;
                    pitch = aligned_pitch(cols);
                    if (t == 0) {
                        set_job(&r.job[0], c.weight, a.n, room_w, pitch, (long long)c.groups * rows, cols);
                        if (a.offsets) r.job[0].by_expert.set(rows);
                    }
                    c.weight = room_w;
                }
                if (align_x && (tokens < a.tokens || (g == 0 && o == 0)))
                    set_job(&r.job[1], c.x, a.ldx, room, px, c.tokens, k);
                if (align_x) c.x = room, c.ldx = px;
                // an expert's weights are wanted by any of its tokens, not by this chunk's alone
                r.a.first = 0, r.a.tokens = a.tokens;
                int blocks[2];
                constexpr int kBlock = kAlignThreads * kAlignUnroll;
                for (int i = 0; i < 2; ++i) blocks[i] = std::min((r.job[i].pieces + kBlock - 1) / kBlock, 12 * sm_count);
                r.blocks = blocks[0];
                if (blocks[0] + blocks[1] > 0) {
                    const cudaError_t e =
                        launch_pdl(k_align_rows, dim3(blocks[0] + blocks[1]), dim3(kAlignThreads), 0, s, r);
                    if (e != cudaSuccess) return e;
                }
                c.m = a.transposed ? a.m : n_out, c.n = a.transposed ? n_out : a.n;
                const cudaError_t e = launch_aligned(c, n_out, pitch, sm_count, s);
                if (e != cudaSuccess) return e;
            }
    return cudaSuccess;
}

}  // namespace muon
