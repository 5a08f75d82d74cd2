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
// even CTA's), warps 2-5 are the epilogue; where rows are not 16-byte aligned, 16 more warps copy them into
// shared memory instead of TMA.  A step is 64 values of the contraction: 16 KB of the weight and up to
// 16 KB of tokens per CTA, in a ring of six.
//
// How the work is dealt out (every CTA derives the same plan from the offsets): tiles in the order experts,
// bands of kBand token tiles, outputs, token tiles, so that the tiles in flight share operands in L2.  All but
// the last turns of long launches go round the CTA pairs; what is left is cut into stretches of equal
// cost, one per pair, that may begin and end inside a tile's sum.  Such tiles' partial sums meet in the
// workspace, and the part that comes last adds them up in their order.
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
constexpr int kEpiFirst = 2, kEpi = 4;             // epilogue warps
constexpr int kCopyFirst = kEpiFirst + kEpi;
constexpr int kCopyGroups = 4, kGroupWarps = 4;    // copying warps: groups that take steps in turn
template <bool COPY>
constexpr int kThreadsOf = 32 * (kCopyFirst + (COPY ? kCopyGroups * kGroupWarps : 0));
constexpr int kBand = 8;
constexpr int kBins = 512;                         // experts are searched in at most this many bins
constexpr int kItems = 96;                         // items decoded at the start
constexpr int kMostPairs = 76;

struct Cfg {
    static constexpr int A_BYTES = 128 * kStepK * 2;
    static constexpr int CHUNK_BYTES = 64 * kStepK * 2;   // 64 outputs of an MN-major weight
    static constexpr int SLOT_BYTES = 2 * A_BYTES;
    static constexpr int OUT_OFFSET = kRing * SLOT_BYTES;
    static constexpr int OUT_WARP = 2 * 2048;             // two blocks of 32 outputs x 32 tokens in bf16
    static constexpr int BAR_OFFSET = OUT_OFFSET + kEpi * OUT_WARP;
    static constexpr int SIGNAL_OFFSET = BAR_OFFSET + 256;   // 16 bytes per copying warp
    static constexpr int PLAN_OFFSET = SIGNAL_OFFSET + 256;
    static constexpr int ITEM_OFFSET = PLAN_OFFSET + 2 * (kBins + 4) * 4 + 2 * (kMostPairs + 4) * 4 + 64;
    static constexpr int SMEM_BYTES = ITEM_OFFSET + kItems * 32 + 1024;
};
static_assert(Cfg::SMEM_BYTES <= 232448, "product kernel exceeds the shared memory of one CTA");
static_assert(Cfg::ITEM_OFFSET % 16 == 0, "items are loaded 16 bytes at a time");

struct ProductLaunch {
    CUtensorMap map_w, map_x[4];   // map_x: boxes of 128, 64, 32 and 16 tokens
    ProductArgs a;
    int out, k, steps, tiles_m;    // outputs, contraction, its steps, tiles along the outputs
    int tma_w, tma_x;              // rows are aligned to 16 bytes
    int wide;                      // rows of y are aligned to four elements
};

// The launch's plan in shared memory.
struct Plan {
    int tiles[kBins + 4];      // token tiles before each bin of experts
    int cost[kBins + 4];       // their cost
    int unit[kMostPairs + 4];  // begins of the pairs' stretches: tile and step
    int step[kMostPairs + 4];
    int count[4];              // token tiles when they are 256, 128, 64 tokens high
    int cap, stride, turns, pairs;   // tile height, experts per bin, whole turns, stretches
    int units;
    int pad[7];
};
static_assert(sizeof(Plan) == Cfg::ITEM_OFFSET - Cfg::PLAN_OFFSET, "plan's place");

struct __align__(16) Item {
    int m0, t0, end, group;    // first output, first token, end of the expert's tokens
    int k0, k1, n;             // steps, height in tokens (a multiple of 32)
    int part;                  // parts << 16 | part << 8 | first pair; 0: the whole sum
};

// Cost of a tile's step, in 32 cycles: the weight's 16 KB take as long as 256 tokens' MMAs do.
__device__ __forceinline__ int tile_cost(int n) { return 8 + (n >> 5); }

__device__ __forceinline__ void expert_range(const ProductArgs& a, int g, int* begin, int* end) {   // tokens < 2^31
    *begin = a.offsets ? min(max(a.offsets[g], 0), (int)a.tokens) : 0;
    *end = a.offsets ? min(max(a.offsets[g + 1], *begin), (int)a.tokens) : (int)a.tokens;
}

// An expert's token tiles: all `cap` high but the last.
struct Tiles {
    int begin, end, count, tail;   // tail: the last one's height in steps of 32
    __device__ __forceinline__ Tiles(const ProductArgs& a, int g, int cap) {
        expert_range(a, g, &begin, &end);
        count = (int)((uint32_t)(end - begin + cap - 1) / (uint32_t)cap);
        const int left = end - begin - (count - 1) * cap;
        tail = (left + 31) & ~31;
    }
    __device__ __forceinline__ int cost(int cap) const {
        return count ? (count - 1) * tile_cost(cap) + tile_cost(tail) : 0;
    }
};

// The expert that tile `v` of all experts' token tiles (or cost, by `key`) lies in.
__device__ __forceinline__ int find_bin(const int* key, int bins, int v) {
    int lo = 0, hi = bins - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (key[mid] <= v)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

struct Where {
    int group, m, t;   // expert, tile along the outputs, token tile
};

// Tile u of the launch.
__device__ __forceinline__ Where decode_unit(const ProductLaunch& L, const Plan& p, int u) {
    const int bins = (L.a.groups + p.stride - 1) / p.stride;
    const int v = u / L.tiles_m;
    Where w;
    const int b = find_bin(p.tiles, bins, v);
    int before = p.tiles[b];
    w.group = b * p.stride;
    Tiles e(L.a, w.group, p.cap);
    while (before + e.count <= v && w.group + 1 < L.a.groups) {
        before += e.count;
        e = Tiles(L.a, ++w.group, p.cap);
    }
    int r = u - before * L.tiles_m;
    const int band = r / (kBand * L.tiles_m);
    r -= band * kBand * L.tiles_m;
    const int wide = min(kBand, e.count - band * kBand);
    w.m = r / wide;
    w.t = band * kBand + r - w.m * wide;
    return w;
}

// Cost of all tiles before tile u, in steps times tile_cost.
__device__ __forceinline__ long long cost_before(const ProductLaunch& L, const Plan& p, int u) {
    if (u == 0) return 0;
    const Where w = decode_unit(L, p, u);
    const int b = w.group / p.stride;
    int before = p.cost[b];
    for (int g = b * p.stride; g < w.group; ++g) before += Tiles(L.a, g, p.cap).cost(p.cap);
    const Tiles e(L.a, w.group, p.cap);
    const int full = tile_cost(p.cap), band = w.t / kBand;
    const int wide = min(kBand, e.count - band * kBand);
    long long c = (long long)before * L.tiles_m + (long long)band * kBand * L.tiles_m * full;
    const int column = wide * full - (band * kBand + wide == e.count ? full - tile_cost(e.tail) : 0);
    c += (long long)w.m * column + (long long)(w.t - band * kBand) * full;
    return c * L.steps;
}

// The tile and step where the cost before is c: T is wide enough for the whole cost.
template <typename T>
__device__ __forceinline__ void locate(const ProductLaunch& L, const Plan& p, T c, int* unit, int* step) {
    const int bins = (L.a.groups + p.stride - 1) / p.stride;
    const T scale = (T)L.tiles_m * (T)L.steps;
    const int b = find_bin(p.cost, bins, (int)(c / scale));
    T left = c - (T)p.cost[b] * scale;
    int g = b * p.stride, before = p.tiles[b];
    Tiles e(L.a, g, p.cap);
    while (left >= (T)e.cost(p.cap) * scale && g + 1 < L.a.groups) {
        left -= (T)e.cost(p.cap) * scale;
        before += e.count;
        e = Tiles(L.a, ++g, p.cap);
    }
    const int full = tile_cost(p.cap);
    const int band = min((int)(left / ((T)(kBand * full) * scale)), (e.count - 1) / kBand);
    left -= (T)band * (T)(kBand * full) * scale;
    const int wide = min(kBand, e.count - band * kBand);
    const bool ends = band * kBand + wide == e.count;
    const T column = (T)(wide * full - (ends ? full - tile_cost(e.tail) : 0)) * (T)L.steps;
    const int m = min((int)(left / column), L.tiles_m - 1);
    left -= (T)m * column;
    const int t = min((int)(left / (T)(full * L.steps)), wide - 1);
    left -= (T)t * (T)(full * L.steps);
    *unit = (before + band * kBand) * L.tiles_m + m * wide + t;
    *step = min((int)(left / (T)(ends && t == wide - 1 ? tile_cost(e.tail) : full)), L.steps);
}

// Fills the plan: all threads of the CTA.
__device__ void make_plan(const ProductLaunch& L, Plan& p, int threads) {
    const int tid = threadIdx.x, lane = tid & 31, pairs = gridDim.x >> 1;
    if (tid < 4) p.count[tid] = 0;
    __syncthreads();
    // heights of tiles: 256 tokens if those fill the GPU once, else 128 or 64
    int c0 = 0, c1 = 0, c2 = 0;
    for (int g = tid; g < L.a.groups; g += threads) {
        int b, e;
        expert_range(L.a, g, &b, &e);
        c0 += (e - b + 255) >> 8, c1 += (e - b + 127) >> 7, c2 += (e - b + 63) >> 6;
    }
    c0 = __reduce_add_sync(0xffffffffu, c0), c1 = __reduce_add_sync(0xffffffffu, c1);
    c2 = __reduce_add_sync(0xffffffffu, c2);
    if (lane == 0 && c2 > 0) atomicAdd(p.count, c0), atomicAdd(p.count + 1, c1), atomicAdd(p.count + 2, c2);
    __syncthreads();
    const int need = (pairs + L.tiles_m - 1) / L.tiles_m;
    const int most = p.count[0] == p.count[2] ? 64 : p.count[0] == p.count[1] ? 128 : 256;   // no expert has more
    const int cap = min(p.count[0] >= need ? 256 : p.count[1] >= need ? 128 : 64, most);
    const int stride = (L.a.groups + kBins - 1) / kBins, bins = (L.a.groups + stride - 1) / stride;
    for (int b = tid; b < bins; b += threads) {
        int tiles = 0, cost = 0;
        for (int g = b * stride; g < min((b + 1) * stride, L.a.groups); ++g) {
            const Tiles e(L.a, g, cap);
            tiles += e.count, cost += e.cost(cap);
        }
        p.tiles[b] = tiles, p.cost[b] = cost;
    }
    __syncthreads();
    if (tid < 32) {   // sums of the bins before
        int tiles = 0, cost = 0;
        for (int b0 = 0; b0 < bins; b0 += 32) {
            const int b = b0 + lane, t = b < bins ? p.tiles[b] : 0, c = b < bins ? p.cost[b] : 0;
            int st = t, sc = c;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int x = __shfl_up_sync(0xffffffffu, st, d), y = __shfl_up_sync(0xffffffffu, sc, d);
                if (lane >= d) st += x, sc += y;
            }
            if (b < bins) p.tiles[b] = tiles + st - t, p.cost[b] = cost + sc - c;
            tiles += __shfl_sync(0xffffffffu, st, 31), cost += __shfl_sync(0xffffffffu, sc, 31);
        }
        if (lane == 0) {
            p.tiles[bins] = tiles, p.cost[bins] = cost;
            p.cap = cap, p.stride = stride;
            p.units = tiles * L.tiles_m;
            p.turns = p.units / pairs >= 8 ? p.units / pairs - 3 : 0;
        }
    }
    __syncthreads();
    // stretches of equal cost; parts of a tile have at least `least` steps, and tiles are cut only if that
    // shortens the longest stretch by more than joining the parts takes
    const int first = p.turns * pairs, rest = p.units - first, full = tile_cost(cap), least = 2 + cap / 32;
    const long long from = cost_before(L, p, first);
    const long long total = (long long)p.cost[bins] * L.tiles_m * L.steps, span = total - from;
    const int whole = (rest + pairs - 1) / pairs;
    const bool cut = span / pairs + (long long)least * full < (long long)whole * full * L.steps;
    int stretches = pairs;
    if (cut) stretches = (int)min((long long)pairs, max(span / (least * full), 1ll));
    for (int i = tid; i <= stretches; i += threads) {
        int u = i == 0 ? first : p.units, k = 0;
        if (i > 0 && i < stretches && span > 0) {
            const long long c = from + span * i / stretches;
            if (total < (1ll << 27))   // 8 tiles' cost, at most 15 times a tile's least, is below 2^31
                locate<uint32_t>(L, p, (uint32_t)c, &u, &k);
            else
                locate<unsigned long long>(L, p, (unsigned long long)c, &u, &k);
            const int edge = max(min(least, L.steps / 2), 1);
            if (cut ? k > L.steps - edge : 2 * k >= L.steps)
                ++u, k = 0;
            else if (!cut || k < edge)
                k = 0;
        }
        p.unit[i] = u, p.step[i] = k;
    }
    if (tid == 0) p.pairs = stretches;
    __syncthreads();
}

// What a CTA pair does, one item per turn.
struct Items {
    int pair, pairs, turns, count;
    __device__ __forceinline__ Items(const Plan& p) : pair(blockIdx.x >> 1), pairs(gridDim.x >> 1), turns(p.turns) {
        count = turns;
        if (pair < p.pairs) count += p.unit[pair + 1] - p.unit[pair] + (p.step[pair + 1] > 0);
    }
    __device__ __forceinline__ Item decode(const ProductLaunch& L, const Plan& p, int turn) const {
        Item it;
        int u;
        it.k0 = 0, it.k1 = L.steps, it.part = 0;
        if (turn < turns) {   // every other turn backwards: a pair gets tiles of every height
            u = turn * pairs + (turn & 1 ? pairs - 1 - pair : pair);
        } else {
            u = p.unit[pair] + turn - turns;
            if (turn == turns) it.k0 = p.step[pair];
            if (u == p.unit[pair + 1]) it.k1 = p.step[pair + 1];
            if (it.k0 > 0 || it.k1 < L.steps) {
                int a = it.k0 > 0 ? pair - 1 : pair;   // the pair that has the tile's first steps
                while (p.unit[a] == u && p.step[a] > 0) --a;
                int z = pair;                          // the one that has its last
                while (z + 1 < p.pairs && p.unit[z + 1] == u) ++z;
                it.part = (z - a + 1) << 16 | (pair - a) << 8 | a;
            }
        }
        const Where w = decode_unit(L, p, u);
        const Tiles e(L.a, w.group, p.cap);
        it.group = w.group, it.m0 = w.m * 256, it.t0 = e.begin + w.t * p.cap, it.end = e.end;
        it.n = w.t == e.count - 1 ? e.tail : p.cap;
        return it;
    }
    __device__ __forceinline__ Item get(const ProductLaunch& L, const Plan& p, uint32_t table, int turn) const {
        if (turn >= kItems) return decode(L, p, turn);
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

__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t x) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}

// Rows first, first + step, ... of a swizzled operand box of 64 values a row (kBatch at a time), from rows
// that are not 16-byte aligned: a lane makes 16 bytes from the two aligned pieces that hold them.  Every piece
// loaded holds a value of its row.  Rows at and beyond `rows` and columns at and beyond `cols` become zero.
constexpr int kBatch = 4;
__device__ __forceinline__ void copy_rows(const char* base, long long pitch, int rows, int col, int cols, uint32_t dst,
                                          int count, int lane, int warp) {
    const int j = lane & 7, c = col + 8 * j;
    for (int r0 = 4 * warp; r0 < count; r0 += 4 * kGroupWarps * kBatch) {
        uint32_t v[kBatch][8];
        int d[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * 4 * kGroupWarps + (lane >> 3);
            const uintptr_t line = reinterpret_cast<uintptr_t>(base) + (uintptr_t)(r * pitch);
            const uintptr_t at = line + (uintptr_t)(2ll * c);
            d[i] = (int)(at & 15);
            const uint4* q = reinterpret_cast<const uint4*>(at & ~(uintptr_t)15);
            const bool live = r < rows && r < count && c < cols;
            uint4 x = make_uint4(0, 0, 0, 0), y = x;
            if (live) x = *q;
            if (live && d[i] && reinterpret_cast<uintptr_t>(q + 1) < line + 2ull * cols) y = q[1];
            v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
            v[i][4] = y.x, v[i][5] = y.y, v[i][6] = y.z, v[i][7] = y.w;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * 4 * kGroupWarps + (lane >> 3);
            words_down<true>(v[i], d[i]);
            const int left = cols - c;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i][k] &= left > 2 * k + 1 ? 0xffffffffu : left > 2 * k ? 0xffffu : 0u;
            if (r < count) sts128(dst + r * 128 + ((j ^ (r & 7)) << 4), make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]));
        }
    }
}

struct Epilogue {
    uint32_t tmem_base, tempty_lead, blk, table;
    uint64_t* tfull;
    volatile int* abort_flag;
    int q, wq, lane;
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
__device__ __forceinline__ void store_block(const ProductLaunch& L, const Epilogue& e, const float (&f)[32], int c0, int t,
                                            int end, uint32_t blk) {
    char* y = static_cast<char*>(L.a.y);
    if (L.wide) {
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
                    *reinterpret_cast<uint2*>(to) = make_uint2(__byte_perm(x[i].x, x[i].y, 0x5410), __byte_perm(x[i].z, x[i].w, 0x5410));
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
__device__ __forceinline__ void part_store(float* p, const uint32_t (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4*>(p + i * 128) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
template <bool FIRST>
__device__ __forceinline__ void part_add(const float* p, float (&f)[32]) {
    float4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __ldcg(reinterpret_cast<const float4*>(p + i * 128));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f[4 * i] = FIRST ? x[i].x : f[4 * i] + x[i].x, f[4 * i + 1] = FIRST ? x[i].y : f[4 * i + 1] + x[i].y;
        f[4 * i + 2] = FIRST ? x[i].z : f[4 * i + 2] + x[i].z, f[4 * i + 3] = FIRST ? x[i].w : f[4 * i + 3] + x[i].w;
    }
}

// One epilogue warp: TMEM lane quarter wq, that is 32 outputs of a tile.
__device__ __forceinline__ void epilogue(const ProductLaunch& L, const Plan& plan, const Items& items, const Epilogue& e) {
    int local = 0;
    for (int turn = 0; turn < items.count; ++turn, ++local) {
        const Item w = items.get(L, plan, e.table, turn);
        const uint32_t acc = local & 1;
        if (!mbar_wait_idle(e.tfull + acc, local >> 1 & 1u, e.abort_flag, L.a.status, kStatusTimeoutEpilogue, true)) return;
        tc_fence_after();
        const uint32_t tbase = e.tmem_base + acc * 256 + (static_cast<uint32_t>(e.wq * 32) << 16);
        const int c0 = w.m0 + 128 * e.q + 32 * e.wq, mine = 4 * e.q + e.wq;
        const int parts = w.part >> 16, part = w.part >> 8 & 255, first = w.part & 255;
        // a pair has at most two parts of tiles: one that begins inside its tile, one that begins with it
        auto slot = [&](int k) {
            return L.a.partial + ((2 * (first + k) + (k == 0)) * 8ll + mine) * 8192 + e.lane * 4;
        };
        for (int c = 0; c < w.n; c += 32) {
            uint32_t v[32];
            tmem_ld32(tbase + c, v);
            tmem_ld_wait();
            if (c + 32 >= w.n) release_tmem(e, acc);
            if (parts) {
                part_store(slot(part) + c * 32, v);
            } else {
                float f[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);
                store_block(L, e, f, c0, w.t0 + c, w.end, e.blk + (c & 32) * 64);
            }
        }
        if (parts) {
            __threadfence();
            __syncwarp();
            int* count = L.a.counters + first * 8 + mine;
            int seen = 0;
            if (e.lane == 0) seen = atomicAdd(count, 1);
            if (__shfl_sync(0xffffffffu, seen, 0) == parts - 1) {
                if (e.lane == 0) *count = 0;   // for the next call
                __threadfence();
                for (int c = 0; c < w.n; c += 32) {
                    float f[32];
                    part_add<true>(slot(0) + c * 32, f);
                    for (int k = 1; k < parts; ++k) part_add<false>(slot(k) + c * 32, f);
                    store_block(L, e, f, c0, w.t0 + c, w.end, e.blk + (c & 32) * 64);
                }
            }
        }
    }
}

// MN: the weight is MN-major (dx = dy W).  COPY: an operand's rows are not aligned.
template <bool MN, bool COPY>
__global__ void __launch_bounds__(kThreadsOf<COPY>) k_product(const __grid_constant__ ProductLaunch L) {
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
            mbar_init(full + s, 1 + (COPY ? kGroupWarps : 0));
            mbar_init(empty + s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull + a, 1);
            mbar_init(tempty + a, 2 * kEpi);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        if (!COPY || L.tma_w) tma_prefetch_desc(&L.map_w);
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
    make_plan(L, plan, kThreadsOf<COPY>);
    const Items items(plan);
    for (int t = threadIdx.x; t < min(items.count, kItems); t += kThreadsOf<COPY>)
        reinterpret_cast<Item*>(smem + Cfg::ITEM_OFFSET)[t] = items.decode(L, plan, t);
    __syncthreads();

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA, completion on the even CTA's barrier
            uint32_t slot = 0, ph = 1;
            bool ok = true;
            for (int turn = 0; ok && turn < items.count; ++turn) {
                const Item w = items.get(L, plan, table, turn);
                const int rows = w.n >> 1, t0 = w.t0 + (int)q * rows, m0 = w.m0 + 128 * (int)q;
                const uint32_t bytes = (!COPY || L.tma_w ? 2 * Cfg::A_BYTES : 0) + (!COPY || L.tma_x ? 2 * rows * 128 : 0) +
                                       (COPY ? 16 * kGroupWarps : 0);
                for (int k = w.k0; k < w.k1; ++k) {
                    if (!mbar_wait_idle(empty + slot, ph, abort_flag, L.a.status, kStatusTimeoutProducer, true)) {
                        ok = false;
                        break;
                    }
                    uint8_t *sa = smem + slot * Cfg::SLOT_BYTES, *sb = sa + Cfg::A_BYTES;
                    const uint32_t fb = mapa_shared(smem_u32(full + slot), 0);
                    if (leader) mbar_arrive_expect_tx(full + slot, bytes);
                    const int kk = k * kStepK;
                    if (!COPY || L.tma_w) {
                        if (MN) {
                            tma_load_3d_pair(sa, &L.map_w, fb, m0, kk, w.group);
                            tma_load_3d_pair(sa + Cfg::CHUNK_BYTES, &L.map_w, fb, m0 + 64, kk, w.group);
                        } else {
                            tma_load_3d_pair(sa, &L.map_w, fb, kk, m0, w.group);
                        }
                    }
                    if (!COPY || L.tma_x) {
                        int at = 0;
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            if (rows & (128 >> b)) {
                                tma_load_2d_pair(sb + at * 128, &L.map_x[b], fb, kk, t0 + at);
                                at += 128 >> b;
                            }
                        }
                    }
                    if (++slot == kRing) slot = 0, ph ^= 1u;
                }
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
                const Item w = items.get(L, plan, table, turn);
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
    } else if (warp < kCopyFirst) {
        // ---------------- epilogue
        Epilogue e;
        e.tmem_base = tmem_base;
        e.tempty_lead = mapa_shared(smem_u32(tempty), 0);
        e.blk = smem_u32(smem + Cfg::OUT_OFFSET + (warp - kEpiFirst) * Cfg::OUT_WARP);
        e.table = table;
        e.tfull = tfull;
        e.abort_flag = abort_flag;
        e.q = (int)q, e.wq = warp & 3, e.lane = lane;
        epilogue(L, plan, items, e);
    } else if (COPY) {
        // ---------------- copies of rows that are not aligned: group g takes every kCopyGroups-th step
        const int cw = (warp - kCopyFirst) % kGroupWarps;
        const uint32_t g = (warp - kCopyFirst) / kGroupWarps;
        const uint32_t full_lead = mapa_shared(smem_u32(full), 0);
        const uint32_t signal_lead = mapa_shared(smem_u32(smem + Cfg::SIGNAL_OFFSET), 0) + 16 * (warp - kCopyFirst);
        uint32_t it = 0, slot = 0, ph = 1;
        bool ok = true;
        for (int turn = 0; ok && turn < items.count; ++turn) {
            const Item w = items.get(L, plan, table, turn);
            const int rows = w.n >> 1, t0 = w.t0 + (int)q * rows, m0 = w.m0 + 128 * (int)q;
            const char* wp = static_cast<const char*>(L.a.weight) + (long long)w.group * L.a.m * L.a.n * 2;
            const char* xp = static_cast<const char*>(L.a.x) + t0 * L.a.ldx * 2;
            for (int k = w.k0; k < w.k1; ++k, ++it) {
                const uint32_t s = slot, parity = ph;
                if (++slot == kRing) slot = 0, ph ^= 1u;
                if (it % kCopyGroups != g) continue;
                if (!mbar_wait_idle(empty + s, parity, abort_flag, L.a.status, kStatusTimeoutProducer, true)) {
                    ok = false;
                    break;
                }
                const uint32_t sa = smem_u32(smem + s * Cfg::SLOT_BYTES);
                const int kk = k * kStepK;
                if (!L.tma_w) {
                    if (MN) {
                        const char* p = wp + (long long)kk * L.a.n * 2;
                        copy_rows(p, L.a.n * 2ll, L.a.m - kk, m0, L.a.n, sa, kStepK, lane, cw);
                        copy_rows(p, L.a.n * 2ll, L.a.m - kk, m0 + 64, L.a.n, sa + Cfg::CHUNK_BYTES, kStepK, lane, cw);
                    } else {
                        copy_rows(wp + (long long)m0 * L.a.n * 2, L.a.n * 2ll, L.a.m - m0, kk, L.a.n, sa, 128, lane, cw);
                    }
                }
                if (!L.tma_x) copy_rows(xp, L.a.ldx * 2, w.end - t0, kk, L.k, sa + Cfg::A_BYTES, rows, lane, cw);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // writes visible to the MMAs
                __syncwarp();
                if (lane == 0) {
                    // the odd CTA's arrival is a copy of 16 bytes that mean nothing, whose completion releases
                    // at cluster scope, which no thread has to wait for
                    if (leader)
                        mbar_arrive(full + s);
                    else
                        bulk_signal(signal_lead, smem + Cfg::SIGNAL_OFFSET + 16 * (warp - kCopyFirst), full_lead + s * 8);
                }
            }
        }
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

typedef void (*ProductKernel)(ProductLaunch);
ProductKernel pick(bool mn, bool copy) {
    static const ProductKernel k[2][2] = {{k_product<false, false>, k_product<false, true>},
                                          {k_product<true, false>, k_product<true, true>}};
    return k[mn][copy];
}

}  // namespace

cudaError_t product_prepare() {
    for (int i = 0; i < 4; ++i) {
        const cudaError_t e = cudaFuncSetAttribute(pick(i & 1, i >> 1), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   Cfg::SMEM_BYTES);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_product(const ProductArgs& a, int sm_count, cudaStream_t s) {
    ProductLaunch L;
    L.a = a;
    L.out = a.transposed ? a.n : a.m;
    L.k = a.transposed ? a.m : a.n;
    L.steps = (L.k + kStepK - 1) / kStepK;
    L.tiles_m = (L.out + 255) / 256;
    if ((a.tokens / 64 + a.groups) * L.tiles_m >= (1ll << 31)) return cudaErrorInvalidValue;
    L.tma_w = a.n % 8 == 0 && (reinterpret_cast<uintptr_t>(a.weight) & 15) == 0;
    L.tma_x = ((reinterpret_cast<uintptr_t>(a.x) | (uintptr_t)(a.ldx * 2)) & 15) == 0;
    L.wide = L.out % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.y) | (uintptr_t)(a.ldy * 2)) & 7) == 0;
    if (L.tma_w && !muon_impl::make_map(&L.map_w, const_cast<void*>(a.weight), true, a.n, a.m, a.groups, a.n, 64,
                                        a.transposed ? 64 : 128))
        return cudaErrorInvalidValue;
    for (int b = 0; L.tma_x && b < 4; ++b)
        if (!map_tokens(&L.map_x[b], a.x, L.k, a.tokens, a.ldx * 2, 128 >> b)) return cudaErrorInvalidValue;
    const bool copy = !L.tma_w || !L.tma_x;
    return launch_pdl_cluster(pick(a.transposed, copy), dim3(2 * std::min(sm_count / 2, kMostPairs)),
                              dim3(copy ? kThreadsOf<true> : kThreadsOf<false>), Cfg::SMEM_BYTES, s, 2u, L);
}

}  // namespace muon
