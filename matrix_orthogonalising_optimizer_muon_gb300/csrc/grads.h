// Lists of gradients as the norm and the clipping take them.  Host entry points in acts.cu,
// kernels in gradnorm.cu.
#pragma once
#include <algorithm>

#include "acts.h"

namespace muon {

// A gradient is walked in groups of eight values, the first of which may begin before it so that every
// whole group is aligned to 16 bytes on the side that is written (the norm: read), in chunks of 32 KB, one per
// block and turn.
constexpr int kChunkGroups16 = 2048, kChunkGroups32 = 1024;   // groups of a chunk, by the type that is read

struct GradEntry {
    const void* p;
    long long count;
    uint32_t first;          // first chunk
    uint8_t bf16, out_bf16;
    uint16_t pad;            // values by which the first group begins before the gradient
};

// Parameters of one launch: at most 32764 bytes, the few for short lists.
constexpr int kTableFew = 30, kTableSome = 220, kTableNorm = 1280, kTableClip = 960;
constexpr int kMostBlocks = 640;
template <int N, bool OUT>
struct GradTable {
    static constexpr bool kOut = OUT;
    GradEntry e[N];
    void* out[OUT ? N : 1];        // clip: where the result goes
    uint16_t start[kMostBlocks];   // the gradient that each block's first chunk lies in
    int n;
    uint32_t chunks;
};
static_assert(sizeof(GradTable<kTableNorm, false>) <= 32764 - 64 && sizeof(GradTable<kTableClip, true>) <= 32764 - 64,
              "a launch's parameters");

struct GradList {
    const void* const* p;
    const int64_t* counts;
    const int32_t* dtypes;       // 0 fp32, 1 bf16
    void* const* out;            // null: the norm alone
    const int32_t* out_dtypes;
    int n;
    bool in_place;

    // The table of gradients from .. to - 1 for at most `most` blocks, which share the chunks evenly; returns how many.
    template <typename Table>
    int table(int from, int to, int most, Table* t) const {
        t->n = to - from;
        long long chunks = 0;
        for (int i = from; i < to; ++i) {
            GradEntry& e = t->e[i - from];
            e.p = p[i], e.count = counts[i];
            e.bf16 = dtypes[i] == 1, e.out_bf16 = Table::kOut ? out_dtypes[i] == 1 : 0;
            if (Table::kOut) t->out[i - from] = out[i];
            const uintptr_t at = reinterpret_cast<uintptr_t>(Table::kOut ? out[i] : p[i]);
            const int esz = (Table::kOut ? e.out_bf16 : e.bf16) ? 2 : 4, groups = e.bf16 ? kChunkGroups16 : kChunkGroups32;
            e.pad = (uint16_t)((at & 15) / esz);
            e.first = (uint32_t)chunks;
            if (counts[i] > 0) chunks += ((counts[i] + e.pad + 7) / 8 + groups - 1) / groups;
        }
        t->chunks = (uint32_t)chunks;
        const int blocks = (int)std::max<long long>(std::min<long long>(chunks, std::min(most, kMostBlocks)), 1);
        for (int b = 0, i = 0; b < blocks; ++b) {
            const uint32_t c = (uint32_t)(t->chunks * (uint64_t)b / blocks);
            while (i + 1 < t->n && t->e[i + 1].first <= c) ++i;
            t->start[b] = (uint16_t)i;
        }
        return blocks;
    }
};

struct GradNormArgs {
    double* partial;   // a sum per block
    double* running;   // the sum of the launches so far
    int* arrived;      // zero between calls
    float* norm;
    int sm_count;
};
cudaError_t launch_grad_norm(const GradList& l, const GradNormArgs& a, cudaStream_t s);
cudaError_t launch_grad_clip(const GradList& l, const float* norm, float max_norm, int sm_count, cudaStream_t s);

}  // namespace muon
