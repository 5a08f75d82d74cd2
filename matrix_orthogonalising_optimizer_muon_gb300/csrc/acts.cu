// C entry points of the layer-side operators (include/muon.h): argument checks, the grad
// plan, launches.  Host code only.
#include "acts.h"
#include "grads.h"
#include "plan.h"

struct muon_grad_plan_s {
    int device = 0;
    int sm_count = 0;
    void* ws = nullptr;       // status word, counters, partial sums
    int* status = nullptr;
    int* arrived = nullptr;     // blocks of the norm in progress
    double* running = nullptr;  // squares of the norm's launches so far
    int* counters = nullptr;
    float* partial = nullptr;
    int64_t aligned = 0;        // bytes behind the partial sums, for the products' copies
};

namespace {
using namespace muon_impl;

constexpr size_t kWsHeader = 256 + kCounters * sizeof(int);   // status word, counters
constexpr int64_t kGradWorkspace = (int64_t)kWsHeader + kPartialFloats * 4;   // and the plan's aligned bytes
static_assert(kWsHeader % 256 == 0, "the partial sums are aligned");

constexpr int64_t kMostPitch = 1ll << 32;   // bytes from row to row
constexpr int64_t kMostValues = 1ll << 43;  // of a list of gradients

// A strided range of device memory: `rows` rows of `width` bytes, `pitch` bytes apart.
struct Range {
    uintptr_t p;
    long long rows, width, pitch;
};

bool overlap(const Range& a, const Range& b) {
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0) return false;
    const uintptr_t ea = a.p + (uintptr_t)((a.rows - 1) * a.pitch + a.width);
    const uintptr_t eb = b.p + (uintptr_t)((b.rows - 1) * b.pitch + b.width);
    if (a.p >= eb || b.p >= ea) return false;
    if (a.pitch != b.pitch) return true;
    // rows interleave: disjoint when the column intervals are, modulo the pitch
    const long long d = (long long)(b.p > a.p ? (b.p - a.p) % (uintptr_t)a.pitch
                                              : (a.pitch - (long long)((a.p - b.p) % (uintptr_t)a.pitch)) % a.pitch);
    return !(d >= a.width && d + b.width <= a.pitch);
}

bool same(const Range& a, const Range& b) { return a.p == b.p && a.pitch == b.pitch; }

// One call's operands, checked together: every output against everything else.
struct Operands {
    static constexpr int kMax = 16;
    Range r[kMax];
    int alias[kMax];   // operands (bits) that may be this output itself
    bool out[kMax];
    int n = 0;
    bool bad = false;

    int add(const void* p, long long rows, long long width, long long pitch, bool output, int may_alias = 0) {
        r[n] = {reinterpret_cast<uintptr_t>(p), rows, width, pitch};
        alias[n] = may_alias;
        out[n] = output;
        return n++;
    }
    bool clash() const {
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < n; ++j) {
                if (i == j || !out[i] || (out[j] && j < i)) continue;
                if ((alias[i] >> j & 1) && same(r[i], r[j])) continue;
                if (overlap(r[i], r[j])) return true;
            }
        return false;
    }
};

bool aligned16(const void* p, long long pitch) {
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)pitch) & 15) == 0;
}

// Checks one tensor and records it.  `vec` stays set while every row is 16-byte aligned.
struct Call {
    long long rows, cols;
    int esz;
    bool vec = true, ok = true;
    Operands ops;

    int mat(Mat* m, const void* p, int64_t ld, bool output, bool optional, int may_alias = 0) {
        m->p = const_cast<void*>(p);
        m->pitch = 0;
        if (!p) {
            ok = ok && optional;
            return ops.add(nullptr, 0, 0, 0, output);
        }
        ok = ok && ld >= cols && ld < kMostPitch / esz && (reinterpret_cast<uintptr_t>(p) & (esz - 1)) == 0;
        m->pitch = ok ? (uint32_t)(ld * esz) : 0;
        vec = vec && aligned16(p, ld * esz);
        return ops.add(p, rows, cols * esz, ld * esz, output, may_alias);
    }
    void vector(const void* p, long long count, bool output, bool optional) {
        ok = ok && (p || optional) && (reinterpret_cast<uintptr_t>(p) & 3) == 0;
        ops.add(p, count > 0, count * 4, count * 4 + 4, output);
    }
    void act(Act8* q, const muon_act8* a, bool output, bool optional) {
        *q = Act8{};
        if (!a) {
            ok = ok && optional;
            return;
        }
        ok = ok && ((a->codes && a->scales) || rows == 0) && (a->format == MUON_ACT_E4M3 || a->format == MUON_ACT_INT8) &&
             a->reserved == 0 && a->ldq >= cols && a->lds >= (cols + kActGroup - 1) / kActGroup &&
             a->ldq < kMostPitch && a->lds < kMostPitch && aligned16(a->codes, a->ldq) &&
             aligned16(a->scales, a->lds);
        if (!ok) return;
        *q = Act8{static_cast<uint8_t*>(a->codes), static_cast<uint8_t*>(a->scales), (uint32_t)a->ldq, (uint32_t)a->lds,
                  a->format};
        // whole 16-byte pieces, as readers fetch them
        ops.add(a->codes, rows, round_up(cols, 16), a->ldq, output);
        ops.add(a->scales, rows, round_up((cols + kActGroup - 1) / kActGroup, 16), a->lds, output);
    }
    muon_status status() const { return ok && !ops.clash() ? MUON_OK : MUON_ERR_INVALID_ARG; }
};

muon_status begin(Call* c, int64_t rows, int64_t cols, muon_dtype dtype, int64_t most_cols) {
    if (rows < 0 || cols < 1) return MUON_ERR_INVALID_ARG;
    if (dtype != MUON_F32 && dtype != MUON_BF16) return MUON_ERR_UNSUPPORTED;
    if (rows >= (1ll << 31) || cols > most_cols) return MUON_ERR_UNSUPPORTED;
    c->rows = rows;
    c->cols = cols;
    c->esz = dtype == MUON_BF16 ? 2 : 4;
    return MUON_OK;
}

muon_status check_grad_plan(const muon_grad_plan_s* p) {
    int dev = -1;
    if (!p) return MUON_ERR_INVALID_ARG;
    if (cudaGetDevice(&dev) != cudaSuccess) return MUON_ERR_CUDA;
    return dev == p->device ? MUON_OK : MUON_ERR_INVALID_ARG;
}

#define MUON_CALL(expr)                       \
    do {                                      \
        const muon_status st__ = (expr);      \
        if (st__ != MUON_OK) return st__;     \
    } while (0)

constexpr int kMostExperts = 4096;
constexpr int kMostChoices = 64;

// The moves between the tokens' order and the experts': c's rows are the tokens'.
muon_status begin_move(Call* c, int64_t tokens, int32_t choices, int64_t rows, int64_t cols, muon_dtype dtype) {
    MUON_CALL(begin(c, tokens, cols, dtype, kMaxDim));
    if (choices < 1 || choices > kMostChoices || rows < 0) return MUON_ERR_INVALID_ARG;
    if (tokens * choices >= (1ll << 31) || rows >= (1ll << 31)) return MUON_ERR_UNSUPPORTED;
    return MUON_OK;
}
void set_move(MoveArgs* a, const int32_t* slots, const float* weights, int64_t tokens, int32_t choices, int64_t rows,
              int64_t cols) {
    a->slots = slots, a->weights = weights, a->tokens = (uint32_t)tokens, a->rows = (uint32_t)rows;
    a->choices = choices, a->cols = (int)cols;
}

muon_status product(muon_grad_plan_s* p, const void* x, int64_t ldx, const void* weight, int64_t tokens, int64_t m,
                    int64_t n, const int32_t* offsets, int32_t groups, void* y, int64_t ldy, bool transposed,
                    void* stream) {
    Call cx, cy;
    ProductArgs a{};
    Mat mat{};
    MUON_CALL(begin(&cx, tokens, transposed ? m : n, MUON_BF16, kMaxDim));
    MUON_CALL(begin(&cy, tokens, transposed ? n : m, MUON_BF16, kMaxDim));
    if (!p || groups < 0 || groups > kMostExperts || (groups > 0) != (offsets != nullptr)) return MUON_ERR_INVALID_ARG;
    if (tokens > (1ll << 31) - 4096) return MUON_ERR_UNSUPPORTED;   // rows of the last tile are counted in 32 bits
    cx.mat(&mat, x, ldx, false, tokens == 0);
    if (!cx.ok) return MUON_ERR_INVALID_ARG;
    cy.ops.add(x, tokens, cx.cols * 2, ldx * 2, false);
    cy.mat(&mat, y, ldy, true, tokens == 0);
    cy.vector(offsets, groups ? groups + 1 : 0, false, true);
    cy.ok = cy.ok && weight && (reinterpret_cast<uintptr_t>(weight) & 1) == 0;
    cy.ops.add(weight, (long long)std::max(groups, 1) * m, n * 2, n * 2, false);
    MUON_CALL(cy.status());
    MUON_CALL(check_grad_plan(p));
    if (tokens == 0) return MUON_OK;
    a.x = x, a.ldx = ldx, a.weight = weight, a.y = y, a.ldy = ldy, a.tokens = tokens, a.m = (int)m, a.n = (int)n;
    a.transposed = transposed, a.offsets = offsets, a.groups = std::max(groups, 1);
    a.status = p->status, a.partial = p->partial, a.counters = p->counters;
    a.aligned = p->partial + kJoinFloats, a.room = kSharedRoom + p->aligned;
    if (!product_fits(a)) return MUON_ERR_UNSUPPORTED;
    return cuda_status(launch_product(a, p->sm_count, static_cast<cudaStream_t>(stream)));
}

muon_status check_list(const void* const* p, const int64_t* counts, const int32_t* dtypes, int32_t n) {
    if (n < 0 || (n > 0 && (!p || !counts || !dtypes))) return MUON_ERR_INVALID_ARG;
    int64_t left = kMostValues;
    for (int i = 0; i < n; ++i) {
        if (dtypes[i] != MUON_F32 && dtypes[i] != MUON_BF16) return MUON_ERR_UNSUPPORTED;
        if (counts[i] < 0) return MUON_ERR_INVALID_ARG;
        if (counts[i] > left) return MUON_ERR_UNSUPPORTED;
        left -= counts[i];
        if (counts[i] > 0 && (!p[i] || (reinterpret_cast<uintptr_t>(p[i]) & (dtypes[i] == MUON_BF16 ? 1 : 3))))
            return MUON_ERR_INVALID_ARG;
    }
    return MUON_OK;
}

// Whether a tensor that is written overlaps another one or the norm; out null: the gradients are written.
bool lists_overlap(const void* const* grads, const int64_t* counts, const int32_t* dtypes, int32_t n, void* const* out,
                   const int32_t* out_dtypes, const float* norm) {
    struct Span {
        uintptr_t from, to;
        bool written;
    };
    std::vector<Span> spans;
    spans.reserve(2 * (size_t)n + 1);
    spans.push_back({reinterpret_cast<uintptr_t>(norm), reinterpret_cast<uintptr_t>(norm) + 4, false});
    for (int i = 0; i < n; ++i) {
        if (counts[i] == 0) continue;
        const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]);
        const uintptr_t o = out ? reinterpret_cast<uintptr_t>(out[i]) : g;
        const int32_t od = out ? out_dtypes[i] : dtypes[i];
        spans.push_back({o, o + (uintptr_t)counts[i] * (od == MUON_BF16 ? 2 : 4), true});
        if (o != g || od != dtypes[i])   // a tensor that is its own output counts once
            spans.push_back({g, g + (uintptr_t)counts[i] * (dtypes[i] == MUON_BF16 ? 2 : 4), false});
    }
    std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.from < b.from; });
    uintptr_t read_to = 0, written_to = 0;   // ends of what came before
    for (const Span& s : spans) {
        if (s.from < written_to || (s.written && s.from < read_to)) return true;
        (s.written ? written_to : read_to) = std::max(s.written ? written_to : read_to, s.to);
    }
    return false;
}

}  // namespace

extern "C" {

muon_status muon_act_pack(const void* x, int64_t rows, int64_t cols, int64_t ldx, muon_dtype dtype,
                          const muon_act8* out, void* stream) {
    Call c;
    PackArgs a{};
    MUON_CALL(begin(&c, rows, cols, dtype, kMaxDim));
    c.mat(&a.x, x, ldx, false, rows == 0);
    c.act(&a.q, out, true, false);
    MUON_CALL(c.status());
    if (rows == 0) return MUON_OK;
    a.rows = (uint32_t)rows, a.cols = (int)cols;
    return cuda_status(launch_act_pack(a, dtype == MUON_BF16, c.vec, static_cast<cudaStream_t>(stream)));
}

muon_status muon_act_unpack(const muon_act8* in, int64_t rows, int64_t cols, void* y, int64_t ldy, muon_dtype dtype,
                            void* stream) {
    Call c;
    PackArgs a{};
    MUON_CALL(begin(&c, rows, cols, dtype, kMaxDim));
    c.act(&a.q, in, false, false);
    c.mat(&a.x, y, ldy, true, rows == 0);
    MUON_CALL(c.status());
    if (rows == 0) return MUON_OK;
    a.rows = (uint32_t)rows, a.cols = (int)cols;
    return cuda_status(launch_act_unpack(a, dtype == MUON_BF16, c.vec, static_cast<cudaStream_t>(stream)));
}

muon_status muon_rmsnorm_forward(const void* x, int64_t ldx, const void* residual, int64_t ldr, const float* weight,
                                 int64_t rows, int64_t cols, muon_dtype dtype, float eps, void* h, int64_t ldh,
                                 void* y, int64_t ldy, const muon_act8* saved, int32_t saved_weighted, float* rstd,
                                 void* stream) {
    Call c;
    NormArgs a{};
    MUON_CALL(begin(&c, rows, cols, dtype, kNormMaxCols));
    if (!std::isfinite(eps) || eps <= 0.f || (!h && !y && !saved && !rstd && rows > 0)) return MUON_ERR_INVALID_ARG;
    const int ix = c.mat(&a.x, x, ldx, false, rows == 0), ir = c.mat(&a.residual, residual, ldr, false, true);
    c.mat(&a.h, h, ldh, true, true, 1 << ix | 1 << ir);
    c.mat(&a.y, y, ldy, true, true, 1 << ix);
    c.act(&a.saved, saved, true, true);
    c.vector(weight, cols, false, false);
    c.vector(rstd, rows, true, true);
    MUON_CALL(c.status());
    if (rows == 0) return MUON_OK;
    a.weight = weight, a.rstd = rstd, a.saved_weighted = saved_weighted != 0;
    a.rows = rows, a.cols = (int)cols, a.eps = eps;
    const bool vec = c.vec && aligned16(weight, 0);
    return cuda_status(launch_rmsnorm_forward(a, dtype == MUON_BF16, vec, static_cast<cudaStream_t>(stream)));
}

muon_status muon_swiglu_forward(const void* gate, int64_t ldg, const void* up, int64_t ldu, int64_t rows, int64_t cols,
                                muon_dtype dtype, void* out, int64_t lda, const muon_act8* saved_gate,
                                const muon_act8* saved_up, const muon_act8* saved_out, void* stream) {
    Call c;
    SwigluArgs a{};
    MUON_CALL(begin(&c, rows, cols, dtype, kMaxDim));
    if (!out && !saved_gate && !saved_up && !saved_out && rows > 0) return MUON_ERR_INVALID_ARG;
    const int ig = c.mat(&a.gate, gate, ldg, false, rows == 0), iu = c.mat(&a.up, up, ldu, false, rows == 0);
    c.mat(&a.a, out, lda, true, true, 1 << ig | 1 << iu);
    c.act(&a.gate8, saved_gate, true, true);
    c.act(&a.up8, saved_up, true, true);
    c.act(&a.a8, saved_out, true, true);
    MUON_CALL(c.status());
    if (rows == 0) return MUON_OK;
    a.rows = (uint32_t)rows, a.cols = (int)cols;
    return cuda_status(launch_swiglu_forward(a, dtype == MUON_BF16, c.vec, static_cast<cudaStream_t>(stream)));
}

muon_status muon_swiglu_backward(const void* da, int64_t ldda, const muon_act8* saved_gate, const muon_act8* saved_up,
                                 int64_t rows, int64_t cols, muon_dtype dtype, void* dgate, int64_t lddg, void* dup,
                                 int64_t lddu, const muon_act8* saved_out, void* stream) {
    Call c;
    SwigluArgs a{};
    MUON_CALL(begin(&c, rows, cols, dtype, kMaxDim));
    const int id = c.mat(&a.a, da, ldda, false, rows == 0);
    c.mat(&a.gate, dgate, lddg, true, rows == 0, 1 << id);
    c.mat(&a.up, dup, lddu, true, rows == 0, 1 << id);
    c.act(&a.gate8, saved_gate, false, false);
    c.act(&a.up8, saved_up, false, false);
    c.act(&a.a8, saved_out, true, true);
    MUON_CALL(c.status());
    if (rows == 0) return MUON_OK;
    a.rows = (uint32_t)rows, a.cols = (int)cols;
    return cuda_status(launch_swiglu_backward(a, dtype == MUON_BF16, c.vec, static_cast<cudaStream_t>(stream)));
}

muon_status muon_grad_plan_workspace_size(int64_t* bytes) {
    return muon_grad_plan_workspace_size_ex(kAlignedBytes, bytes);
}

muon_status muon_grad_plan_workspace_size_ex(int64_t aligned_bytes, int64_t* bytes) {
    if (!bytes || aligned_bytes < 0 || aligned_bytes > kMostAligned) return MUON_ERR_INVALID_ARG;
    *bytes = kGradWorkspace + round_up(aligned_bytes, 256);
    return MUON_OK;
}

muon_status muon_grad_plan_create(muon_grad_plan* out) { return muon_grad_plan_create_ex(out, kAlignedBytes); }

muon_status muon_grad_plan_create_ex(muon_grad_plan* out, int64_t aligned_bytes) {
    if (!out) return MUON_ERR_INVALID_ARG;
    *out = nullptr;
    int64_t bytes = 0;
    MUON_CALL(muon_grad_plan_workspace_size_ex(aligned_bytes, &bytes));
    muon_grad_plan_s* p = new (std::nothrow) muon_grad_plan_s;
    if (!p) return MUON_ERR_OOM;
    muon_status st = cuda_status(cudaGetDevice(&p->device));
    if (st == MUON_OK)
        st = cuda_status(cudaDeviceGetAttribute(&p->sm_count, cudaDevAttrMultiProcessorCount, p->device));
    if (st == MUON_OK) {
        const cudaError_t e = cudaMalloc(&p->ws, bytes);
        if (e != cudaSuccess) {
            last_cuda_error() = e;
            (void)cudaGetLastError();
            st = e == cudaErrorMemoryAllocation ? MUON_ERR_OOM : MUON_ERR_CUDA;
        }
    }
    if (st == MUON_OK) st = cuda_status(wgrad_prepare());
    if (st == MUON_OK) st = cuda_status(rmsnorm_prepare());
    if (st == MUON_OK) st = cuda_status(product_prepare());
    if (st == MUON_OK) st = cuda_status(cudaMemset(p->ws, 0, kWsHeader));
    if (st == MUON_OK) st = cuda_status(cudaDeviceSynchronize());
    if (st != MUON_OK) {
        if (p->ws) cudaFree(p->ws);
        delete p;
        return st;
    }
    p->status = static_cast<int*>(p->ws);
    p->arrived = p->status + 1;
    p->running = reinterpret_cast<double*>(p->status + 2);
    p->counters = reinterpret_cast<int*>(static_cast<char*>(p->ws) + 256);
    p->partial = reinterpret_cast<float*>(static_cast<char*>(p->ws) + kWsHeader);
    p->aligned = bytes - kGradWorkspace;
    *out = p;
    return MUON_OK;
}

void muon_grad_plan_destroy(muon_grad_plan p) {
    if (!p) return;
    cudaDeviceSynchronize();
    if (p->ws) cudaFree(p->ws);
    delete p;
}

muon_status muon_grad_plan_sync(muon_grad_plan p, void* stream) {
    MUON_CALL(check_grad_plan(p));
    MUON_TRY(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
    int st = 0;
    MUON_TRY(cudaMemcpy(&st, p->status, sizeof(int), cudaMemcpyDeviceToHost));
    if (st == 0) return MUON_OK;
    MUON_TRY(cudaMemset(p->ws, 0, kWsHeader));   // a call that gave up may have left counters behind
    return MUON_ERR_TIMEOUT;
}

muon_status muon_rmsnorm_backward(muon_grad_plan p, const void* dy, int64_t lddy, const muon_act8* saved,
                                  const void* h, int64_t ldh, const float* rstd, const float* weight, const void* dres,
                                  int64_t lddres, int64_t rows, int64_t cols, muon_dtype dtype, void* dx,
                                  int64_t lddx, float* dweight, int32_t accumulate, void* stream) {
    Call c;
    NormBwdArgs a{};
    MUON_CALL(begin(&c, rows, cols, dtype, kNormMaxCols));
    if (!p || (saved != nullptr && h != nullptr) || (!saved && !h && rows > 0) || (!dx && !dweight && rows > 0))
        return MUON_ERR_INVALID_ARG;
    const int iy = c.mat(&a.dy, dy, lddy, false, rows == 0), ih = c.mat(&a.h, h, ldh, false, true);
    const int ir = c.mat(&a.dres, dres, lddres, false, true);
    c.mat(&a.dx, dx, lddx, true, true, 1 << iy | 1 << ih | 1 << ir);
    c.act(&a.saved, saved, false, true);
    c.vector(weight, cols, false, false);
    c.vector(rstd, rows, false, rows == 0);
    c.vector(dweight, cols, true, true);
    MUON_CALL(c.status());
    MUON_CALL(check_grad_plan(p));
    a.weight = weight, a.rstd = rstd, a.dweight = dweight, a.accumulate = accumulate != 0;
    a.partial = dweight ? p->partial : nullptr;
    a.status = p->status;
    a.rows = (uint32_t)rows, a.cols = (int)cols;
    const bool vec = c.vec && aligned16(weight, 0);
    return cuda_status(
        launch_rmsnorm_backward(a, dtype == MUON_BF16, vec, p->sm_count, static_cast<cudaStream_t>(stream)));
}

muon_status muon_wgrad(muon_grad_plan p, const void* dy, int64_t lddy, const muon_act8* x, int64_t tokens, int64_t m,
                       int64_t n, const int32_t* offsets, int32_t groups, const float* col_scale, void* grad,
                       muon_dtype grad_dtype, int32_t accumulate, void* stream) {
    Call c, cy;
    WgradArgs a{};
    Mat dym{};
    MUON_CALL(begin(&c, tokens, n, grad_dtype, kMaxDim));
    MUON_CALL(begin(&cy, tokens, m, MUON_BF16, kMaxDim));
    if (!p || groups < 0 || groups > 4096 || (groups > 0) != (offsets != nullptr)) return MUON_ERR_INVALID_ARG;
    cy.mat(&dym, dy, lddy, false, tokens == 0);
    if (!cy.ok) return MUON_ERR_INVALID_ARG;
    c.ops.add(dy, tokens, m * 2, lddy * 2, false);
    c.act(&a.x, x, false, tokens == 0);
    c.vector(col_scale, n, false, true);
    c.vector(offsets, groups ? groups + 1 : 0, false, true);
    const int esz = grad_dtype == MUON_BF16 ? 2 : 4;
    c.ok = c.ok && grad && (reinterpret_cast<uintptr_t>(grad) & (esz - 1)) == 0;
    c.ops.add(grad, (long long)std::max(groups, 1) * m, n * esz, n * esz, true);
    MUON_CALL(c.status());
    MUON_CALL(check_grad_plan(p));
    a.dy = dy, a.lddy = lddy, a.tokens = tokens, a.m = (int)m, a.n = (int)n;
    a.offsets = offsets, a.groups = std::max(groups, 1), a.col_scale = col_scale;
    a.grad = grad, a.accumulate = accumulate != 0, a.status = p->status;
    a.partial = p->partial, a.counters = p->counters;
    return cuda_status(launch_wgrad(a, grad_dtype == MUON_BF16, p->sm_count, static_cast<cudaStream_t>(stream)));
}

muon_status muon_product(muon_grad_plan p, const void* x, int64_t ldx, const void* weight, int64_t tokens, int64_t m,
                         int64_t n, const int32_t* offsets, int32_t groups, void* y, int64_t ldy, void* stream) {
    return product(p, x, ldx, weight, tokens, m, n, offsets, groups, y, ldy, false, stream);
}

muon_status muon_dgrad(muon_grad_plan p, const void* dy, int64_t lddy, const void* weight, int64_t tokens, int64_t m,
                       int64_t n, const int32_t* offsets, int32_t groups, void* dx, int64_t lddx, void* stream) {
    return product(p, dy, lddy, weight, tokens, m, n, offsets, groups, dx, lddx, true, stream);
}

muon_status muon_expert_order(const int32_t* ids, int64_t tokens, int32_t choices, int32_t experts, int32_t* offsets,
                              int32_t* slots, void* stream) {
    Call c;
    MUON_CALL(begin_move(&c, tokens, choices, 0, 1, MUON_F32));
    if (experts < 1 || experts > kMostExperts) return MUON_ERR_INVALID_ARG;
    const long long n = (long long)tokens * choices;
    c.vector(ids, n, false, n == 0);
    c.vector(offsets, experts + 1, true, false);
    c.vector(slots, n, true, n == 0);
    MUON_CALL(c.status());
    OrderArgs a{ids, n, experts, offsets, slots};
    return cuda_status(launch_expert_order(a, static_cast<cudaStream_t>(stream)));
}

muon_status muon_expert_dispatch(const void* x, int64_t ldx, const int32_t* slots, int64_t tokens, int32_t choices,
                                 int64_t rows, int64_t cols, muon_dtype dtype, void* out, int64_t ldo, void* stream) {
    Call c;
    MoveArgs a{};
    MUON_CALL(begin_move(&c, tokens, choices, rows, cols, dtype));
    c.mat(&a.x, x, ldx, false, tokens == 0);
    c.rows = rows;
    c.mat(&a.y, out, ldo, true, rows == 0);
    c.vector(slots, (long long)tokens * choices, false, tokens == 0);
    MUON_CALL(c.status());
    if (tokens == 0 || rows == 0) return MUON_OK;
    set_move(&a, slots, nullptr, tokens, choices, rows, cols);
    return cuda_status(launch_expert_dispatch(a, dtype == MUON_BF16, c.vec, static_cast<cudaStream_t>(stream)));
}

muon_status muon_expert_combine(const void* expert_rows, int64_t ldr, const int32_t* slots, const float* weights,
                                int64_t tokens, int32_t choices, int64_t rows, int64_t cols, muon_dtype dtype, void* out,
                                int64_t ldo, void* stream) {
    Call c;
    MoveArgs a{};
    MUON_CALL(begin_move(&c, tokens, choices, rows, cols, dtype));
    c.mat(&a.x, out, ldo, true, tokens == 0);
    c.rows = rows;
    c.mat(&a.y, expert_rows, ldr, false, rows == 0);
    c.vector(slots, (long long)tokens * choices, false, tokens == 0);
    c.vector(weights, (long long)tokens * choices, false, true);
    MUON_CALL(c.status());
    if (tokens == 0) return MUON_OK;
    set_move(&a, slots, weights, tokens, choices, rows, cols);
    return cuda_status(launch_expert_combine(a, dtype == MUON_BF16, c.vec, static_cast<cudaStream_t>(stream)));
}

muon_status muon_expert_combine_backward(const void* dout, int64_t ldd, const int32_t* slots, const float* weights,
                                         const void* expert_rows, int64_t ldr, int64_t tokens, int32_t choices,
                                         int64_t rows, int64_t cols, muon_dtype dtype, void* drows, int64_t lddr,
                                         float* dweights, void* stream) {
    Call c;
    MoveArgs a{};
    MUON_CALL(begin_move(&c, tokens, choices, rows, cols, dtype));
    if (tokens > 0 && ((!drows && !dweights) || (dweights && !expert_rows && rows > 0))) return MUON_ERR_INVALID_ARG;
    c.mat(&a.x, dout, ldd, false, tokens == 0);
    c.rows = rows;
    c.mat(&a.y, expert_rows, ldr, false, true);
    c.mat(&a.dy, drows, lddr, true, true);
    c.vector(slots, (long long)tokens * choices, false, tokens == 0);
    c.vector(weights, (long long)tokens * choices, false, tokens == 0);
    c.vector(dweights, (long long)tokens * choices, true, true);
    MUON_CALL(c.status());
    if (tokens == 0) return MUON_OK;
    set_move(&a, slots, weights, tokens, choices, rows, cols);
    a.dweights = dweights;
    return cuda_status(launch_expert_combine_backward(a, dtype == MUON_BF16, c.vec, static_cast<cudaStream_t>(stream)));
}

muon_status muon_grad_norm(muon_grad_plan p, const void* const* grads, const int64_t* counts, const int32_t* dtypes,
                           int32_t n, float* norm, void* stream) {
    if (!p || !norm || (reinterpret_cast<uintptr_t>(norm) & 3)) return MUON_ERR_INVALID_ARG;
    MUON_CALL(check_list(grads, counts, dtypes, n));
    const uintptr_t at = reinterpret_cast<uintptr_t>(norm);
    for (int i = 0; i < n; ++i) {   // written: not inside a gradient
        const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]);
        if (counts[i] > 0 && g < at + 4 && at < g + (uintptr_t)counts[i] * (dtypes[i] == MUON_BF16 ? 2 : 4))
            return MUON_ERR_INVALID_ARG;
    }
    MUON_CALL(check_grad_plan(p));
    const GradList l{grads, counts, dtypes, nullptr, nullptr, n, false};
    const GradNormArgs a{reinterpret_cast<double*>(p->partial), p->running, p->arrived, norm, p->sm_count};
    return cuda_status(launch_grad_norm(l, a, static_cast<cudaStream_t>(stream)));
}

muon_status muon_grad_clip(muon_grad_plan p, const void* const* grads, const int64_t* counts, const int32_t* dtypes,
                           int32_t n, const float* norm, float max_norm, void* const* out, const int32_t* out_dtypes,
                           void* stream) {
    if (!p || !norm || (reinterpret_cast<uintptr_t>(norm) & 3) || !std::isfinite(max_norm) || max_norm <= 0.f ||
        (out == nullptr) != (out_dtypes == nullptr))
        return MUON_ERR_INVALID_ARG;
    MUON_CALL(check_list(grads, counts, dtypes, n));
    if (out) MUON_CALL(check_list(const_cast<const void* const*>(out), counts, out_dtypes, n));
    try {
        if (lists_overlap(grads, counts, dtypes, n, out, out_dtypes, norm)) return MUON_ERR_INVALID_ARG;
    } catch (const std::bad_alloc&) {
        return MUON_ERR_OOM;
    }
    MUON_CALL(check_grad_plan(p));
    const GradList l{grads, counts, dtypes, out ? out : const_cast<void* const*>(grads), out ? out_dtypes : dtypes, n,
                     out == nullptr};
    return cuda_status(launch_grad_clip(l, norm, max_norm, p->sm_count, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
