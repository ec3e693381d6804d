// z3_head_api.cpp -- the entry points of include/z3.h for the losses over a
// vocabulary: argument validation on the host, then the launchers of z3_head.h.
#include <cmath>
#include <new>
#include <string>

#include "z3_check.h"
#include "z3_head.h"

namespace z3 {
namespace {

// A buffer of a call: `bytes` from ptr on, aligned to `align`.
struct Span {
    const void *ptr;
    int64_t bytes;
    const char *name;
    int align;
    bool written;
};

// NULL and misaligned buffers, and written ones that overlap any other.
z3_status check_spans(const char *fn, const Span *b, int n) {
    for (int i = 0; i < n; ++i) {
        if (b[i].bytes == 0) continue;
        auto refuse = [&](z3_status st, const std::string &what) {
            return fail(st, std::string(fn) + ": " + b[i].name + what);
        };
        if (b[i].ptr == nullptr) return refuse(Z3_ERR_INVALID_ARG, " is NULL");
        if (reinterpret_cast<uintptr_t>(b[i].ptr) % (uintptr_t)b[i].align != 0)
            return refuse(Z3_ERR_ALIGNMENT,
                          " is not " + std::to_string(b[i].align) + "-byte aligned");
        for (int j = 0; j < i; ++j) {
            if (b[j].bytes == 0 || !(b[i].written || b[j].written)) continue;
            const uintptr_t x = reinterpret_cast<uintptr_t>(b[i].ptr);
            const uintptr_t y = reinterpret_cast<uintptr_t>(b[j].ptr);
            if (x < y + (uintptr_t)b[j].bytes && y < x + (uintptr_t)b[i].bytes)
                return refuse(Z3_ERR_INVALID_ARG, std::string(" overlaps ") + b[j].name);
        }
    }
    return Z3_OK;
}

// The bytes that `rows` rows of `dim` bf16 values span, `stride` values apart.
z3_status check_matrix(const char *fn, const char *name, int64_t rows, int64_t dim, int64_t stride,
                       int64_t *bytes) {
    auto refuse = [&](z3_status st, const char *what) {
        return fail(st, std::string(fn) + ": " + name + what);
    };
    if (stride < dim) return refuse(Z3_ERR_INVALID_ARG, "_stride < dim");
    if (stride % kVec != 0)
        return refuse(Z3_ERR_ALIGNMENT, "_stride is not a multiple of 8 elements");
    int64_t n;
    // a tensor map's strides have 40 bits
    if (stride >= (1ll << 39) || __builtin_mul_overflow(rows, stride, &n) || n > (1ll << 60))
        return refuse(Z3_ERR_OVERFLOW, " does not fit");
    *bytes = rows ? ((rows - 1) * stride + dim) * 2 : 0;
    return Z3_OK;
}

z3_status check_sizes(const char *fn, int64_t tokens, int64_t dim, int64_t vocab, int64_t k,
                      bool grads, HeadPlan *plan) {
    auto refuse = [&](z3_status st, const std::string &what) {
        return fail(st, std::string(fn) + ": " + what);
    };
    if (tokens < 0) return refuse(Z3_ERR_INVALID_ARG, "tokens < 0");
    if (vocab < 1) return refuse(Z3_ERR_INVALID_ARG, "vocab < 1");
    if (dim < 1) return refuse(Z3_ERR_INVALID_ARG, "dim < 1");
    if (dim % kVec != 0) return refuse(Z3_ERR_INVALID_ARG, "dim is not a multiple of 8");
    if (k < 0 || k > kHeadMaxList)
        return refuse(Z3_ERR_INVALID_ARG,
                      "k is not within 0.." + std::to_string(kHeadMaxList));
    if (!head_plan(tokens, dim, vocab, k, grads, plan))
        return refuse(Z3_ERR_OVERFLOW, "the sizes do not fit");
    return Z3_OK;
}

// What every call takes: fills `a`, and `spans` from 0 on (six of them).
z3_status check_head(const char *fn, const z3_head *h, const void *index, int32_t index_bytes,
                     const z3_teacher *t, bool grads, void *ws, int64_t ws_bytes, HeadArgs *a,
                     Span *spans) {
    auto refuse = [&](const std::string &what) {
        return fail(Z3_ERR_INVALID_ARG, std::string(fn) + ": " + what);
    };
    if (h == nullptr) return refuse("head is NULL");
    a->temperature = 1.0f;
    int64_t k = 0;
    if (t != nullptr) {
        k = t->k;
        if (k < 1 || k > kHeadMaxList)
            return refuse("k is not within 1.." + std::to_string(kHeadMaxList));
        if (t->dtype != Z3_BF16 && t->dtype != Z3_F32)
            return refuse("the teacher's logits are Z3_BF16 or Z3_F32");
        const float tau = t->temperature;
        if (!(tau > 0.0f) || !std::isfinite(tau * tau) || !std::isfinite(2.0f / tau))
            return refuse("temperature");
        index = t->index;
        index_bytes = t->index_bytes;
        a->teacher = t->logits;
        a->teacher_bytes = t->dtype == Z3_BF16 ? 2 : 4;
        a->temperature = tau;
    }
    if (index_bytes != 4 && index_bytes != 8)
        return refuse("index_bytes must be 4 or 8");
    z3_status st = check_sizes(fn, h->tokens, h->dim, h->vocab, k, grads, &a->plan);
    if (st != Z3_OK) return st;
    if (ws_bytes < a->plan.bytes)
        return refuse("the workspace has " + std::to_string(ws_bytes) + " bytes, needs " +
                      std::to_string(a->plan.bytes));
    int64_t hb, wb;
    if ((st = check_matrix(fn, "hidden", h->tokens, h->dim, h->hidden_stride, &hb)) != Z3_OK ||
        (st = check_matrix(fn, "weight", h->vocab, h->dim, h->weight_stride, &wb)) != Z3_OK)
        return st;
    const int64_t entries = h->tokens * (t ? k : 1);
    spans[0] = {h->hidden, hb, "hidden", 16, false};
    spans[1] = {h->weight, wb, "weight", 16, false};
    spans[2] = {h->weights, h->weights ? 4 * h->tokens : 0, "weights", 4, false};
    spans[3] = {index, entries * index_bytes, t ? "index" : "targets", index_bytes, false};
    spans[4] = {a->teacher, t ? entries * a->teacher_bytes : 0, "logits",
                t ? a->teacher_bytes : 1, false};
    spans[5] = {ws, a->plan.bytes, "workspace", 16, true};
    a->hidden = h->hidden;
    a->hidden_stride = h->hidden_stride;
    a->weight = h->weight;
    a->weight_stride = h->weight_stride;
    a->weights = h->weights;
    a->index = index;
    a->index_bytes = index_bytes;
    a->ws = static_cast<char *>(ws);
    return Z3_OK;
}

z3_status forward(const char *fn, const char *range, const z3_head *h, const void *targets,
                  int32_t index_bytes, const z3_teacher *t, float *loss, float *lse, float *total,
                  void *ws, int64_t ws_bytes, z3_stream stream) {
    HeadArgs a{};
    Span spans[9];
    z3_status st = check_head(fn, h, targets, index_bytes, t, false, ws, ws_bytes, &a, spans);
    if (st != Z3_OK) return st;
    spans[6] = {loss, 4 * h->tokens, "loss", 4, true};
    spans[7] = {lse, 4 * h->tokens, "lse", 4, true};
    spans[8] = {total, 8, "total", 4, true};
    if ((st = check_spans(fn, spans, 9)) != Z3_OK) return st;
    a.loss = loss;
    a.lse = lse;
    a.total = total;
    Range r(range);
    return launched(fn, launch_head_forward(a, (cudaStream_t)stream));
}

z3_status gradient(const char *fn, const char *range, const z3_head *h, const void *targets,
                   int32_t index_bytes, const z3_teacher *t, const float *lse, const float *total,
                   float scale, uint16_t *d_hidden, int64_t d_hidden_stride, uint16_t *d_weight,
                   int64_t d_weight_stride, void *ws, int64_t ws_bytes, z3_stream stream) {
    HeadArgs a{};
    Span spans[10];
    if (!std::isfinite(scale)) return fail(Z3_ERR_INVALID_ARG, std::string(fn) + ": scale");
    z3_status st = check_head(fn, h, targets, index_bytes, t, true, ws, ws_bytes, &a, spans);
    if (st != Z3_OK) return st;
    int64_t hb = 0, wb = 0;
    if (d_hidden)
        st = check_matrix(fn, "d_hidden", h->tokens, h->dim, d_hidden_stride, &hb);
    if (st == Z3_OK && d_weight)
        st = check_matrix(fn, "d_weight", h->vocab, h->dim, d_weight_stride, &wb);
    if (st != Z3_OK) return st;
    spans[6] = {lse, 4 * h->tokens, "lse", 4, false};
    spans[7] = {total, total ? 8 : 0, "total", 4, false};
    spans[8] = {d_hidden, hb, "d_hidden", 16, true};
    spans[9] = {d_weight, wb, "d_weight", 16, true};
    if ((st = check_spans(fn, spans, 10)) != Z3_OK) return st;
    if (d_hidden == nullptr && d_weight == nullptr) return Z3_OK;
    a.lse = const_cast<float *>(lse);
    a.total = const_cast<float *>(total);
    a.scale = scale;
    a.d_hidden = d_hidden;
    a.d_hidden_stride = d_hidden_stride;
    a.d_weight = d_weight;
    a.d_weight_stride = d_weight_stride;
    Range r(range);
    return launched(fn, launch_head_grad(a, (cudaStream_t)stream));
}

}  // namespace
}  // namespace z3

using namespace z3;

extern "C" z3_status z3_head_workspace_bytes(int64_t tokens, int64_t dim, int64_t vocab, int32_t k,
                                             int32_t grads, int64_t *bytes) {
    const char *fn = "z3_head_workspace_bytes";
    try {
        if (bytes == nullptr)
            return fail(Z3_ERR_INVALID_ARG, "z3_head_workspace_bytes: bytes is NULL");
        HeadPlan plan;
        const z3_status st = check_sizes(fn, tokens, dim, vocab, k, grads != 0, &plan);
        if (st == Z3_OK) *bytes = plan.bytes;
        return st;
    } catch (const std::bad_alloc &) {
        return fail_host_memory(fn);
    }
}

extern "C" z3_status z3_xent(const z3_head *head, const void *targets, int32_t index_bytes,
                             float *loss, float *lse, float *total, void *workspace,
                             int64_t workspace_bytes, z3_stream stream) {
    const char *fn = "z3_xent";
    try {
        return forward(fn, "z3/xent", head, targets, index_bytes, nullptr, loss, lse, total,
                       workspace, workspace_bytes, stream);
    } catch (const std::bad_alloc &) {
        return fail_host_memory(fn);
    }
}

extern "C" z3_status z3_xent_grad(const z3_head *head, const void *targets, int32_t index_bytes,
                                  const float *lse, const float *total_or_NULL, float scale,
                                  uint16_t *d_hidden_or_NULL, int64_t d_hidden_stride,
                                  uint16_t *d_weight_or_NULL, int64_t d_weight_stride,
                                  void *workspace, int64_t workspace_bytes, z3_stream stream) {
    const char *fn = "z3_xent_grad";
    try {
        return gradient(fn, "z3/xent_grad", head, targets, index_bytes, nullptr, lse,
                        total_or_NULL, scale, d_hidden_or_NULL, d_hidden_stride, d_weight_or_NULL,
                        d_weight_stride, workspace, workspace_bytes, stream);
    } catch (const std::bad_alloc &) {
        return fail_host_memory(fn);
    }
}

extern "C" z3_status z3_distill(const z3_head *head, const z3_teacher *teacher, float *loss,
                                float *lse, float *total, void *workspace,
                                int64_t workspace_bytes, z3_stream stream) {
    const char *fn = "z3_distill";
    try {
        if (teacher == nullptr) return fail(Z3_ERR_INVALID_ARG, "z3_distill: teacher is NULL");
        return forward(fn, "z3/distill", head, nullptr, 0, teacher, loss, lse, total, workspace,
                       workspace_bytes, stream);
    } catch (const std::bad_alloc &) {
        return fail_host_memory(fn);
    }
}

extern "C" z3_status z3_distill_grad(const z3_head *head, const z3_teacher *teacher,
                                     const float *lse, const float *total_or_NULL, float scale,
                                     uint16_t *d_hidden_or_NULL, int64_t d_hidden_stride,
                                     uint16_t *d_weight_or_NULL, int64_t d_weight_stride,
                                     void *workspace, int64_t workspace_bytes, z3_stream stream) {
    const char *fn = "z3_distill_grad";
    try {
        if (teacher == nullptr) return fail(Z3_ERR_INVALID_ARG, "z3_distill_grad: teacher is NULL");
        return gradient(fn, "z3/distill_grad", head, nullptr, 0, teacher, lse, total_or_NULL, scale,
                        d_hidden_or_NULL, d_hidden_stride, d_weight_or_NULL, d_weight_stride,
                        workspace, workspace_bytes, stream);
    } catch (const std::bad_alloc &) {
        return fail_host_memory(fn);
    }
}
