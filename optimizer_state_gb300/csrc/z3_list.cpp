// z3_list.cpp -- host side of a list of tensors: the checks, and the launch
// tables of the kernels that walk it (z3_clip.cu).
#include <algorithm>
#include <new>
#include <string>

#include "z3_clip.h"

namespace z3 {
namespace {

int64_t dtype_bytes(int32_t dtype) { return dtype == Z3_BF16 ? 2 : dtype == Z3_F32 ? 4 : 8; }

uintptr_t begin_of(const z3_tensor &t) { return reinterpret_cast<uintptr_t>(t.data); }
uintptr_t end_of(const z3_tensor &t) {
    return begin_of(t) + (uintptr_t)(t.numel * dtype_bytes(t.dtype));
}

// Fills tab from ts[at...], as many as it holds; returns the next index.
template <typename TAB>
size_t fill(TAB &tab, const std::vector<z3_tensor> &ts, size_t at) {
    tab.count = 0;
    int64_t vecs = 0;
    for (; at < ts.size() && tab.count < TAB::kCap; ++at) {
        const uint64_t a = begin_of(ts[at]), z = end_of(ts[at]);
        ListEntry &e = tab.e[tab.count++];
        e.base_kind = (a & ~(uint64_t)15) | (uint64_t)ts[at].dtype;
        e.vec0_ends = (uint64_t)vecs << 8 | (a & 15) << 4 | (z & 15);
        vecs += (int64_t)((z + 15) / 16 - a / 16);
    }
    tab.e[tab.count].base_kind = 0;
    tab.e[tab.count].vec0_ends = (uint64_t)vecs << 8;
    tab.vecs = vecs;
    tab.shift = 0;
    while ((vecs >> tab.shift) >= kListBuckets) ++tab.shift;
    int32_t i = 0;
    for (int64_t b = 0; b <= (vecs >> tab.shift) + 1; ++b) {
        while (i + 1 < tab.count && (int64_t)(tab.e[i + 1].vec0_ends >> 8) <= b << tab.shift) ++i;
        tab.first[b] = (uint16_t)i;
    }
    return at;
}

template <typename TAB>
void fill_all(std::vector<TAB> &tabs, const std::vector<z3_tensor> &ts) {
    size_t at = 0;
    do {
        tabs.emplace_back();
        at = fill(tabs.back(), ts, at);
    } while (at < ts.size());
}

// Two tensors that overlap, if any do: neighbours in the order of addresses.
void find_clash(z3_tensor_list *list) {
    const std::vector<z3_tensor> &ts = list->tensors;
    std::vector<int32_t> order(ts.size());
    for (size_t i = 0; i < ts.size(); ++i) order[i] = (int32_t)i;
    std::sort(order.begin(), order.end(),
              [&](int32_t a, int32_t b) { return begin_of(ts[a]) < begin_of(ts[b]); });
    for (size_t k = 1; k < order.size(); ++k)
        if (begin_of(ts[order[k]]) < end_of(ts[order[k - 1]])) {
            list->clash[0] = list->index[order[k]];
            list->clash[1] = list->index[order[k - 1]];
            return;
        }
}

}  // namespace

z3_status build_list(const char *fn, const z3_tensor *tensors, int32_t n, z3_tensor_list *list) {
    auto at = [&](int32_t i) {
        return std::string(fn) + ": tensors[" + std::to_string(i) + "]";
    };
    if (n < 0) return fail(Z3_ERR_INVALID_ARG, std::string(fn) + ": n < 0");
    if (n > 0 && tensors == nullptr)
        return fail(Z3_ERR_INVALID_ARG, std::string(fn) + ": tensors is NULL");
    list->tensors.reserve((size_t)n);
    list->index.reserve((size_t)n);
    for (int32_t i = 0; i < n; ++i) {
        const z3_tensor &t = tensors[i];
        if (t.dtype != Z3_BF16 && t.dtype != Z3_F32 && t.dtype != Z3_SUMSQ)
            return fail(Z3_ERR_INVALID_ARG, at(i) + ": unknown dtype");
        if (t.numel < 0) return fail(Z3_ERR_INVALID_ARG, at(i) + ": numel < 0");
        if (t.dtype == Z3_SUMSQ && list->sums < 0) list->sums = i;
        if (t.numel == 0) continue;
        if (t.data == nullptr) return fail(Z3_ERR_INVALID_ARG, at(i) + ": data is NULL");
        const int64_t size = dtype_bytes(t.dtype);
        const uintptr_t lo = begin_of(t);
        int64_t bytes;
        uintptr_t hi;
        // addresses stay far below 2^55, the widest that an entry's vectors hold
        if (__builtin_mul_overflow(t.numel, size, &bytes) ||
            __builtin_add_overflow(lo, (uintptr_t)bytes, &hi) || hi > (uintptr_t)INT64_MAX >> 8)
            return fail(Z3_ERR_OVERFLOW, at(i) + ": size overflows");
        if (lo % (uintptr_t)size != 0)
            return fail(Z3_ERR_ALIGNMENT, at(i) + " is not aligned to its elements");
        list->tensors.push_back(t);
        list->index.push_back(i);
        list->lo = std::min(list->lo, lo);
        list->hi = std::max(list->hi, hi);
    }
    find_clash(list);
    const size_t count = list->tensors.size();
    if (count <= (size_t)ListTab4::kCap) fill_all(list->tabs4, list->tensors);
    else if (count <= (size_t)ListTab8::kCap) fill_all(list->tabs8, list->tensors);
    else if (count <= (size_t)ListTab16::kCap) fill_all(list->tabs16, list->tensors);
    else fill_all(list->tabs32, list->tensors);
    return Z3_OK;
}

}  // namespace z3

using namespace z3;

extern "C" z3_status z3_tensor_list_create(const z3_tensor *tensors, int32_t n,
                                           z3_tensor_list **out) {
    const char *fn = "z3_tensor_list_create";
    if (out == nullptr) return fail(Z3_ERR_INVALID_ARG, std::string(fn) + ": out is NULL");
    *out = nullptr;
    z3_tensor_list *list = nullptr;
    try {
        list = new z3_tensor_list();
        const z3_status st = build_list(fn, tensors, n, list);
        if (st == Z3_OK) *out = list;
        else delete list;
        return st;
    } catch (const std::bad_alloc &) {
        delete list;
        return fail_host_memory(fn);
    }
}

extern "C" void z3_tensor_list_destroy(z3_tensor_list *list) { delete list; }
