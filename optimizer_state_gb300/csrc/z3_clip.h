// z3_clip.h -- argument blocks and launchers of the gradient-clipping kernels
// (z3_clip.cu), shared with the C-ABI entry points (z3_api.cpp).  Not part of
// the public ABI.  As in z3_launch.h, a launcher enqueues and returns the
// launch error; its caller has validated everything.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <vector>

#include "z3_launch.h"

namespace z3 {

// A list of tensors is walked as one run of 16-byte vectors, each tensor
// contributing the aligned vectors that its bytes touch, and the run is cut
// into equal tiles, whatever the tensors' lengths.
constexpr int kSMs = 152;  // of a GB300
constexpr int kListThreads = 256;
constexpr int kListBuckets = 512;

struct ListEntry {
    uint64_t base_kind;  // address rounded down to 16 bytes | z3_dtype
    uint64_t vec0_ends;  // first vector of the run << 8 | head << 4 | tail:
                         // the byte offsets within a vector at which the
                         // tensor starts and (0: on a boundary) ends
};

// One launch's tensors (a kernel parameter).  first[b] is the entry that
// holds vector b << shift, so that a lookup searches between two buckets
// only; entry `count` closes the last tensor.
template <int CAP>
struct ListTab {
    static constexpr int kCap = CAP;
    int32_t count;
    int32_t shift;
    int64_t vecs;
    uint16_t first[kListBuckets + 2];
    ListEntry e[CAP + 1];
};

// The tensors of a table that fills `bytes` of kernel parameters together with
// the kernel's other argument (32 bytes at most).
constexpr int list_cap(int bytes) {
    return (bytes - (int)offsetof(ListTab<0>, e) - 32) / (int)sizeof(ListEntry) - 1;
}

// A table travels with its launch, so its size is host time.  Each size is
// twice the one before, from the classic 4 KB of kernel parameters to the
// 32,764 bytes that sm_103 takes.  A norm of tensors of 5,000 fp32 takes the
// host 4.1 us with 187 of them, 4.2 with 188, 5.4 | 6.2 with 443 | 444, 9.0 | 9.7
// with 955 | 956 and 15.0 with 1,979: always less than the GPU takes (5.2,
// 6.8, 10.0 and 15.7).
using ListTab4 = ListTab<list_cap(4096)>;    //   187 tensors
using ListTab8 = ListTab<list_cap(8192)>;    //   443
using ListTab16 = ListTab<list_cap(16384)>;  //   955
using ListTab32 = ListTab<list_cap(32764)>;  // 1,979

// Device workspace of z3_grad_norm.
constexpr int kNormCtas = 6;                     // resident on an SM
constexpr int kNormMaxGrid = kNormCtas * kSMs;
struct NormWorkspace {
    double partial[kNormMaxGrid];  // one per CTA of a launch
    double carry;                  // sum over the earlier launches of a call
};

}  // namespace z3

// Immutable once built.  Its tables are of the least size that holds all
// tensors in one launch, or several of the largest.
struct z3_tensor_list {
    std::vector<z3_tensor> tensors;     // those with elements
    std::vector<int32_t> index;         // their places in the caller's list
    uintptr_t lo = UINTPTR_MAX, hi = 0; // the addresses they span
    int32_t sums = -1;                  // a tensor that holds sums of squares, if any
    int32_t clash[2] = {-1, -1};        // two tensors that overlap, if any do
    std::vector<z3::ListTab4> tabs4;
    std::vector<z3::ListTab8> tabs8;
    std::vector<z3::ListTab16> tabs16;
    std::vector<z3::ListTab32> tabs32;
};

namespace z3 {

struct NormOut {
    float *clip;  // {norm, coef}
    NormWorkspace *ws;
    float max_norm;
    int32_t first;  // this launch is the call's first: no carry
    int32_t last;   // its last: write clip
};

static_assert(sizeof(NormOut) <= 32 && sizeof(ListTab4) + 32 <= 4096 &&
                  sizeof(ListTab8) + 32 <= 8192 && sizeof(ListTab16) + 32 <= 16384 &&
                  sizeof(ListTab32) + 32 <= 32764,
              "a table and the other argument are one launch's parameters");

struct ReduceNormArgs {
    const uint16_t *grads;  // [N][stride] bf16
    int64_t stride;
    float scale;
    float *grad_shards;
    double *sumsq;  // one per tile, over the layout's reduce tables in order
};

// One launch's units (a kernel parameter); unit i's first CTA is block0[i].
template <int CAP>
struct AdamUnits {
    static constexpr int kCap = CAP;
    int32_t count;
    uint32_t block0[CAP];
    AdamArgs u[CAP];
};

// Tiles of the layout's reduce tables: the length of a sumsq buffer.
inline int64_t sumsq_len(const z3_layout *L) {
    int64_t n = 0;
    for (const Tab &t : L->reduce_tabs) n += t.tiles;
    return n;
}

// Checks the tensors and fills the list (z3_list.cpp); host memory may throw.
z3_status build_list(const char *fn, const z3_tensor *tensors, int32_t n, z3_tensor_list *list);

cudaError_t launch_grad_norm(const z3_tensor_list *list, float max_norm, float *clip,
                             NormWorkspace *ws, cudaStream_t stream);
cudaError_t launch_clip(const z3_tensor_list *list, const float *clip, cudaStream_t stream);
// early: as for launch_reduce (the stream's previous kernel, enqueued by the
// same call, writes none of grads and grad_shards)
cudaError_t launch_reduce_norm(const z3_layout *L, const ReduceNormArgs &a, bool accumulate,
                               cudaStream_t stream, bool early);
// The units' updates, in as few launches as hold them.
cudaError_t launch_adam_clipped(const AdamArgs *a, int32_t n, const float *clip,
                                cudaStream_t stream);

}  // namespace z3
