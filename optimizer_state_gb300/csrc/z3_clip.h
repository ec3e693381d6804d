// z3_clip.h -- argument blocks and launchers of the gradient-clipping kernels
// (z3_clip.cu), shared with the C-ABI entry points (z3_api.cpp).  Not part of
// the public ABI.  As in z3_launch.h, a launcher enqueues and returns the
// launch error; its caller has validated everything.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "z3_launch.h"

namespace z3 {

// A list of tensors is walked as one run of 16-byte vectors, each tensor
// contributing the aligned vectors that its bytes touch, and the run is cut
// into tiles of kListTile vectors, whatever the tensors' lengths.
constexpr int kSMs = 152;
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

// The first size stays within the classic 4 KB of kernel parameters, the
// last within the 32,764 bytes that sm_103 takes; copying a table to the GPU
// costs a launch 3 us at the last size.
using ListSmall = ListTab<180>;
using ListMedium = ListTab<700>;
using ListLarge = ListTab<1900>;

// Device workspace of z3_grad_norm.
constexpr int kNormCtas = 7;                     // resident on an SM
constexpr int kNormMaxGrid = kNormCtas * kSMs;
struct NormWorkspace {
    double partial[kNormMaxGrid];  // one per CTA of a launch
    double carry;                  // sum over the earlier launches of a call
};

struct NormOut {
    float *clip;  // {norm, coef}
    NormWorkspace *ws;
    float max_norm;
    int32_t first;  // this launch is the call's first: no carry
    int32_t last;   // its last: write clip
    int32_t alone;  // both, with one CTA: no partials
};

struct ReduceNormArgs {
    const uint16_t *__restrict__ grads;  // [N][stride] bf16
    int64_t stride;
    float scale;
    float *grad_shards;
    double *sumsq;  // one per tile, over the layout's reduce tables in order
};

struct AdamClipArgs {
    AdamArgs a;
    const float *clip;
};

// Bytes of one element of a listed tensor.
inline int64_t list_dtype_bytes(int32_t dtype) {
    return dtype == Z3_BF16 ? 2 : dtype == Z3_F32 ? 4 : 8;
}

// Tiles of the layout's reduce tables: the length of a sumsq buffer.
inline int64_t sumsq_len(const z3_layout *L) {
    int64_t n = 0;
    for (const Tab &t : L->reduce_tabs) n += t.tiles;
    return n;
}

cudaError_t launch_grad_norm(const z3_tensor *tensors, int32_t n, float max_norm, float *clip,
                             NormWorkspace *ws, cudaStream_t stream);
cudaError_t launch_clip(const z3_tensor *tensors, int32_t n, const float *clip,
                        cudaStream_t stream);
// early: as for launch_reduce (the stream's previous kernel, enqueued by the
// same call, writes none of grads and grad_shards)
cudaError_t launch_reduce_norm(const z3_layout *L, const ReduceNormArgs &a, bool accumulate,
                               cudaStream_t stream, bool early);
// early: the previous kernel writes none of master, m, v, the gradient and clip
cudaError_t launch_adam_clipped(const AdamClipArgs &a, cudaStream_t stream, bool early);

}  // namespace z3
