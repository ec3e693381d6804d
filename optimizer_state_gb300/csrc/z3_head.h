// z3_head.h -- sizes, argument blocks and launchers of the losses over a
// vocabulary (z3_head.cu), shared with their entry points (z3_head_api.cpp).
// Not part of the public ABI.  As in z3_launch.h, a launcher enqueues and
// returns the launch error; its caller has validated everything.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "z3_internal.h"

namespace z3 {

constexpr int kHeadSMs = 152;      // of a GB300
constexpr int kHeadMaxList = 1024; // a token's teacher logits
// Values of a row.  A tile of logits sums whole rows, 64 values in 1,400 clocks
// where they come from memory: 7.4e8 clocks at most, of the 4e9 that a wait takes.
constexpr int64_t kHeadMaxDim = 1ll << 25;

// A grid of products: how a [M][N] result of depth K is cut into tiles, and the
// depth of a tile into splits.
struct Cut {
    int32_t cg;        // CTAs to a tile
    int32_t swap;      // rows and columns are exchanged (few tokens)
    int32_t tile_m;    // rows of a CTA's: 128, or with swap fewer
    int32_t bn;        // columns of a tile
    int32_t m_tiles, n_tiles;
    int32_t k_tiles;   // of 64
    int32_t k_chunk;   // k tiles of a split
    int32_t splits;
};

// The sizes of a call and its workspace.
struct HeadPlan {
    int64_t tokens, vocab, dim, k;
    Cut logits;          // [tokens][vocab] of depth dim, in the forward calls
    int32_t parts;       // maxima and sums that its tiles leave of a token
    int64_t piece;       // words of a piece (a multiple of 256)
    int64_t pieces;
    // byte offsets into the workspace
    int64_t part;        // float2 [parts][tokens]: maximum, sum of exponentials
    int64_t z;           // float [tokens][max(k, 1)]: logits of the target or the list
    int64_t sums;        // float4 [blocks]: the join's
    int64_t done;        // int: joined blocks
    int64_t state;       // int8 [tokens]: Row
    int64_t index, q;    // int32, float [tokens][k]: the list by ascending word
    int64_t first;       // uint16 [tokens][..]: where the entries of some words begin
    int64_t rows;        // float2 [tokens]: factor, lse * log2 e
    int64_t words;       // int32 [tokens]: the target
    int64_t target;      // float [tokens]: dz there
    int64_t hidden;      // bf16 [tokens][hidden_pitch]: zero where the row is left out
    int64_t hidden_pitch;
    int64_t dz;          // bf16 [tokens][piece]
    int64_t slab_h;      // float [splits][tokens][dim]
    int64_t slab_w;      // float [splits][piece][dim]
    int64_t bytes;
};

// False where a size does not fit.
bool head_plan(int64_t tokens, int64_t dim, int64_t vocab, int64_t k, bool grads, HeadPlan *p);

enum Row : int8_t { kLeftOut = 0, kCounts = 1, kBad = 2 };

struct HeadArgs {
    HeadPlan plan;
    const uint16_t *hidden;
    int64_t hidden_stride;
    const uint16_t *weight;
    int64_t weight_stride;
    const float *weights;      // or null
    const void *index;         // targets [tokens], or the lists [tokens][k]
    int32_t index_bytes;       // 4 or 8
    const void *teacher;       // [tokens][k]; null: cross entropy
    int32_t teacher_bytes;     // 2 or 4
    float temperature;
    char *ws;
    // forward
    float *loss, *lse, *total;
    // gradient: lse and total (or null) are read
    float scale;
    uint16_t *d_hidden;        // or null
    int64_t d_hidden_stride;
    uint16_t *d_weight;        // or null
    int64_t d_weight_stride;
};

cudaError_t launch_head_forward(const HeadArgs &a, cudaStream_t s);
cudaError_t launch_head_grad(const HeadArgs &a, cudaStream_t s);

}  // namespace z3
