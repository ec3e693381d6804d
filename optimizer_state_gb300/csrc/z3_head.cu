// z3_head.cu -- softmax cross entropy and distillation over a large
// vocabulary, whose logits are never stored.
//
// With z = hidden weight^T, a forward call is one product whose epilogue keeps
// of each tile only every row's maximum and sum of exponentials (and the few
// logits that the row's target or list names); k_head_join joins the tiles.
// A gradient call walks the vocabulary in pieces: the piece's logits are
// computed once more, their epilogue turns them into dz (bf16, in the
// workspace), and two products of dz give this piece's rows of d_weight and
// its share of d_hidden.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "z3_device.cuh"
#include "z3_head.h"
#include "z3_mma.cuh"

namespace z3 {
namespace {

constexpr int kBK = 64;           // values of K in a stage: one swizzled row of 128 bytes
constexpr int kEpilogueWarps = 8;
constexpr int kMmaThreads = 128 + 32 * kEpilogueWarps;  // TMA, products, tensor memory, -
constexpr int kGrain = 128;       // words: a list's entries are found by these
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// --------------------------------------------------------------------------
// the tiled product
// --------------------------------------------------------------------------

// What becomes of a result's tiles: each row's maximum and sum of exponentials;
// the gradient of the logits; the values themselves.
enum Kind : int32_t { kStats, kDz, kOut };

// One product D[m][n] = sum_k A(m, k) B(n, k), by tiles that persistent CTAs take
// in turn.
struct Job {
    CUtensorMap a, b, out;
    Cut cut;
    int32_t steps;         // of 16 values in the last k tile
    int32_t a_mn;          // kOut without SWAP: a's rows run along M rather than K ...
    int32_t box_k;         // ... and boxes of a and b hold this many of K's
    int32_t n_fast;        // walk a row of tiles before the next row
    int32_t a_m, a_k;      // where in the maps this product begins
    int32_t b_n, b_k;
    uint16_t *out_at;      // kOut: the bf16 result
    int64_t out_pitch;
    int32_t out_f32;       // binary32 results instead, by split
    int32_t add;           // kOut: added to what is there
    int64_t rows, cols;    // tokens x words, or the rows and columns of kOut's result
};

// The splits' sums of a result [rows][cols], rounded once to bf16.
struct Slabs {
    const float *slab;     // [splits][rows][cols]; null: none to join
    int32_t splits;
    int64_t rows, cols;
    uint16_t *out;
    int64_t pitch;
};

struct Sum8 {
    float4 a, b;
    __device__ __forceinline__ Sum8() : a(make_float4(0.0f, 0.0f, 0.0f, 0.0f)), b(a) {}
    __device__ __forceinline__ void add(const float4 &x, const float4 &y) {
        a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
        b.x += y.x; b.y += y.y; b.z += y.z; b.w += y.w;
    }
};

// Every `step`-th split's eight values from i on, `first` the first.
__device__ __forceinline__ Sum8 sum_splits(const Slabs &p, int64_t i, int first, int step) {
    Sum8 x;
    const int64_t stride = p.rows * p.cols;
#pragma unroll 8
    for (int s = first; s < p.splits; s += step) {
        const float4 *f = reinterpret_cast<const float4 *>(p.slab + s * stride + i);
        x.add(f[0], f[1]);
    }
    return x;
}

__device__ __forceinline__ void store_sum(const Slabs &p, int64_t i, const Sum8 &x) {
    const int64_t r = i / p.cols, c = i - r * p.cols;
    *reinterpret_cast<uint4 *>(p.out + r * p.pitch + c) =
        make_uint4(pack_bf16x2(x.a.x, x.a.y), pack_bf16x2(x.a.z, x.a.w),
                   pack_bf16x2(x.b.x, x.b.y), pack_bf16x2(x.b.z, x.b.w));
}

struct MmaArgs {
    // JOINT: the first product's tiles go round the groups, which leaves the first
    // `more` groups with one more than the others.  The second's go round the
    // others `ahead` times, then round all.
    Job job[2];
    int32_t more, ahead;
    int32_t early;         // the operands may be read before the kernel before has ended
    Slabs join;            // kOut without SWAP: what the launch before left to join
    // kStats, kDz
    float beta;            // log2(e) / temperature: exponents are powers of two
    int32_t word0;         // the word of column 0
    int32_t k;             // list length
    int32_t first_pitch;
    const int32_t *index;  // lists by ascending word, where each grain's entries begin
    const float *q;
    const uint16_t *first;
    // kStats
    float2 *part;
    float *z;
    unsigned *done;        // zeroed for the join
    const void *targets;
    int32_t target_bytes;
    const uint16_t *hidden, *weight;
    int64_t hidden_stride, weight_stride, vocab;
    int32_t dim;
    // kDz
    const float2 *row;
    const int32_t *words;
    const float *target;   // dz at the target
    uint16_t *dz;
    int64_t dz_pitch;
};

__device__ __forceinline__ int64_t load_index(const void *p, int bytes, int64_t i) {
    return bytes == 8 ? static_cast<const int64_t *>(p)[i]
                      : (int64_t)static_cast<const int32_t *>(p)[i];
}

// The logit of a token's target, by LANES neighbours of a warp.  Products of bf16
// are exact, their sums rounded to nearest, in the same order for every LANES: 256
// chains, eight to each of 32 places, joined by a tree.  So the loss, the gradient
// and lse between them are of one logit.
template <int LANES>
__device__ __forceinline__ float target_logit(const uint16_t *x, const uint16_t *y, int64_t dim,
                                              int lane) {
    constexpr int kPlaces = 32 / LANES;  // of a lane: every LANES-th
    float s[kPlaces][8] = {};
#pragma unroll LANES / 4
    for (int64_t i = lane % LANES * 8; i < dim; i += 256) {
#pragma unroll
        for (int n = 0; n < kPlaces; ++n) {
            const int64_t at = i + n * LANES * 8;
            if (at >= dim) break;
            float a[8], b[8];
            unpack8(ld8b(x + at), a);
            unpack8(ld8b(y + at), b);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[n][j] = __fmaf_rn(a[j], b[j], s[n][j]);
        }
    }
    float z[kPlaces];
#pragma unroll
    for (int n = 0; n < kPlaces; ++n)
        z[n] = ((s[n][0] + s[n][1]) + (s[n][2] + s[n][3])) +
               ((s[n][4] + s[n][5]) + (s[n][6] + s[n][7]));
#pragma unroll
    for (int o = kPlaces / 2; o > 0; o /= 2)  // places 16 lanes apart, then 8
#pragma unroll
        for (int n = 0; n < o; ++n) z[n] += z[n + o];
    const unsigned lanes = LANES == 32 ? ~0u : (0xffu << (lane & 24));
#pragma unroll
    for (int o = LANES / 2; o > 0; o /= 2) z[0] += __shfl_xor_sync(lanes, z[0], o);
    return z[0];
}

template <int BN, int CG>
__host__ __device__ constexpr int stage_bytes() {
    return 128 * kBK * 2 + BN / CG * kBK * 2;
}
template <int BN, int CG>
__host__ __device__ constexpr int stages() {
    return 196608 / stage_bytes<BN, CG>();
}
constexpr int kStaging = 4096;  // a warp's: 32 rows of 128 bytes
constexpr int kSmem = 196608 + kEpilogueWarps * kStaging + 1024 + 512;
static_assert(kSmem <= 232448 && kSmem > 116736,
              "fits an SM, and no second CTA beside it competes for its tensor memory");

template <int N>
struct Steps {
    static constexpr int value = N;
};

struct Tile {
    int m, n, split;
};

__device__ __forceinline__ Tile tile_of(const Job &jb, int item) {
    const int tiles = jb.cut.m_tiles * jb.cut.n_tiles;
    Tile t;
    t.split = item / tiles;
    int i = item - t.split * tiles;
    if (jb.n_fast) {
        t.m = i / jb.cut.n_tiles;
        t.n = i - t.m * jb.cut.n_tiles;
    } else {
        constexpr int kGroup = 32;  // row tiles whose operand stays in L2
        const int per = kGroup * jb.cut.n_tiles;
        const int g = i / per;
        const int rows = min(kGroup, jb.cut.m_tiles - g * kGroup);
        i -= g * per;
        t.n = i / rows;
        t.m = g * kGroup + i - t.n * rows;
    }
    return t;
}

// The value at a place of a thread's own choice among its registers: by the
// place's bits, 31 selections.
__device__ __forceinline__ float pick(const float (&v)[32], uint32_t j) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = (j & 1) ? v[2 * i + 1] : v[2 * i];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (j & 2) ? x[2 * i + 1] : x[2 * i];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (j & 4) ? x[2 * i + 1] : x[2 * i];
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = (j & 8) ? x[2 * i + 1] : x[2 * i];
    x[0] = (j & 16) ? x[1] : x[0];
    return x[0];
}

// The entries of a token's list (or its target) among some columns of a
// tile, in turn.  The next four are held, so that hardly any load is waited for
// where an entry is met (with one, 501 lists of 200 over 32003 words took 59
// us to turn into dz, 44 with four).
template <bool LIST, bool Q>
struct Walk {
    static constexpr int kNone = 0x7fffffff;
    static constexpr int kHeld = LIST ? 4 : 1;
    int column[kHeld];
    float share[kHeld];  // q
    int at, end, word0;
    const int32_t *index;
    const float *q;

    __device__ __forceinline__ Walk() : at(0), end(0), word0(0), index(nullptr), q(nullptr) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            column[i] = kNone;
            share[i] = 1.0f;
        }
    }
    __device__ __forceinline__ int next() const { return column[0]; }
    __device__ __forceinline__ void load(int i) {
        const bool there = at + i < end;
        column[i] = there ? index[at + i] - word0 : kNone;
        if constexpr (Q)
            if (there) share[i] = q[at + i];
    }
    __device__ __forceinline__ void advance() {
#pragma unroll
        for (int i = 0; i + 1 < kHeld; ++i) {
            column[i] = column[i + 1];
            share[i] = share[i + 1];
        }
        if constexpr (LIST) {
            ++at;
            load(kHeld - 1);
        } else {
            column[0] = kNone;
        }
    }
};

// A warp's box of 32 rows of 128 bytes goes out, where it meets the result at all.
__device__ __forceinline__ void store_box(const Job &jb, uint32_t stage, int lane, int col,
                                          int64_t row, int split) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0 && row < jb.rows && col < jb.cols)
        tma_store(&jb.out, stage, col, (int)row, split, jb.add != 0);
}

// The staging rows may be written again.
__device__ __forceinline__ void await_box(int lane) {
    if (lane == 0) tma_wait_read();
    __syncwarp();
}

// 64 columns of this thread's row as bf16 into the staging rows; or the first 32
// straight to the result, where a tile ends with half a box and the next
// tile's columns lie behind it.
__device__ __forceinline__ void put64(uint32_t stage, int lane, const uint32_t (&w)[32], bool part,
                                      bool live, uint16_t *out) {
    if (part) {
        if (!live) return;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4 *>(out + 8 * j) =
                make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        return;
    }
    await_box(lane);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        st_shared(stage + lane * 128 + ((j ^ (lane & 7)) << 4), w[4 * j], w[4 * j + 1],
                  w[4 * j + 2], w[4 * j + 3]);
}

// D tile by tile: 128 x CG rows by BN columns.  One thread feeds TMA, one issues
// the products, eight warps take a finished tile out of tensor memory (a
// quarter of a CTA's rows, half of the columns each) while the next one is
// computed beside it.
// SWAP, for few tokens: M runs along words (or, for d_hidden, along its columns)
// and N along tokens, so that the weight fills the tiles; a warp turns its 32
// x 32 values over in shared memory, after which thread, row and columns mean
// what they mean without SWAP.
// Bound by the tensor cores: 256 x 256 values of one k tile take 528 clocks, 512
// at their nominal rate.  6 stages of 64 values of K hide L2's latency; the
// epilogue takes 2,800 clocks a tile beside the next one's products (8,450 at
// depth 1024), which it slows by 7%.  4608 x 32768 x 1024: 168 us, 1.84
// PFLOP/s; in long calls the power limit sets the clocks.
// Every wait ends (mbar_wait); an epilogue whose tile did not come takes NaN for
// its values.
// AMN, BMN: an operand's rows run along M or N rather than K.
// JOINT: d_hidden and d_weight in one launch, whose tiles fill each other's last
// wave; a's rows run either way, by job.
template <int CG, int BN, bool SWAP, bool AMN, bool BMN, Kind KIND, bool LIST, bool JOINT>
__global__ void __launch_bounds__(kMmaThreads, 1)
k_head_mma(const __grid_constant__ MmaArgs p) {
    constexpr int S = stages<BN, CG>();
    constexpr int kA = 128 * kBK * 2;
    constexpr int kStage = stage_bytes<BN, CG>();
    constexpr int kCols = 2 * BN;    // of tensor memory: two tiles
    const int bn = SWAP ? BN : p.job[0].cut.bn;  // columns of a tile
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023) & ~1023u;
    const uint32_t staging = base + S * kStage;
    const uint32_t bars = staging + kEpilogueWarps * kStaging;
    auto full = [&](int i) { return bars + 8 * i; };
    auto empty = [&](int i) { return bars + 8 * (S + i); };
    auto tfull = [&](int i) { return bars + 8 * (2 * S + i); };
    auto tempty = [&](int i) { return bars + 8 * (2 * S + 2 + i); };
    const uint32_t tmem_at = bars + 8 * (2 * S + 4);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = CG == 1 ? 0 : cluster_rank();  // in the pair
    const int group = blockIdx.x / CG, groups = gridDim.x / CG;
    const int items = p.job[0].cut.m_tiles * p.job[0].cut.n_tiles * p.job[0].cut.splits;
    [[maybe_unused]] const int second_items =
        JOINT ? p.job[1].cut.m_tiles * p.job[1].cut.n_tiles * p.job[1].cut.splits : 0;
    const int first_items = items > group ? (items - group + groups - 1) / groups : 0;
    // this group's n-th tile: which of which job
    auto take = [&](int n, int *job, int *item) {
        *job = 0;
        *item = group + n * groups;
        if (n < first_items) return true;
        if constexpr (!JOINT) return false;
        *job = 1;
        n -= first_items;
        const int others = groups - p.more;
        if (group >= p.more && n < p.ahead) {
            *item = n * others + group - p.more;
        } else {
            if (group >= p.more) n -= p.ahead;
            *item = p.ahead * others + n * groups + group;
        }
        return *item < second_items;
    };
    int job, item;

    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&p.job[0].a);
        tma_prefetch_map(&p.job[0].b);
        for (int i = 0; i < S; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull(i), 1);
            mbar_init(tempty(i), kEpilogueWarps * CG);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tmem_alloc<CG>(tmem_at, kCols);
    __syncwarp();
    tmem_fence_before();
    group_sync<CG>();
    if constexpr (CG > 1) __syncthreads();
    tmem_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(tmem_at) : "memory");
    // Barriers and tensor memory are set up beside the kernel before.  With `early`
    // that one writes neither operand, and waited itself before it let this one
    // start: loads and products begin, the epilogue waits.
    if (!p.early || warp >= 2) pdl_enter();
    if (KIND == kStats && blockIdx.x == 0 && threadIdx.x == 0) *p.done = 0;

    if (warp == 0 && lane == 0) {
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        // SWAP: a tile may have fewer than 128 rows; the others are not loaded, and
        // what their sums are is not looked at
        const int b_boxes = BMN ? (bn / CG + 63) / 64 : 0;  // of 64 columns
        for (int n = 0; ok && take(n, &job, &item); ++n) {
            const Job &jb = p.job[JOINT ? job : 0];
            const Tile t = tile_of(jb, item);
            const bool a_mn = JOINT ? jb.a_mn != 0 : AMN;
            const uint32_t bytes =
                KIND == kOut && !SWAP
                      ? CG * (uint32_t)((a_mn ? 2 * jb.box_k : 128) * 128 +
                                        b_boxes * jb.box_k * 128)
                      : CG * (uint32_t)(jb.cut.tile_m * 128 +
                                        (BMN ? b_boxes * 64 : bn / CG) * kBK * 2);
            const int m0 = jb.a_m + t.m * (jb.cut.tile_m * CG) + (int)rank * 128;
            const int n0 = jb.b_n + t.n * bn + (int)rank * (bn / CG);
            const int k0 = t.split * jb.cut.k_chunk;
            const int k1 = min(jb.cut.k_tiles, k0 + jb.cut.k_chunk);
            for (int kt = k0; kt < k1; ++kt) {
                ok = mbar_wait(empty(stage), phase ^ 1);
                if (!ok) break;
                const uint32_t a = base + stage * kStage, b = a + kA;
                if (rank == 0) mbar_expect(full(stage), bytes);
                const uint32_t bar = CG == 1 ? full(stage) : in_cta(full(stage), 0);
                const int ka = jb.a_k + kt * kBK, kb = jb.b_k + kt * kBK;
                if (a_mn) {
                    for (int i = 0; i < 2; ++i)
                        tma_load<CG>(a + i * (64 * kBK * 2), &jb.a, bar, m0 + 64 * i, ka);
                } else {
                    tma_load<CG>(a, &jb.a, bar, ka, m0);
                }
                if constexpr (BMN) {
                    for (int i = 0; i < b_boxes; ++i)
                        tma_load<CG>(b + i * (64 * kBK * 2), &jb.b, bar, n0 + 64 * i, kb);
                } else {
                    tma_load<CG>(b, &jb.b, bar, kb, n0);
                }
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        // until the last products have read their stages: the peer's barriers and
        // memory are in use up to then
        for (int i = 0; ok && i < S; ++i) {
            ok = mbar_wait(empty(stage), phase ^ 1);
            if (++stage == S) {
                stage = 0;
                phase ^= 1;
            }
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        constexpr uint32_t kStepB = BMN ? 16 * 128 / 16 : 32 / 16;  // 16 values of K on
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int done = 0; ok && take(done, &job, &item); ++done) {
            const Job &jb = p.job[JOINT ? job : 0];
            const Tile t = tile_of(jb, item);
            const bool a_mn = JOINT ? jb.a_mn != 0 : AMN;
            const uint32_t idesc = mma_desc(128 * CG, bn, a_mn, BMN);
            const uint32_t step_a = a_mn ? 16 * 128 / 16 : 32 / 16;
            const int k0 = t.split * jb.cut.k_chunk;
            const int k1 = min(jb.cut.k_tiles, k0 + jb.cut.k_chunk);
            const int buf = done & 1;
            const uint32_t d = tmem + buf * BN;
            ok = mbar_wait(tempty(buf), ((done >> 1) & 1) ^ 1);
            tmem_fence_after();
            // one k tile; the four products stand without a branch between them
            // (with one, 8192 x 50257 x 1024 took 537 us instead of 511)
            auto product = [&](int kt, auto steps) {
                ok = mbar_wait(full(stage), phase);
                if (!ok) return;
                tmem_fence_after();
                const uint32_t a = base + stage * kStage;
                // (K-major tiles have no use for the distance of their blocks)
                const uint64_t da = operand_desc<AMN || JOINT>(a, 64 * kBK * 2);
                const uint64_t db = operand_desc<BMN>(a + kA, 64 * kBK * 2);
#pragma unroll
                for (int k = 0; k < decltype(steps)::value; ++k)
                    mma<CG>(d, da + k * step_a, db + k * kStepB, idesc, kt > k0 || k > 0);
                mma_commit<CG>(empty(stage));
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
            };
            // the depth's last tile may hold fewer than four times 16 values
            const int whole = k1 == jb.cut.k_tiles && jb.steps < 4 ? k1 - 1 : k1;
            for (int kt = k0; ok && kt < whole; ++kt) product(kt, Steps<4>{});
            if (ok && whole < k1) {
                if (jb.steps == 1) product(whole, Steps<1>{});
                if (jb.steps == 2) product(whole, Steps<2>{});
                if (jb.steps == 3) product(whole, Steps<3>{});
            }
            if (ok) mma_commit<CG>(tfull(buf));
        }
    } else if (KIND == kStats && !LIST && (warp == 2 || warp == 3)) {
        // The targets' logits, summed with rounding: the tensor cores cut off, 1e-6
        // of a sum of 1024 terms.  A likely target's loss is a small difference
        // of lse and its logit, so that the logit's error would be the loss's.
        // Eight lanes to a token.
        const int64_t tokens = p.job[0].rows;
        for (int64_t t0 = 4 * (2 * blockIdx.x + warp - 2); t0 < tokens; t0 += 8 * gridDim.x) {
            const int64_t t = t0 + lane / 8;
            int64_t w = -1;
            if (t < tokens) w = load_index(p.targets, p.target_bytes, t);
            if (w < 0 || w >= p.vocab) continue;
            const float z = target_logit<8>(p.hidden + t * p.hidden_stride,
                                            p.weight + w * p.weight_stride, p.dim, lane);
            if (lane % 8 == 0) p.z[t] = z;
        }
    } else if (KIND == kOut && !SWAP && (warp == 2 || warp == 3)) {
        // few tokens' d_hidden, beside the tiles of d_weight
        if (p.join.slab != nullptr)
            for (int64_t i = ((int64_t)blockIdx.x * 64 + threadIdx.x - 64) * 8;
                 i < p.join.rows * p.join.cols; i += (int64_t)gridDim.x * 64 * 8)
                store_sum(p.join, i, sum_splits(p.join, i, 0, 1));
    } else if (warp >= 4) {
        const int quad = warp % 4;  // its 32 lanes of tensor memory
        const int half = (warp - 4) / 4;
        constexpr int kPer = BN / 2 < 32 ? 32 : BN / 2;  // columns of a warp
        constexpr int kW = SWAP ? 32 : 64;               // ... which it takes at a time
        const int c0 = half * kPer;
        const uint32_t stage = staging + (warp - 4) * kStaging;
        // what a token asks for: its target, its factor and lse
        struct Ask {
            int64_t word;
            float2 rw;
            float target;
        };
        [[maybe_unused]] auto ask = [&](int64_t row) {
            Ask x{-1, make_float2(0.0f, 0.0f), 0.0f};
            if (row >= p.job[0].rows) return x;
            if constexpr (!LIST)
                x.word = KIND == kStats ? load_index(p.targets, p.target_bytes, row)
                                        : (int64_t)p.words[row];
            if constexpr (KIND == kDz) {
                x.rw = p.row[row];
                if constexpr (!LIST) x.target = p.target[row];
            }
            return x;
        };
        [[maybe_unused]] Ask mine[2];
        if constexpr (SWAP && KIND != kOut)  // the same tokens in every tile
            for (int i = 0; i < 2; ++i)
                if (32 * i < kPer) mine[i] = ask(c0 + 32 * i + lane);
        bool ok = true;
        for (int done = 0; take(done, &job, &item); ++done) {
            const Job &jb = p.job[JOINT ? job : 0];
            const Tile t = tile_of(jb, item);
            const int buf = done & 1;
            // this warp's first row and column; with SWAP its columns are those of the
            // quarter, and its rows go on with each 32
            const int64_t row0 = SWAP ? (int64_t)t.n * BN + c0
                                      : (int64_t)t.m * (128 * CG) + rank * 128 + quad * 32;
            const int col0 = SWAP ? t.m * jb.cut.tile_m + quad * 32 : t.n * bn + c0;
            const int cols =  // valid ones among them
                (int)min((int64_t)(SWAP ? min(32, jb.cut.tile_m - quad * 32) : min(kPer, bn - c0)),
                         jb.cols - col0);
            const int per = SWAP ? kPer : max(0, min(kPer, (cols + 31) / 32 * 32));
            int64_t row = row0 + lane;
            bool live = row < jb.rows;
            [[maybe_unused]] Walk<LIST, LIST && KIND == kDz> walk;
            [[maybe_unused]] float2 rw;
            [[maybe_unused]] float target;
            [[maybe_unused]] auto begin_row = [&](const Ask &x) {
                walk = {};
                rw = x.rw;
                target = x.target;
                if (!live || cols <= 0) return;
                if constexpr (LIST) {
                    const uint16_t *f = p.first + row * p.first_pitch;
                    walk.index = p.index + row * p.k;
                    walk.q = p.q + row * p.k;
                    walk.word0 = p.word0 + col0;
                    walk.at = f[walk.word0 / kGrain];
                    walk.end = f[(walk.word0 + cols - 1) / kGrain + 1];
#pragma unroll
                    for (int i = 0; i < walk.kHeld; ++i) walk.load(i);
                    while (walk.next() < 0) walk.advance();  // the grain began before
                } else {
                    const int64_t c = x.word - p.word0 - col0;
                    if (x.word >= 0 && c >= 0 && c < cols) walk.column[0] = (int)c;
                }
            };
            if constexpr (KIND != kOut) begin_row(SWAP ? mine[0] : ask(row));
            if (ok) ok = mbar_wait(tfull(buf), (done >> 1) & 1);
            tmem_fence_after();
            const uint32_t d = tmem + ((uint32_t)(quad * 32) << 16) + buf * BN + c0;
            [[maybe_unused]] float top = -INFINITY, sum = 0.0f;
            auto release = [&] {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(CG == 1 ? tempty(buf) : in_cta(tempty(buf), 0));
            };
            if (c0 >= BN || per == 0) release();
#pragma unroll 1
            for (int i = 0; i < per && c0 + i < BN; i += kW) {
                if (SWAP && i > 0) {
                    row = row0 + i + lane;
                    live = row < jb.rows;
                    if constexpr (KIND != kOut) begin_row(mine[1]);
                }
                float v[kW / 32][32];
                {
                    uint32_t bits[kW / 32][32];
#pragma unroll
                    for (int h = 0; h < kW / 32; ++h) tmem_load32(d + i + 32 * h, bits[h]);
                    tmem_wait_load();
                    if (i + kW >= per) release();
#pragma unroll
                    for (int h = 0; h < kW / 32; ++h)
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[h][j] = __uint_as_float(bits[h][j]);
                }
                if (!ok) {
#pragma unroll
                    for (int h = 0; h < kW / 32; ++h)
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[h][j] = NAN;
                }
                if constexpr (SWAP) {
                    // [token][word], each row turned by its number: no two lanes meet
                    // in a bank
                    await_box(lane);
                    auto at = [&](int r, int c) { return stage + (r * 32 + ((c + r) & 31)) * 4; };
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(at(j, lane)), "f"(v[0][j])
                                     : "memory");
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[0][j]) : "r"(at(lane, j))
                                     : "memory");
                    __syncwarp();
                    top = -INFINITY;
                    sum = 0.0f;
                }
                const int c = SWAP ? 0 : i;  // column of v[0][0] from col0 on
                if constexpr (KIND == kStats) {
#pragma unroll
                    for (int h = 0; h < kW / 32; ++h)
                        while (walk.next() < min(c + 32 * h + 32, cols)) {
                            const int hit = walk.next() - c - 32 * h;
                            if constexpr (LIST) {
                                p.z[row * p.k + walk.at] = pick(v[h], (uint32_t)hit);
                            } else {  // the target's share of the sum is added exactly
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    if (j == hit) v[h][j] = -INFINITY;
                            }
                            walk.advance();
                        }
                    if (c + kW > cols) {
#pragma unroll
                        for (int h = 0; h < kW / 32; ++h)
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                v[h][j] = c + 32 * h + j < cols ? v[h][j] : -INFINITY;
                    }
                    // four chains of each; exp(z / temperature) = 2^(beta z)
                    float m[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) m[j] = fmaxf(v[0][2 * j], v[0][2 * j + 1]);
#pragma unroll
                    for (int j = 8; j < kW; j += 2)
                        m[j / 2 % 4] = max3(m[j / 2 % 4], v[j / 32][j % 32], v[j / 32][j % 32 + 1]);
                    const float new_top =
                        fmaxf(top, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * p.beta);
                    const float shift = new_top == -INFINITY ? 0.0f : -new_top;
                    const float2 beta2 = make_float2(p.beta, p.beta);
                    const float2 shift2 = make_float2(shift, shift);
                    float2 s[4];
#pragma unroll
                    for (int j = 0; j < kW; j += 2) {
                        float2 e = fma2(make_float2(v[j / 32][j % 32], v[j / 32][j % 32 + 1]),
                                        beta2, shift2);
                        e.x = exp2_fast(e.x);
                        e.y = exp2_fast(e.y);
                        s[j / 2 % 4] = j < 8 ? e : add2(s[j / 2 % 4], e);
                    }
                    const float2 s2 = add2(add2(s[0], s[1]), add2(s[2], s[3]));
                    sum = __fmaf_rn(sum, exp2_fast(top + shift), s2.x + s2.y);
                    top = new_top;
                    if constexpr (SWAP)
                        if (live) p.part[(t.m * 4 + quad) * jb.rows + row] = make_float2(top, sum);
                } else if constexpr (KIND == kDz) {
                    const bool none = rw.x == 0.0f;  // also where the logits are not finite
                    const float2 beta2 = make_float2(p.beta, p.beta);
                    const float2 lse2 = make_float2(-rw.y, -rw.y);
                    const float2 factor2 = make_float2(rw.x, rw.x);
#pragma unroll
                    for (int h = 0; h < kW / 32; ++h)
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float2 e = fma2(make_float2(v[h][j], v[h][j + 1]), beta2, lse2);
                            e.x = exp2_fast(e.x);
                            e.y = exp2_fast(e.y);
                            e = mul2(e, factor2);
                            v[h][j] = e.x;
                            v[h][j + 1] = e.y;
                        }
                    // rounded once to bf16, the type of the products' operands
                    uint32_t w[kW / 2];
#pragma unroll
                    for (int j = 0; j < kW / 2; ++j)
                        w[j] = none ? 0u
                                    : pack_bf16x2(v[j / 16][2 * j % 32], v[j / 16][2 * j % 32 + 1]);
                    // the few words that the token asks for, in place of what was
                    // written for them
                    auto patch = [&](uint16_t *at, int swizzle) {
#pragma unroll
                        for (int h = 0; h < kW / 32; ++h)
                            while (walk.next() < min(c + 32 * h + 32, cols)) {
                                const int hit = walk.next();
                                float x = target;
                                if constexpr (LIST) {
                                    x = pick(v[h], (uint32_t)(hit - c - 32 * h));
                                    do {  // all shares of a word
                                        x -= rw.x * walk.share[0];
                                        walk.advance();
                                    } while (walk.next() == hit);
                                } else {
                                    walk.advance();
                                }
                                const int col = hit - c;
                                at[((col / 8 ^ swizzle) << 3) + col % 8] =
                                    none ? (uint16_t)0 : f32_to_bf16(x);
                            }
                    };
                    if constexpr (SWAP) {
                        uint16_t *o = p.dz + row * p.dz_pitch + col0;
                        if (live) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)  // a pitch of 8s: room beyond the last word
                                if (8 * j < cols)
                                    *reinterpret_cast<uint4 *>(o + 8 * j) = make_uint4(
                                        w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                            patch(o, 0);
                        }
                    } else {
                        const bool part = i + 32 == bn - c0 && col0 + i + 32 < jb.cols;
                        uint16_t *o = p.dz + row * p.dz_pitch + col0 + i;
                        put64(stage, lane, w, part, live, o);
                        if (part)
                            patch(o, 0);
                        else
                            patch(reinterpret_cast<uint16_t *>(raw + (stage - smem_u32(raw)) +
                                                               lane * 128),
                                  lane & 7);
                        if (!part) store_box(jb, stage, lane, col0 + i, row0, 0);
                    }
                } else if (SWAP || jb.out_f32) {
#pragma unroll
                    for (int h = 0; h < kW / 32; ++h) {
                        if (h > 0 && i + 32 >= per) break;
                        if constexpr (!SWAP) await_box(lane);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            st_shared(stage + lane * 128 + ((j ^ (lane & 7)) << 4),
                                      __float_as_uint(v[h][4 * j]),
                                      __float_as_uint(v[h][4 * j + 1]),
                                      __float_as_uint(v[h][4 * j + 2]),
                                      __float_as_uint(v[h][4 * j + 3]));
                        store_box(jb, stage, lane, col0 + c + 32 * h, SWAP ? row0 + i : row0,
                                  t.split);
                    }
                } else if constexpr (!SWAP) {
                    uint32_t w[kW / 2];
#pragma unroll
                    for (int j = 0; j < kW / 2; ++j)
                        w[j] = pack_bf16x2(v[j / 16][2 * j % 32], v[j / 16][2 * j % 32 + 1]);
                    const bool part = i + 32 == bn - c0 && col0 + i + 32 < jb.cols;
                    put64(stage, lane, w, part, live, jb.out_at + row * jb.out_pitch + col0 + i);
                    if (!part) store_box(jb, stage, lane, col0 + i, row0, 0);
                }
            }
            if constexpr (KIND == kStats && !SWAP)
                if (live) p.part[(t.n * 2 + half) * jb.rows + row] = make_float2(top, sum);
        }
        if (lane == 0) tma_wait_all();
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    group_sync<CG>();
    tmem_fence_after();
    if (warp == 2) tmem_free<CG>(tmem, kCols);
}

// --------------------------------------------------------------------------
// the small kernels around it
// --------------------------------------------------------------------------

// Everything the forward's join and the gradient's factors need of a token.
struct RowArgs {
    int64_t tokens, vocab, dim;
    int32_t k;             // 0: cross entropy
    int32_t parts;         // maxima and sums of a token
    int32_t index_bytes, teacher_bytes;
    const void *index;
    const void *teacher;
    const float *weights;
    float temperature;
    int8_t *state;
    int32_t *list;
    float *q;
    uint16_t *first;
    int32_t first_pitch;
};

__device__ __forceinline__ Row state_of(const RowArgs &a, int64_t t, int64_t *word) {
    if (a.k > 0) return (Row)a.state[t];
    *word = load_index(a.index, a.index_bytes, t);
    return *word < 0 ? kLeftOut : *word < a.vocab ? kCounts : kBad;
}

constexpr int kSortThreads = 128;

// The larger one; a NaN stays.
__device__ __forceinline__ float larger(float x, float y) {
    return isnan(x) ? x : isnan(y) || y > x ? y : x;
}

// A token's list by ascending word, with q = softmax(teacher / temperature), and
// where the entries of every kGrain words begin.  Entries of a negative word
// or a logit of -Inf are left out (at the end, q = 0); a word beyond the
// vocabulary spoils the row.  Equal words keep their order.
// RANK, for lists of up to 64: an entry's place is the number of entries before
// it, counted four words a load (a forward call with 777 lists of 19: 25.7 us,
// 26.5 by a sort).  The counting grows as the square: longer lists take a
// bitonic sort (501 lists of 200: 10.5 us, 13.5 by counting).
// N threads to a token: a warp, which needs no barrier of the CTA, for many short
// lists; else 128 (92 lists of 48, with the beginnings of 643 grains each, take a
// warp 11 us, 128 threads 7).
template <int N, bool RANK>
__global__ void __launch_bounds__(kSortThreads) k_head_lists(const RowArgs a, int room) {
    extern __shared__ uint64_t keys[];
    __shared__ float red[2][kSortThreads / 32];
    pdl_enter();
    const int tid = threadIdx.x % N;
    const int64_t t = (int64_t)blockIdx.x * (kSortThreads / N) + threadIdx.x / N;
    // (word, place); behind them, in the order given, the logits and by rank the words
    uint64_t *key = keys + threadIdx.x / N * (RANK ? 2 * room : room + room / 2);
    float *logits = reinterpret_cast<float *>(key + room);
    uint32_t *given = reinterpret_cast<uint32_t *>(logits + room);
    if (t >= a.tokens) return;  // all threads of the token
    auto sync = [] {
        if constexpr (N == 32) __syncwarp(); else __syncthreads();
    };
    auto logit = [&](int i) {
        return a.teacher_bytes == 2
                   ? bf16_to_f32(static_cast<const uint16_t *>(a.teacher)[t * a.k + i])
                   : static_cast<const float *>(a.teacher)[t * a.k + i];
    };
    bool bad = false;
    float top = -INFINITY;
    for (int i = tid; i < room; i += N) {
        uint32_t word = 0x7fffffffu;
        if (i < a.k) {
            const int64_t w = load_index(a.index, a.index_bytes, t * a.k + i);
            const float x = logit(i);
            logits[i] = x;
            if (w >= a.vocab) {
                bad = true;
            } else if (w >= 0 && x != -INFINITY) {
                word = (uint32_t)w;
                top = larger(top, x);
            }
        }
        if constexpr (RANK) given[i] = word;
        else key[i] = (uint64_t)word << 32 | (uint32_t)i;
    }
    for (int o = 16; o > 0; o /= 2) top = larger(top, __shfl_xor_sync(~0u, top, o));
    if constexpr (N == 32) {
        bad = __any_sync(~0u, bad);
    } else {
        if (tid % 32 == 0) red[0][tid / 32] = top;
        bad = __syncthreads_or(bad);
        for (int i = 0; i < N / 32; ++i) top = larger(top, red[0][i]);
    }
    if constexpr (RANK) {
        sync();
        for (int i = tid; i < room; i += N) {
            const uint32_t mine = given[i];
            int before = 0;
            for (int j = 0; j < room; j += 4) {  // room is a multiple of 4
                const uint4 w = *reinterpret_cast<const uint4 *>(given + j);
                before += w.x < mine || (w.x == mine && j < i);
                before += w.y < mine || (w.y == mine && j + 1 < i);
                before += w.z < mine || (w.z == mine && j + 2 < i);
                before += w.w < mine || (w.w == mine && j + 3 < i);
            }
            key[before] = (uint64_t)mine << 32 | (uint32_t)i;
        }
    } else {
        for (int size = 2; size <= room; size *= 2) {
            for (int stride = size / 2; stride > 0; stride /= 2) {
                sync();
                for (int i = tid; i < room / 2; i += N) {
                    const int lo = 2 * i - (i & (stride - 1)), hi = lo + stride;
                    const uint64_t x = key[lo], y = key[hi];
                    if ((x > y) == ((lo & size) == 0)) {
                        key[lo] = y;
                        key[hi] = x;
                    }
                }
            }
        }
    }
    sync();
    auto begin = [&](uint32_t word) {  // the first entry of this word or a later one
        int lo = 0, hi = a.k;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if ((uint32_t)(key[mid] >> 32) < word) lo = mid + 1; else hi = mid;
        }
        return lo;
    };
    const int count = begin(0x7fffffffu);
    const float inv = __fdiv_rn(1.0f, a.temperature);
    float sum = 0.0f;
    for (int i = tid; i < count; i += N)
        sum += exp2f((logits[(uint32_t)key[i]] - top) * inv * kLog2e);
    for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(~0u, sum, o);
    if constexpr (N > 32) {
        if (tid % 32 == 0) red[1][tid / 32] = sum;
        __syncthreads();
        sum = 0.0f;
        for (int i = 0; i < N / 32; ++i) sum += red[1][i];
    }
    const float norm = __fdiv_rn(1.0f, sum);
    for (int i = tid; i < a.k; i += N) {
        a.list[t * a.k + i] = (int32_t)(key[i] >> 32);
        a.q[t * a.k + i] =
            i < count ? exp2f((logits[(uint32_t)key[i]] - top) * inv * kLog2e) * norm : 0.0f;
    }
    for (int n = tid; n < a.first_pitch; n += N)
        a.first[t * a.first_pitch + n] =
            (uint16_t)min(count, begin((uint32_t)min((int64_t)n * kGrain, (int64_t)0x7fffffff)));
    if (tid == 0) a.state[t] = bad ? kBad : count > 0 ? kCounts : kLeftOut;
}

struct JoinArgs {
    RowArgs row;
    const float2 *part;
    const float *z;
    float4 *sums;          // of each block
    unsigned *done;        // 0 at the start
    float *loss, *lse, *total;
};

constexpr int kJoinThreads = 256;

__device__ __forceinline__ float2 join2(float2 x, float2 y) {
    const float m = fmaxf(x.x, y.x);
    const float s = m == -INFINITY ? 0.0f : m;
    return make_float2(m, __fmaf_rn(x.y, exp2_fast(x.x - s), y.y * exp2_fast(y.x - s)));
}

// A sum as a pair of binary32 (Knuth's two-sum): {sum, what its roundings lost}.
// Binary64 additions are too few a clock here: with them the join of 8192
// tokens took 19 us.
__device__ __forceinline__ float2 pair_add(float2 x, float2 y) {
    const float s = __fadd_rn(x.x, y.x), b = __fsub_rn(s, x.x);
    const float e = __fadd_rn(__fsub_rn(x.x, __fsub_rn(s, b)), __fsub_rn(y.x, b));
    // beyond binary32, or not a number, the sum has no remainder
    return make_float2(s, isfinite(s) ? __fadd_rn(e, __fadd_rn(x.y, y.y)) : 0.0f);
}

// Two sums over groups of 2 FROM lanes, in a fixed order.
template <int FROM>
__device__ __forceinline__ float4 pairs_over_lanes(float4 v) {
#pragma unroll
    for (int o = FROM; o > 0; o /= 2) {
        const float2 x = pair_add(make_float2(v.x, v.y),
                                  make_float2(__shfl_xor_sync(~0u, v.x, o),
                                              __shfl_xor_sync(~0u, v.y, o)));
        const float2 y = pair_add(make_float2(v.z, v.w),
                                  make_float2(__shfl_xor_sync(~0u, v.z, o),
                                              __shfl_xor_sync(~0u, v.w, o)));
        v = make_float4(x.x, x.y, y.x, y.y);
    }
    return v;
}

// Joins the tiles' maxima and sums, TOK tokens to a block, and finishes each
// token's loss; the last block adds up the blocks' sums in their order.
// Bound by latency: with 8192 tokens it reads 26 MB (10 us), eight loads of a thread in
// flight.  Few tokens take a block each.
template <int TOK>
__global__ void __launch_bounds__(kJoinThreads) k_head_join(const JoinArgs a) {
    constexpr int kSlices = kJoinThreads / TOK;
    constexpr int kWarps = kJoinThreads / 32;
    __shared__ float2 joined[kWarps][TOK];
    __shared__ float lists[kWarps][TOK];
    __shared__ bool beyond[kWarps][TOK];
    __shared__ float4 warps[kWarps];
    __shared__ bool last;
    pdl_enter();
    const int tok = threadIdx.x % TOK, slice = threadIdx.x / TOK, warp = threadIdx.x / 32;
    const int64_t t = (int64_t)blockIdx.x * TOK + tok;
    const bool live = t < a.row.tokens;
    // what the loss needs beside the sums, asked for before them
    int64_t word = 0;
    Row state = kLeftOut;
    float weight = 1.0f, z = 0.0f;
    if (live) {
        state = state_of(a.row, t, &word);
        if (a.row.weights) weight = a.row.weights[t];
        if (a.row.k == 0) z = a.z[t];
    }
    float2 acc = make_float2(-INFINITY, 0.0f);
    if (live) {
        const float2 *part = a.part + t;
        for (int n = slice; n < a.row.parts; n += 8 * kSlices) {
            float2 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)  // none is left to a branch: all are on their way
                x[i] = part[min(n + i * kSlices, a.row.parts - 1) * a.row.tokens];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (n + i * kSlices >= a.row.parts) x[i] = make_float2(-INFINITY, 0.0f);
            float m = acc.x;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = fmaxf(m, x[i].x);
            const float shift = m == -INFINITY ? 0.0f : m;
            float sum = acc.y * exp2_fast(acc.x - shift);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum = __fmaf_rn(x[i].y, exp2_fast(x[i].x - shift), sum);
            acc = make_float2(m, sum);
        }
    }
#pragma unroll
    for (int o = 16; o >= TOK; o /= 2)
        acc = join2(acc, make_float2(__shfl_xor_sync(~0u, acc.x, o),
                                     __shfl_xor_sync(~0u, acc.y, o)));
    if (threadIdx.x % 32 < TOK) joined[warp][tok] = acc;
    __syncthreads();
    if (a.row.k > 0 || warp == 0) {
        acc = joined[0][tok];
        for (int w = 1; w < kWarps; ++w) acc = join2(acc, joined[w][tok]);
    }
    // a sum that is not a number stays one through the logarithms
    float lse = (acc.x + log2f(acc.y)) * kLn2;
    float loss1 = 0.0f;
    if (a.row.k == 0 && state == kCounts) {
        // the sums are without the target's term: loss = log(1 + the others / its)
        const float more = __fmaf_rn(-z, kLog2e, acc.x);
        if (!isfinite(z)) {  // of which the others' sums know nothing
            lse = loss1 = NAN;
        } else if (acc.y == 0.0f) {  // a vocabulary of one, or all others below binary32
            lse = z;
        } else if (more < 64.0f) {
            loss1 = log1pf(acc.y * exp2f(more));
            lse = z + loss1;
        } else {  // its term is below the sum's last bit
            loss1 = lse - z;
        }
    }
    if (a.row.k > 0) {
        float part = 0.0f;
        bool wild = false;  // a word with a share whose logit is not finite
        const float inv = __fdiv_rn(1.0f, a.row.temperature);
        if (state == kCounts) {
            for (int i = slice; i < a.row.k; i += 4 * kSlices) {
                float q[4], x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int at = i + j * kSlices;
                    q[j] = at < a.row.k ? a.row.q[t * a.row.k + at] : 0.0f;
                    x[j] = at < a.row.k ? a.z[t * a.row.k + at] : 0.0f;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    // 0 log 0 = 0: an entry left out, or one whose q is below binary32
                    if (q[j] != 0.0f) {
                        part += q[j] * (logf(q[j]) - x[j] * inv + lse);
                        wild |= !isfinite(x[j]);
                    }
            }
        }
#pragma unroll
        for (int o = 16; o >= TOK; o /= 2) {
            part += __shfl_xor_sync(~0u, part, o);
            wild |= __shfl_xor_sync(~0u, (int)wild, o) != 0;
        }
        if (threadIdx.x % 32 < TOK) {
            lists[warp][tok] = part;
            beyond[warp][tok] = wild;
        }
        __syncthreads();
    }
    if (warp == 0) {
        float4 mine = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (slice == 0 && live) {
            float loss = 0.0f;
            if (state == kBad) {
                loss = NAN;
            } else if (state == kCounts && a.row.k > 0) {
                for (int w = 0; w < kWarps; ++w) {
                    loss += lists[w][tok];
                    if (beyond[w][tok]) lse = NAN;
                }
                loss = isnan(lse) ? NAN : loss * (a.row.temperature * a.row.temperature);
            } else if (state == kCounts) {
                loss = loss1;
            }
            a.loss[t] = loss;
            a.lse[t] = state == kLeftOut ? 0.0f : lse;
            if (state != kLeftOut && weight != 0.0f) {
                const float x = weight * loss;
                mine = make_float4(x, isfinite(x) ? __fmaf_rn(weight, loss, -x) : 0.0f, weight,
                                   0.0f);
            }
        }
        mine = pairs_over_lanes<TOK / 2>(mine);
        if (threadIdx.x == 0) {
            if (gridDim.x == 1) {
                a.total[0] = mine.x + mine.y;
                a.total[1] = mine.z + mine.w;
            } else {
                a.sums[blockIdx.x] = mine;
                __threadfence();
                last = atomicAdd(a.done, 1u) == gridDim.x - 1;
                __threadfence();
            }
        }
    }
    if (gridDim.x == 1) return;
    __syncthreads();
    if (!last) return;
    float2 x = make_float2(0.0f, 0.0f), y = x;
    for (unsigned i = threadIdx.x; i < gridDim.x; i += kJoinThreads) {
        const float4 v = __ldcg(a.sums + i);  // from L2, where the other blocks left them
        x = pair_add(x, make_float2(v.x, v.y));
        y = pair_add(y, make_float2(v.z, v.w));
    }
    const float4 v = pairs_over_lanes<16>(make_float4(x.x, x.y, y.x, y.y));
    if (threadIdx.x % 32 == 0) warps[warp] = v;
    __syncthreads();
    if (threadIdx.x != 0) return;
    x = y = make_float2(0.0f, 0.0f);
    for (int w = 0; w < kWarps; ++w) {
        x = pair_add(x, make_float2(warps[w].x, warps[w].y));
        y = pair_add(y, make_float2(warps[w].z, warps[w].w));
    }
    a.total[0] = x.x + x.y;
    a.total[1] = y.x + y.y;
}

struct FactorArgs {
    RowArgs row;
    const float *lse;
    const float *total;    // or null
    float scale;
    float2 *factor;
    int32_t *words;
    float *target;
    const uint16_t *hidden;
    int64_t stride;
    const uint16_t *weight;
    int64_t weight_stride;
    uint16_t *copy;        // null: not needed
    int64_t copy_stride;
};

// Each token's factor a = scale w / total[1] (times the temperature), its lse in
// powers of two and, with a target, dz there: a (exp(z - lse) - 1) of the very
// logit that lse was made with, which leaves lse's own rounding as the error of a
// likely target's small dz.  And the hidden states
// with zeros in the rows left out: what stands there may be anything, and 0 *
// NaN would reach d_weight.  The copy costs 4 bytes a value, the targets' rows
// of the weight 2 more: 10 us of the 2.1 ms at 8192 x 1024.
// A warp to a token.
__global__ void __launch_bounds__(128) k_head_factors(const FactorArgs a) {
    pdl_enter();
    const int lane = threadIdx.x % 32;
    const int64_t t = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    if (t >= a.row.tokens) return;
    int64_t word = -1;
    const Row state = state_of(a.row, t, &word);
    float f = a.scale;
    if (a.total) f = a.total[1] == 0.0f ? 0.0f : __fdiv_rn(f, a.total[1]);
    float w = state == kLeftOut ? 0.0f : 1.0f;
    if (a.row.weights && state != kLeftOut) w = a.row.weights[t];
    f = __fmul_rn(f, w);
    if (a.row.k > 0) f = __fmul_rn(f, a.row.temperature);
    if (state == kBad) f = NAN;
    if (w == 0.0f) f = 0.0f;  // out of the gradients, whatever else there is
    const float lse = a.lse[t];
    const uint16_t *row = a.hidden + t * a.stride;
    float z = lse;
    if (a.row.k == 0 && state == kCounts)
        z = target_logit<32>(row, a.weight + word * a.weight_stride, a.row.dim, lane);
    if (lane == 0) {
        a.factor[t] = make_float2(f, __fmul_rn(lse, kLog2e));
        if (a.row.k == 0) {
            a.words[t] = state == kCounts ? (int32_t)word : -1;
            a.target[t] = f * expm1f(z - lse);
        }
    }
    if (a.copy == nullptr) return;
    const bool keep = f != 0.0f;
#pragma unroll 4
    for (int64_t i = lane * 8; i < a.row.dim; i += 32 * 8) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (keep) x = ld8b(row + i);
        *reinterpret_cast<uint4 *>(a.copy + t * a.copy_stride + i) = x;
    }
}

// The splits' sums, in a fixed order.  Eight values to a thread; SLICES threads
// share the splits of small results, whose time is the loads' latency (8 x 336 by
// 50 splits: 9 us with one slice, 4.5 with eight).
template <int SLICES>
__global__ void __launch_bounds__(256) k_head_slabs(const Slabs p) {
    constexpr int kWide = 256 / SLICES;
    __shared__ float4 sums[SLICES > 1 ? 256 : 1][2];
    pdl_enter();
    const int at = threadIdx.x % kWide, slice = threadIdx.x / kWide;
    const int64_t i = ((int64_t)blockIdx.x * kWide + at) * 8;
    const bool live = i < p.rows * p.cols;
    Sum8 x;
    if (live) x = sum_splits(p, i, slice, SLICES);
    if constexpr (SLICES > 1) {
        sums[threadIdx.x][0] = x.a;
        sums[threadIdx.x][1] = x.b;
        __syncthreads();
        if (slice > 0) return;
        for (int s = 1; s < SLICES; ++s) x.add(sums[s * kWide + at][0], sums[s * kWide + at][1]);
    }
    if (live) store_sum(p, i, x);
}

// --------------------------------------------------------------------------
// host side: cutting, tensor maps, launches
// --------------------------------------------------------------------------

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A kernel that begins with pdl_enter.
template <typename... KArgs, typename... Args>
void launch_small(void (*kernel)(KArgs...), int64_t grid, int block, size_t smem, cudaStream_t s,
                  Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    (void)cudaLaunchKernelEx(&cfg, kernel, args...);  // errors: cudaGetLastError
}

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
    static const EncodeTiled f = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                             cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return (EncodeTiled)fn;
    }();
    return f;
}

// Rows of `inner` bf16 values, `pitch` apart, in boxes of 64 values by box_rows;
// zeros outside.
bool make_map(CUtensorMap *m, const void *p, int64_t inner, int64_t outer, int64_t pitch,
              int box_rows) {
    const EncodeTiled encode = encoder();
    if (encode == nullptr) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
    const cuuint64_t strides[1] = {(cuuint64_t)pitch * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    const cuuint32_t ones[2] = {1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides, box,
                  ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A result in boxes of 32 rows of 128 bytes: bf16 [rows][pitch], or binary32
// [splits][rows][pitch].
bool make_out(CUtensorMap *m, void *p, bool f32, int64_t cols, int64_t rows, int64_t pitch,
              int64_t splits) {
    const EncodeTiled encode = encoder();
    if (encode == nullptr) return false;
    const int size = f32 ? 4 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)splits};
    const cuuint64_t strides[2] = {(cuuint64_t)(pitch * size),
                                   (cuuint64_t)((splits > 1 ? rows : 1) * pitch * size)};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / size), 32, 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    return encode(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p,
                  dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs or pairs that the GPU holds at a time.
int64_t room(int cg) { return kHeadSMs / cg; }

int64_t tiles(const Cut &c) { return (int64_t)c.m_tiles * c.n_tiles * c.splits; }

template <int CG, int BN, bool SWAP, bool AMN, bool BMN, Kind KIND, bool LIST, bool JOINT = false>
cudaError_t launch_mma(const MmaArgs &p, cudaStream_t s) {
    auto *kernel = k_head_mma<CG, BN, SWAP, AMN, BMN, KIND, LIST, JOINT>;
    // once for each device (1 us of host time)
    static std::atomic<uint64_t> allowed{0};
    int device;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (device & 63);
    if (device > 63 || !(allowed.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    const int64_t items = tiles(p.job[0].cut) + (JOINT ? tiles(p.job[1].cut) : 0);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(CG * std::min<int64_t>(items, room(CG))));
    cfg.blockDim = dim3(kMmaThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e == cudaErrorInvalidValue) {  // the device was reset since
        (void)cudaGetLastError();
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        (void)cudaLaunchKernelEx(&cfg, kernel, p);
    }
    return cudaGetLastError();
}

// tokens x words
template <Kind KIND, bool LIST>
cudaError_t launch_logits(const MmaArgs &p, cudaStream_t s) {
    const Cut &c = p.job[0].cut;
    if (!c.swap) return launch_mma<2, 256, false, false, false, KIND, LIST>(p, s);
    if (c.bn == 32) return launch_mma<1, 32, true, false, false, KIND, LIST>(p, s);
    return launch_mma<1, 128, true, false, false, KIND, LIST>(p, s);
}

// One product of dz; or both, in any order.
template <bool AMN>
cudaError_t launch_out(const MmaArgs &p, cudaStream_t s) {
    return p.job[0].cut.bn > 128 ? launch_mma<2, 256, false, AMN, true, kOut, false>(p, s)
                                 : launch_mma<2, 128, false, AMN, true, kOut, false>(p, s);
}

cudaError_t launch_both(MmaArgs &p, cudaStream_t s) {
    // a tile's cost: its depth, and two k tiles' time between tiles
    auto cost = [](const Job &jb) { return (int64_t)jb.cut.k_chunk + 2; };
    if (cost(p.job[0]) < cost(p.job[1])) std::swap(p.job[0], p.job[1]);
    const int64_t first = tiles(p.job[0].cut), second = tiles(p.job[1].cut);
    const int64_t groups = std::min(room(2), first + second);
    const int64_t more = first % groups, each = first / groups;
    const int64_t c0 = cost(p.job[0]), c1 = cost(p.job[1]);
    // tiles of the second that a group ends in this time after `firsts` of the first
    auto fits = [&](int64_t time, int64_t firsts) {
        return std::max<int64_t>(0, (time - firsts * c0) / c1);
    };
    int64_t lo = 0, hi = (each + 1) * c0 + second * c1;
    while (lo < hi) {  // the least time in which all groups end all of them
        const int64_t mid = (lo + hi) / 2;
        if (more * fits(mid, each + 1) + (groups - more) * fits(mid, each) >= second)
            hi = mid;
        else
            lo = mid + 1;
    }
    p.more = (int32_t)more;
    p.ahead = more > 0 ? (int32_t)(fits(lo, each) - fits(lo, each + 1)) : 0;
    return p.job[0].cut.bn > 128
               ? launch_mma<2, 256, false, false, true, kOut, false, true>(p, s)
               : launch_mma<2, 128, false, false, true, kOut, false, true>(p, s);
}

// d_hidden of few tokens
cudaError_t launch_d_hidden_few(const MmaArgs &p, cudaStream_t s) {
    return p.job[0].cut.bn == 32 ? launch_mma<1, 32, true, true, false, kOut, false>(p, s)
                                 : launch_mma<1, 128, true, true, false, kOut, false>(p, s);
}

constexpr int64_t kFew = 128;  // tokens that SWAP takes

// The logits' tiles, for all words or a piece of them.  Few tokens: the weight's
// rows are cut so that every SM has the same number of tiles, none more than
// 128 rows (50257 rows by 128 leave the third wave of tiles 58% full, by 112
// 95%).
Cut cut_logits(int64_t tokens, int64_t words, int64_t dim) {
    Cut c{};
    c.k_tiles = c.k_chunk = (int32_t)ceil_div(dim, kBK);
    c.splits = 1;
    c.swap = tokens <= kFew;
    if (c.swap) {
        c.cg = 1;
        c.bn = tokens <= 32 ? 32 : 128;
        const int64_t waves = ceil_div(words, kHeadSMs * 128);
        c.tile_m = (int32_t)(ceil_div(ceil_div(words, kHeadSMs * waves), 8) * 8);
        c.m_tiles = (int32_t)ceil_div(words, c.tile_m);
        c.n_tiles = 1;
    } else {
        c.cg = 2;
        c.tile_m = 128;
        c.m_tiles = (int32_t)ceil_div(tokens, 256);
        // columns of a tile: what leaves the last wave of tiles fullest, a tile
        // costing as much as 24 columns beside its own
        int64_t best = 0;
        for (int bn = 256; bn >= 128; bn -= 32) {
            const int64_t tiles = c.m_tiles * ceil_div(words, bn);
            const int64_t x = ceil_div(tiles, room(2)) * (bn + 24);
            if (best == 0 || x < best) {
                best = x;
                c.bn = bn;
            }
        }
        c.n_tiles = (int32_t)ceil_div(words, c.bn);
    }
    return c;
}

// The tiles of a product of dz: [m][n] of depth k.  Where they are fewer than
// half of what the GPU holds at a time, the depth is cut until it is full, 4 k
// tiles (256 values) at least to a split.
Cut cut_out(int64_t m, int64_t n, int64_t k, bool swap, int64_t tokens) {
    Cut c{};
    c.swap = swap;
    c.cg = swap ? 1 : 2;
    // the columns in equal tiles of up to 256, in steps of 32
    c.bn = swap ? (tokens <= 32 ? 32 : 128)
                : (int32_t)(ceil_div(ceil_div(n, ceil_div(n, 256)), 32) * 32);
    c.tile_m = 128;
    c.m_tiles = (int32_t)ceil_div(m, 128 * c.cg);
    c.n_tiles = (int32_t)ceil_div(n, c.bn);
    c.k_tiles = (int32_t)ceil_div(k, kBK);
    int64_t splits = 1;
    const int64_t tiles = (int64_t)c.m_tiles * c.n_tiles, at_a_time = room(c.cg);
    if (tiles * 2 <= at_a_time)
        splits = std::max<int64_t>(1, std::min<int64_t>(at_a_time / tiles, c.k_tiles / 4));
    c.k_chunk = (int32_t)ceil_div(c.k_tiles, splits);
    c.splits = (int32_t)ceil_div(c.k_tiles, c.k_chunk);
    return c;
}

Cut cut_d_hidden(int64_t tokens, int64_t dim, int64_t words) {
    return tokens <= kFew ? cut_out(dim, tokens, words, true, tokens)
                          : cut_out(tokens, dim, words, false, tokens);
}

Cut cut_d_weight(int64_t tokens, int64_t dim, int64_t words) {
    return cut_out(words, dim, tokens, false, tokens);
}

// dz of a piece of the vocabulary: 256 MB, but 2048 words at least, so that the
// sums of d_hidden, read and written once a piece, cost less than its products.
constexpr int64_t kPieceBytes = 256ll << 20;
constexpr int64_t kPieceWords = 2048;

// Up to the end of the last tile.
int64_t first_pitch(const HeadPlan &p) { return ceil_div(p.vocab, 256) * (256 / kGrain) + 1; }

int join_tokens(int64_t tokens) { return tokens <= kFew ? 1 : 16; }

RowArgs row_args(const HeadArgs &a) {
    const HeadPlan &p = a.plan;
    RowArgs r{};
    r.tokens = p.tokens;
    r.vocab = p.vocab;
    r.dim = p.dim;
    r.k = a.teacher ? (int32_t)p.k : 0;
    r.parts = p.parts;
    r.index_bytes = a.index_bytes;
    r.teacher_bytes = a.teacher_bytes;
    r.index = a.index;
    r.teacher = a.teacher;
    r.weights = a.weights;
    r.temperature = a.temperature;
    r.state = reinterpret_cast<int8_t *>(a.ws + p.state);
    r.list = reinterpret_cast<int32_t *>(a.ws + p.index);
    r.q = reinterpret_cast<float *>(a.ws + p.q);
    r.first = reinterpret_cast<uint16_t *>(a.ws + p.first);
    r.first_pitch = (int32_t)first_pitch(p);
    return r;
}

cudaError_t launch_lists(const RowArgs &r, cudaStream_t s) {
    constexpr int kN = kSortThreads;
    const int room = (r.k + 3) / 4 * 4;
    int pow2 = 2;
    while (pow2 < r.k) pow2 *= 2;
    if (r.k <= 64 && r.tokens > 1024)
        launch_small(k_head_lists<32, true>, ceil_div(r.tokens, kN / 32), kN, kN / 32 * room * 16,
                     s, r, room);
    else if (r.k <= 64)
        launch_small(k_head_lists<kN, true>, r.tokens, kN, room * 16, s, r, room);
    else
        launch_small(k_head_lists<kN, false>, r.tokens, kN, pow2 * 12, s, r, pow2);
    return cudaGetLastError();
}

void fill_lists(MmaArgs *m, const RowArgs &r) {
    m->k = r.k;
    m->index = r.list;
    m->q = r.q;
    m->first = r.first;
    m->first_pitch = r.first_pitch;
}

cudaError_t launch_slabs(const Slabs &p, cudaStream_t s) {
    const int64_t n = p.rows * p.cols;
    if (p.splits >= 8)
        launch_small(k_head_slabs<8>, ceil_div(n, 256), 256, 0, s, p);
    else
        launch_small(k_head_slabs<1>, ceil_div(n, 2048), 256, 0, s, p);
    return cudaGetLastError();
}

int last_steps(int64_t k) { return (int)ceil_div(k - (ceil_div(k, kBK) - 1) * kBK, 16); }

// The product of the hidden states with the words from w0 on.
bool logits_job(MmaArgs *m, const HeadArgs &a, const Cut &cut, int64_t w0, int64_t words) {
    const HeadPlan &p = a.plan;
    Job &jb = m->job[0];
    jb.cut = cut;
    jb.steps = last_steps(p.dim);
    jb.rows = p.tokens;
    jb.cols = words;
    m->word0 = (int32_t)w0;
    m->beta = kLog2e / a.temperature;
    CUtensorMap *hidden = cut.swap ? &jb.b : &jb.a, *weight = cut.swap ? &jb.a : &jb.b;
    (cut.swap ? jb.a_m : jb.b_n) = (int32_t)w0;
    return make_map(hidden, a.hidden, p.dim, p.tokens, a.hidden_stride, cut.swap ? cut.bn : 128) &&
           make_map(weight, a.weight, p.dim, p.vocab, a.weight_stride,
                    cut.swap ? cut.tile_m : cut.bn / 2);
}

}  // namespace

bool head_plan(int64_t tokens, int64_t dim, int64_t vocab, int64_t k, bool grads, HeadPlan *p) {
    *p = HeadPlan{};
    p->tokens = tokens;
    p->vocab = vocab;
    p->dim = dim;
    p->k = k;
    // tiles and rows are counted in 32 bits, bytes in 64
    constexpr int64_t kMost = (1ll << 31) - 1024;
    if (tokens > kMost || vocab > kMost || dim > kHeadMaxDim) return false;
    int64_t probe;
    if (__builtin_mul_overflow(tokens, vocab, &probe) ||
        __builtin_mul_overflow(std::max(tokens, vocab), dim, &probe) || probe > (1ll << 56) ||
        ceil_div(std::max(tokens, dim), 64) * ceil_div(std::max(vocab, tokens), 64) > kMost)
        return false;
    p->logits = cut_logits(tokens, vocab, dim);
    p->parts = p->logits.swap ? p->logits.m_tiles * 4 : p->logits.n_tiles * 2;
    int64_t at = 0;
    bool fits = true;
    auto take = [&](int64_t n, int64_t size) {
        const int64_t here = at;
        int64_t bytes;
        if (__builtin_mul_overflow(n, size, &bytes) || bytes > (1ll << 60) - at)
            fits = false;
        else
            at += ceil_div(bytes, 256) * 256;
        return here;
    };
    p->part = take((int64_t)p->parts * tokens, 8);
    p->z = take(tokens * std::max<int64_t>(k, 1), 4);
    p->sums = take(ceil_div(tokens, join_tokens(tokens)), 16);
    p->done = take(1, 4);
    p->state = take(k ? tokens : 0, 1);
    p->index = take(tokens * k, 4);
    p->q = take(tokens * k, 4);
    p->first = take(k ? tokens * first_pitch(*p) : 0, 2);
    if (grads && tokens > 0) {
        const int64_t most =
            std::max<int64_t>(kPieceWords / 256, kPieceBytes / 512 / tokens) * 256;
        p->pieces = ceil_div(vocab, most);
        p->piece = ceil_div(ceil_div(vocab, p->pieces), 256) * 256;
        p->pieces = ceil_div(vocab, p->piece);
        p->rows = take(tokens, 8);
        p->words = take(tokens, 4);
        p->target = take(tokens, 4);
        p->hidden_pitch = ceil_div(dim, 64) * 64;
        p->hidden = take(tokens * p->hidden_pitch, 2);
        p->dz = take(tokens * p->piece, 2);
        const Cut h = cut_d_hidden(tokens, dim, p->piece);
        const Cut w = cut_d_weight(tokens, dim, p->piece);
        p->slab_h =
            take(h.swap || h.splits > 1 || p->pieces > 1 ? h.splits * tokens * dim : 0, 4);
        p->slab_w = take(w.splits > 1 ? w.splits * p->piece * dim : 0, 4);
    }
    p->bytes = std::max<int64_t>(at, 256);
    return fits;
}

cudaError_t launch_head_forward(const HeadArgs &a, cudaStream_t s) {
    const HeadPlan &p = a.plan;
    if (p.tokens == 0) return cudaMemsetAsync(a.total, 0, 8, s);
    const RowArgs r = row_args(a);
    cudaError_t e;
    if (r.k > 0 && (e = launch_lists(r, s)) != cudaSuccess) return e;
    MmaArgs m{};
    if (!logits_job(&m, a, p.logits, 0, p.vocab)) return cudaErrorInvalidValue;
    m.early = r.k > 0;  // after the lists' launch
    m.part = reinterpret_cast<float2 *>(a.ws + p.part);
    m.z = reinterpret_cast<float *>(a.ws + p.z);
    m.done = reinterpret_cast<unsigned *>(a.ws + p.done);
    m.targets = a.index;
    m.target_bytes = a.index_bytes;
    m.hidden = a.hidden;
    m.weight = a.weight;
    m.hidden_stride = a.hidden_stride;
    m.weight_stride = a.weight_stride;
    m.vocab = p.vocab;
    m.dim = (int32_t)p.dim;
    fill_lists(&m, r);
    e = r.k > 0 ? launch_logits<kStats, true>(m, s) : launch_logits<kStats, false>(m, s);
    if (e != cudaSuccess) return e;
    JoinArgs j{};
    j.row = r;
    j.part = m.part;
    j.z = m.z;
    j.sums = reinterpret_cast<float4 *>(a.ws + p.sums);
    j.done = m.done;
    j.loss = a.loss;
    j.lse = a.lse;
    j.total = a.total;
    if (join_tokens(p.tokens) == 1)
        launch_small(k_head_join<1>, p.tokens, kJoinThreads, 0, s, j);
    else
        launch_small(k_head_join<16>, ceil_div(p.tokens, 16), kJoinThreads, 0, s, j);
    return cudaGetLastError();
}

cudaError_t launch_head_grad(const HeadArgs &a, cudaStream_t s) {
    const HeadPlan &p = a.plan;
    if (p.tokens == 0) {
        if (a.d_weight == nullptr) return cudaSuccess;
        return cudaMemset2DAsync(a.d_weight, (size_t)a.d_weight_stride * 2, 0, (size_t)p.dim * 2,
                                 (size_t)p.vocab, s);
    }
    const RowArgs r = row_args(a);
    cudaError_t e;
    if (r.k > 0 && (e = launch_lists(r, s)) != cudaSuccess) return e;
    uint16_t *hidden = reinterpret_cast<uint16_t *>(a.ws + p.hidden);
    FactorArgs f{};
    f.row = r;
    f.lse = a.lse;
    f.total = a.total;
    f.scale = a.scale;
    f.factor = reinterpret_cast<float2 *>(a.ws + p.rows);
    f.words = reinterpret_cast<int32_t *>(a.ws + p.words);
    f.target = reinterpret_cast<float *>(a.ws + p.target);
    f.hidden = a.hidden;
    f.stride = a.hidden_stride;
    f.weight = a.weight;
    f.weight_stride = a.weight_stride;
    f.copy = a.d_weight ? hidden : nullptr;
    f.copy_stride = p.hidden_pitch;
    launch_small(k_head_factors, ceil_div(p.tokens, 4), 128, 0, s, f);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;

    // the copy's rows start on lines of 128 bytes, where the caller's do not
    HeadArgs from = a;
    if (a.d_weight && a.hidden_stride % 64 != 0) {
        from.hidden = hidden;
        from.hidden_stride = p.hidden_pitch;
    }
    uint16_t *dz = reinterpret_cast<uint16_t *>(a.ws + p.dz);
    for (int64_t i = 0; i < p.pieces; ++i) {
        const int64_t w0 = i * p.piece, words = std::min(p.piece, p.vocab - w0);
        const bool last = i + 1 == p.pieces;
        MmaArgs m{};
        if (!logits_job(&m, from, cut_logits(p.tokens, words, p.dim), w0, words) ||
            !make_out(&m.job[0].out, dz, false, words, p.tokens, p.piece, 1))
            return cudaErrorInvalidValue;
        m.early = i > 0 || from.hidden == a.hidden;  // else the copy is awaited
        m.row = f.factor;
        m.words = f.words;
        m.target = f.target;
        m.dz = dz;
        m.dz_pitch = p.piece;
        fill_lists(&m, r);
        e = r.k > 0 ? launch_logits<kDz, true>(m, s) : launch_logits<kDz, false>(m, s);
        if (e != cudaSuccess) return e;

        // the two products of dz: in one launch, but for few tokens' d_hidden
        MmaArgs h{}, few{};
        int jobs = 0, splits_h = 0, used_h = 0, splits_w = 0;
        uint16_t *out_w = nullptr;
        float *slab_h = reinterpret_cast<float *>(a.ws + p.slab_h);
        float *slab_w = reinterpret_cast<float *>(a.ws + p.slab_w);
        bool f32_h = false;
        Slabs join_h{};
        if (a.d_hidden) {
            const Cut cut = cut_d_hidden(p.tokens, p.dim, p.piece);
            Job &jb = cut.swap ? few.job[0] : h.job[jobs++];
            jb.cut = cut;
            splits_h = cut.splits;
            jb.cut.k_tiles = (int32_t)ceil_div(words, kBK);
            used_h = jb.cut.splits = (int32_t)ceil_div(jb.cut.k_tiles, jb.cut.k_chunk);
            jb.steps = last_steps(words);
            jb.box_k = kBK;
            jb.n_fast = 1;
            jb.rows = p.tokens;
            jb.cols = p.dim;
            jb.out_f32 = f32_h = cut.swap || splits_h > 1 || p.pieces > 1;
            jb.add = i > 0;
            jb.out_at = a.d_hidden;
            jb.out_pitch = a.d_hidden_stride;
            bool ok;
            if (cut.swap) {
                jb.a_k = (int32_t)w0;
                ok = make_map(&jb.a, a.weight, p.dim, p.vocab, a.weight_stride, kBK) &&
                     make_map(&jb.b, dz, words, p.tokens, p.piece, cut.bn);
            } else {
                jb.b_k = (int32_t)w0;
                ok = make_map(&jb.a, dz, words, p.tokens, p.piece, 128) &&
                     make_map(&jb.b, a.weight, p.dim, p.vocab, a.weight_stride, kBK);
            }
            ok = ok && (f32_h ? make_out(&jb.out, slab_h, true, p.dim, p.tokens, p.dim, splits_h)
                              : make_out(&jb.out, a.d_hidden, false, p.dim, p.tokens,
                                         a.d_hidden_stride, 1));
            if (!ok) return cudaErrorInvalidValue;
            if (last && f32_h)
                join_h = Slabs{slab_h,     p.pieces > 1 ? splits_h : used_h,
                               p.tokens,   p.dim,
                               a.d_hidden, a.d_hidden_stride};
            if (cut.swap) {
                if ((e = launch_d_hidden_few(few, s)) != cudaSuccess) return e;
                if (a.d_weight) {  // joined beside it
                    h.join = join_h;
                    join_h = Slabs{};
                }
            }
        }
        if (a.d_weight) {
            Job &jb = h.job[jobs++];
            jb.cut = cut_d_weight(p.tokens, p.dim, p.piece);
            splits_w = jb.cut.splits;
            jb.cut.m_tiles = (int32_t)ceil_div(words, 256);
            jb.steps = last_steps(p.tokens);
            jb.a_mn = 1;
            // few tokens: boxes of the rows that the products read
            jb.box_k = p.tokens < kBK ? jb.steps * 16 : kBK;
            jb.n_fast = 1;
            jb.rows = words;
            jb.cols = p.dim;
            jb.out_f32 = splits_w > 1;
            out_w = a.d_weight + w0 * a.d_weight_stride;
            jb.out_at = out_w;
            jb.out_pitch = a.d_weight_stride;
            if (!make_map(&jb.a, dz, words, p.tokens, p.piece, jb.box_k) ||
                !make_map(&jb.b, hidden, p.dim, p.tokens, p.hidden_pitch, jb.box_k) ||
                !(splits_w > 1
                      ? make_out(&jb.out, slab_w, true, p.dim, words, p.dim, splits_w)
                      : make_out(&jb.out, out_w, false, p.dim, words, a.d_weight_stride, 1)))
                return cudaErrorInvalidValue;
        }
        if (jobs > 0) {
            e = jobs == 2 ? launch_both(h, s)
                          : h.job[0].a_mn ? launch_out<true>(h, s) : launch_out<false>(h, s);
            if (e != cudaSuccess) return e;
        }
        if (join_h.slab != nullptr && (e = launch_slabs(join_h, s)) != cudaSuccess) return e;
        if (splits_w > 1 &&
            (e = launch_slabs(Slabs{slab_w, splits_w, words, p.dim, out_w, a.d_weight_stride},
                              s)) != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace z3
