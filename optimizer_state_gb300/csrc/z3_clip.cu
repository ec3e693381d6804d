// z3_clip.cu -- gradient clipping by the global norm: the norm over many
// tensors, clipping in place, the reduce-scatter that leaves its sums of
// squares, and the clipped shard Adam.
//
//   norm = sqrt(sum of g^2 over every element of every tensor)
//   coef = max_norm / norm where norm > max_norm, else 1; NaN where the norm
//          is not finite, and then nothing is written by what reads coef
//
// Sums of squares are binary32 over one batch of a thread (in the
// reduce-scatter: over one vector of each lane of a warp) and pairs of binary32
// or binary64 beyond it, added in an order that the sizes and the addresses
// modulo 16 fix (no floating-point atomics): a call gives the same bits every
// time.  Large calls
// are bound by HBM bandwidth, small ones by the latency of their one or two
// launches; nothing contracts, so no tensor cores.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <vector>

#include "z3_clip.h"
#include "z3_device.cuh"

namespace z3 {
namespace {

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// --------------------------------------------------------------------------
// sums of squares
// --------------------------------------------------------------------------

// Squares are added in binary32 within one batch of a thread: at most 24
// elements in two chains, so that at most 12 multiply-adds and one addition
// round on a square's way.  All terms are positive: with u = 2^-24 the batch
// is within 13 u of its exact sum.  The batches' sums are added in pairs of
// binary32 (48 bits): the k-th addition's error, at most u times the sum,
// joins lo with a relative error of u, so n batches per thread add n^2 u^2 / 2
// at most: 0.3 u for 32 GB (n = 3,076), 21 u for 275 GB.  The norm has half of
// the sum's error and one rounding more: 7.7 u for 32 GB, 18 u for 275 GB.  FP64 units are few: an SM takes 16 cycles for a warp's
// binary64 addition.  With one for every element the reduce-scatter of a
// d = 1024 layer with its norm took 98 us instead of 45, and with one for
// every batch and for every step of the CTAs' trees the norm of 700 tensors
// (10 MB) took 11.5 us instead of 9.8 (6.9 now).  A CTA's sum is stored as
// binary64.
//
// A batch whose sum leaves [kSafeLo, kSafeHi] may have lost squares to
// underflow or overflow; it is summed again with its elements scaled by a
// power of two, and goes to a binary64 sum of its own.  Above kSafeLo the
// squares that underflowed change the sum by under 2^-50 of it; scaled up
// from below kSafeLo, elements stay under 2^55 and the least subnormal's
// square is 2^-98; scaled down from above kSafeHi, the squares that underflow
// are those of elements under 2^5.  2^30 safe batches do not overflow.
// Infinities and NaN stay what they are.
constexpr float kSafeLo = 0x1p-90f, kSafeHi = 0x1p+90f;

__device__ __forceinline__ bool is_safe(float s) { return s >= kSafeLo && s <= kSafeHi; }

// The scale for a sum that is not safe, and what undoes it on the squares.
__device__ __forceinline__ float rescale(float s) { return s < kSafeLo ? 0x1p+100f : 0x1p-80f; }
__device__ __forceinline__ double unscale(float s) { return s < kSafeLo ? 0x1p-200 : 0x1p+160; }

struct Sum {
    float hi = 0.0f, lo = 0.0f;  // hi + lo: the safe batches
    double rare = 0.0;           // the others

    // hi + s exactly as the rounded sum and its error (Knuth's two-sum)
    __device__ __forceinline__ void add(float s) {
        const float t = hi + s;
        const float b = t - hi;
        lo += (hi - (t - b)) + (s - b);
        hi = t;
    }
};

// Sum over the CTA's threads, in a fixed order; valid in thread 0.
template <int THREADS>
__device__ __forceinline__ double block_sum(double x) {
    constexpr int WARPS = THREADS / 32;
    __shared__ double warp_sum[WARPS];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_down_sync(0xffffffffu, x, d);
    if (threadIdx.x % 32 == 0) warp_sum[threadIdx.x / 32] = x;
    __syncthreads();
    if (threadIdx.x < 32) {
        x = threadIdx.x < WARPS ? warp_sum[threadIdx.x] : 0.0;
#pragma unroll
        for (int d = WARPS / 2; d > 0; d >>= 1) x += __shfl_down_sync(0xffffffffu, x, d);
    }
    return x;
}

template <int THREADS>
__device__ __forceinline__ double block_sum(Sum s) {
    constexpr int WARPS = THREADS / 32;
    __shared__ float2 warp_sum[WARPS];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float hi = __shfl_down_sync(0xffffffffu, s.hi, d);
        const float lo = __shfl_down_sync(0xffffffffu, s.lo, d);
        s.add(hi);
        s.lo += lo;
    }
    if (threadIdx.x % 32 == 0) warp_sum[threadIdx.x / 32] = make_float2(s.hi, s.lo);
    double rare = 0.0;
    if (__syncthreads_or(s.rare != 0.0)) rare = block_sum<THREADS>(s.rare);
    if (threadIdx.x >= 32) return 0.0;
    if (threadIdx.x < WARPS) {
        s.hi = warp_sum[threadIdx.x].x;
        s.lo = warp_sum[threadIdx.x].y;
    }
#pragma unroll
    for (int d = WARPS / 2; d > 0; d >>= 1) {
        const float hi = __shfl_down_sync(0xffffffffu, s.hi, d);
        const float lo = __shfl_down_sync(0xffffffffu, s.lo, d);
        s.add(hi);
        s.lo += lo;
    }
    return (double)s.hi + (double)s.lo + rare;
}

// --------------------------------------------------------------------------
// walking a list of tensors
// --------------------------------------------------------------------------

__device__ __forceinline__ int64_t first_vec(const ListEntry &e) {
    return (int64_t)(e.vec0_ends >> 8);
}

// The entry that holds vector v of the run.
template <typename TAB>
__device__ __forceinline__ int find_entry(const TAB &tab, int64_t v) {
    const int b = (int)(v >> tab.shift);
    int lo = tab.first[b], hi = tab.first[b + 1];
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first_vec(tab.e[mid]) <= v) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// One vector of the run: bytes [begin, end) of the 16 at p belong to the
// tensor.  begin = end = 0: no vector.
struct VecRef {
    unsigned char *p;
    int kind, begin, end;
    __device__ __forceinline__ bool whole() const { return end - begin == 16; }
    __device__ __forceinline__ bool partial() const { return end - begin != 16 && end != 0; }
};

// The tensor's bytes of a partial vector, zeros in place of the others.
__device__ __forceinline__ uint4 load_partial(const VecRef r) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int x = 0; x < 16; x += 2)
        if (x >= r.begin && x < r.end)
            w[x / 4] |= (uint32_t)*reinterpret_cast<const uint16_t *>(r.p + x) << (x % 4 * 8);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __noinline__ void store_partial(const VecRef r, const uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int x = 0; x < 16; x += 2)
        if (x >= r.begin && x < r.end)
            *reinterpret_cast<uint16_t *>(r.p + x) = (uint16_t)(w[x / 4] >> (x % 4 * 8));
}

// An entry as a tile of several sees it, in vectors from the tile's first.
struct StagedEntry {
    unsigned char *base;  // where the tile's first vector would lie in this tensor
    int32_t start;        // the tensor's first vector (-1: before the tile)
    uint32_t ends;        // kind << 16 | head << 8 | tail
};

// A tile of U vectors per thread.  Most tiles of long tensors hold whole
// vectors of one tensor; the others stage their entries in shared memory
// and every thread finds its vectors' own.
template <int U>
struct Tile {
    static constexpr int kVecs = U * kListThreads;
    int64_t v0, v1;       // its vectors of the run
    unsigned char *p;     // where they lie, when one tensor holds them whole
    int kind;
    int lo, n;            // else: its entries, lo.. of the table, n of them

    template <typename TAB>
    __device__ __forceinline__ bool locate(const TAB &tab, int64_t t) {
        v0 = t * kVecs;
        v1 = min(v0 + kVecs, tab.vecs);
        lo = find_entry(tab, v0);
        const ListEntry &e = tab.e[lo];
        const int64_t a = first_vec(e), z = first_vec(tab.e[lo + 1]);
        const bool head = (e.vec0_ends & 0xf0) != 0, tail = (e.vec0_ends & 15) != 0;
        p = reinterpret_cast<unsigned char *>(e.base_kind & ~(uint64_t)15) + (v0 - a) * 16;
        kind = (int)(e.base_kind & 15);
        return !(head && v0 == a) && v1 <= z - tail;
    }

    // Every thread of the CTA takes part.
    template <typename TAB>
    __device__ __forceinline__ void stage(const TAB &tab, StagedEntry *staged) {
        n = find_entry(tab, v1 - 1) - lo + 1;
        __syncthreads();  // the last tile's entries are done with
        for (int k = threadIdx.x; k <= n; k += kListThreads) {
            const ListEntry &e = tab.e[lo + k];
            const int64_t a = first_vec(e) - v0;
            StagedEntry s;
            s.base = reinterpret_cast<unsigned char *>(e.base_kind & ~(uint64_t)15) - a * 16;
            s.start = (int32_t)min(max(a, (int64_t)-1), (int64_t)kVecs + 1);
            s.ends = (uint32_t)(e.base_kind & 15) << 16 | (uint32_t)(e.vec0_ends & 0xf0) << 4 |
                     (uint32_t)(e.vec0_ends & 15);
            staged[k] = s;
        }
        __syncthreads();
    }

    __device__ __forceinline__ VecRef ref(const StagedEntry *staged, int u) const {
        const int v = u * kListThreads + (int)threadIdx.x;
        if (v >= (int)(v1 - v0)) return VecRef{nullptr, 0, 0, 0};
        int i = 0, hi = n - 1;
        while (i < hi) {
            const int mid = (i + hi + 1) >> 1;
            if (staged[mid].start <= v) i = mid; else hi = mid - 1;
        }
        const StagedEntry s = staged[i];
        const int tail = (int)(s.ends & 0xff);
        VecRef r;
        r.p = s.base + v * 16;
        r.kind = (int)(s.ends >> 16);
        r.begin = v == s.start ? (int)(s.ends >> 8 & 0xff) : 0;
        r.end = tail != 0 && v + 1 == staged[i + 1].start ? tail : 16;
        return r;
    }
};

// --------------------------------------------------------------------------
// the norm
// --------------------------------------------------------------------------

// Adds the squares of two bf16 values: mixed-precision multiply-adds take
// them as they are, in half the instructions of widening them first (707 MB:
// 105 us, against 107).
__device__ __forceinline__ void add_squares(uint32_t w, float &s0, float &s1) {
    asm("{\n\t"
        ".reg .b16 x, y;\n\t"
        "mov.b32 {x, y}, %2;\n\t"
        "fma.rn.f32.bf16 %0, x, x, %0;\n\t"
        "fma.rn.f32.bf16 %1, y, y, %1;\n\t"
        "}"
        : "+f"(s0), "+f"(s1)
        : "r"(w));
}

// Adds the squares of the elements of a vector, times k each, to two chains.
template <bool SCALED>
__device__ __forceinline__ void squares(const uint4 &w, bool f32, float k, float &s0, float &s1) {
    if (f32) {
        const float f[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z),
                            __uint_as_float(w.w)};
#pragma unroll
        for (int l = 0; l < 4; l += 2) {
            const float x = SCALED ? f[l] * k : f[l], y = SCALED ? f[l + 1] * k : f[l + 1];
            s0 = __fmaf_rn(x, x, s0);
            s1 = __fmaf_rn(y, y, s1);
        }
    } else if (!SCALED) {
        add_squares(w.x, s0, s1);
        add_squares(w.y, s0, s1);
        add_squares(w.z, s0, s1);
        add_squares(w.w, s0, s1);
    } else {
        float f[8];
        unpack8(w, f);
#pragma unroll
        for (int l = 0; l < 8; l += 2) {
            const float x = SCALED ? f[l] * k : f[l], y = SCALED ? f[l + 1] * k : f[l + 1];
            s0 = __fmaf_rn(x, x, s0);
            s1 = __fmaf_rn(y, y, s1);
        }
    }
}

// Out of line, so that batches of zeros (the rows of an embedding that no token
// used) branch around its binary64 instructions.
__device__ __noinline__ double add_rare(double rare, float s, double k) {
    return rare + (double)s * k;
}

// Adds a batch of U vectors of gradients; f32(u): vector u holds fp32, not bf16.
template <int U, typename F32>
__device__ __forceinline__ void add_batch(Sum &sum, const uint4 (&w)[U], F32 f32) {
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) squares<false>(w[u], f32(u), 1.0f, s0, s1);
    const float s = s0 + s1;
    if (is_safe(s)) {
        sum.add(s);
        return;
    }
    s0 = s1 = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) squares<true>(w[u], f32(u), rescale(s), s0, s1);
    if (s0 + s1 != 0.0f) sum.rare = add_rare(sum.rare, s0 + s1, unscale(s));
}

// Adds a vector of two sums of squares.
__device__ __forceinline__ void add_sums(Sum &sum, const uint4 &w) {
    sum.rare += __hiloint2double(w.y, w.x) + __hiloint2double(w.w, w.z);
}

// With the CTAs resident on an SM (kNormCtas) this sets how much is in flight.
// 3 and 6 were taken over 4 and 6, which reads 1.41 GB in 197 us instead of
// 202 after reads, but takes 631 us instead of 611 for norm and clipping one
// after the other: its reads crowd out the write-back of what the clipping
// before left in L2.  Lists of small tensors are near their best with 3 and 6
// too (700 of them, 10 MB, one norm after the other: 6.9 us; 2 and 8: 7.1; 4
// and 6: 6.8; 3 and 7: 7.2).
constexpr int kNormU = 3;

// Lists of few tiles (12 KB each) take one launch: a cluster of at most the
// portable 8 CTAs, whose sums meet in shared memory.  Longer ones spread over
// the SMs, and a second launch adds the CTAs' sums.  4,000 fp32: 2.3 us with
// a cluster, 3.2 with two launches; 96,000 (32 tiles): 4.0 and 3.4.  The
// 12,304 sums of a d = 1024 layer take one cluster (9 tiles): its
// reduce-scatter and norm, one after the other, 42.3 us instead of 45.1.
// Tiles of many tensors take longer each: 1,900 of 17 fp32 (13 tiles) 9.3 us
// two tiles to a CTA, 6.6 spread out; so they get one tile per CTA or spread.
constexpr int kNormCluster = 8;

template <typename TAB>
bool fits_cluster(const TAB &tab, int64_t tiles) {
    return tiles <= (tab.count <= tiles ? 2 * kNormCluster : kNormCluster);
}

// The run's last vectors, 64 MB, are left in L2 for the clipping that
// follows from the end; those before are read with the streaming hint, so
// that they make no room for themselves.  Norm and clipping of 1.41 GB: 612
// us, against 628 without the hint; 617 with 32 MB, 614 with 160 MB.  This
// holds for lists of one table: of several, the clipping takes the tables
// first to last (1.52 GB in 4,000 tensors, three tables: 682 us; in 1,900: 660).
constexpr int64_t kNormKeep = (64ll << 20) / 16;
constexpr int kFinishThreads = 256;

__device__ __forceinline__ void write_clip(const NormOut &o, double sum) {
    const float norm = (float)sqrt(sum);
    o.clip[0] = norm;
    o.clip[1] = !isfinite(norm) ? __int_as_float(0x7fc00000)
                                : norm > o.max_norm ? __fdiv_rn(o.max_norm, norm) : 1.0f;
}

// One pass over the run: 2 or 4 bytes read per element and nothing written.
// Tiles go round the CTAs of a grid that is resident at once, so that at any
// time they read one window of the run; 1.41 GB of fp32 take 202 us (7.0
// TB/s), 707 MB of bf16 104 us.  With a contiguous share of the run for each
// CTA the same read was 5% slower.
//
// Its loads are plain ones (or streaming): this kernel may be resident while the
// one before it, a clipping, writes what it will read, and the non-coherent
// path is for memory that nothing writes meanwhile.
//
// CLUSTER: the grid is one cluster, whose first CTA adds the others' sums and
// writes the result.
template <typename TAB, bool CLUSTER>
__global__ void __launch_bounds__(kListThreads, kNormCtas)
k_grad_norm(const __grid_constant__ TAB tab, const NormOut o) {
    if constexpr (CLUSTER) cluster_arrive();
    using T = Tile<kNormU>;
    __shared__ StagedEntry staged[T::kVecs + 1];
    pdl_enter();
    Sum sum;
    const int64_t passing = tab.vecs - kNormKeep;
    const int64_t tiles = (tab.vecs + T::kVecs - 1) / T::kVecs;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        T tile{};
        uint4 w[kNormU];
        if (tile.locate(tab, t)) {
            const uint4 *p = reinterpret_cast<const uint4 *>(tile.p) + threadIdx.x;
            const int n = (int)(tile.v1 - tile.v0) - (int)threadIdx.x;
#pragma unroll
            for (int u = 0; u < kNormU; ++u)
                w[u] = u * kListThreads >= n ? make_uint4(0, 0, 0, 0)
                       : tile.v0 < passing   ? __ldcs(p + u * kListThreads)
                                             : p[u * kListThreads];
            if (tile.kind == Z3_F32) {
                add_batch(sum, w, [](int) { return true; });
            } else if (tile.kind == Z3_BF16) {
                add_batch(sum, w, [](int) { return false; });
            } else {
#pragma unroll
                for (int u = 0; u < kNormU; ++u) add_sums(sum, w[u]);
            }
            continue;
        }
        tile.stage(tab, staged);
        int kind[kNormU];
        bool sums = false;
#pragma unroll
        for (int u = 0; u < kNormU; ++u) {
            const VecRef r = tile.ref(staged, u);
            w[u] = r.whole() ? *reinterpret_cast<const uint4 *>(r.p) : make_uint4(0, 0, 0, 0);
            kind[u] = r.kind;
            if (r.partial()) w[u] = load_partial(r);
            sums |= r.kind == Z3_SUMSQ;
        }
        // a branch of the whole warp: as predicated instructions these binary64
        // additions would take the FP64 units' time in every mixed tile
        if (__any_sync(0xffffffffu, sums)) {
#pragma unroll
            for (int u = 0; u < kNormU; ++u) {
                if (kind[u] != Z3_SUMSQ) continue;
                add_sums(sum, w[u]);
                w[u] = make_uint4(0, 0, 0, 0);
            }
        }
        add_batch(sum, w, [&](int u) { return kind[u] == Z3_F32; });
    }
    const double all = block_sum<kListThreads>(sum);
    if constexpr (CLUSTER) {
        __shared__ double cta_sum[kNormCluster];
        cluster_wait();  // every CTA has started: its shared memory is there
        if (threadIdx.x == 0)
            *cooperative_groups::this_cluster().map_shared_rank(&cta_sum[blockIdx.x], 0) = all;
        cluster_arrive();
        cluster_wait();
        if (blockIdx.x != 0 || threadIdx.x != 0) return;
        double total = cta_sum[0];
        for (int b = 1; b < (int)gridDim.x; ++b) total += cta_sum[b];
        write_clip(o, total);
    } else {
        if (threadIdx.x == 0) o.ws->partial[blockIdx.x] = all;
    }
}

// Adds the n partials of the launch before it, in CTA order, to the sums of
// the call's earlier launches.  As a launch of its own it starts while the
// partials are computed, and its wait for them is shorter than a ticket
// taken by every CTA and a last one's sum: 912 tickets at one address took
// 1 us more.  Letting the next kernel start before this wait, too, gains nothing
// (norms one after the other: 700 tensors, 10 MB, 7.0 us against 7.2, 300
// tensors, 17 MB, 7.7 against 7.0, 707 MB the same), and the early variants of
// other kernels rest on its not being done.
__global__ void __launch_bounds__(kFinishThreads) k_norm_finish(const NormOut o, int n) {
    pdl_enter();
    constexpr int PER = (kNormMaxGrid + kFinishThreads - 1) / kFinishThreads;
    double x[PER];  // all loads in flight at once
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = i * kFinishThreads + threadIdx.x;
        x[i] = b < n ? o.ws->partial[b] : 0.0;
    }
    double sum = x[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) sum += x[i];
    sum = block_sum<kFinishThreads>(sum);
    if (threadIdx.x != 0) return;
    if (!o.first) sum += o.ws->carry;
    if (o.last) write_clip(o, sum);
    else o.ws->carry = sum;
}

// --------------------------------------------------------------------------
// clipping
// --------------------------------------------------------------------------

__device__ __forceinline__ uint4 scaled(const uint4 &w, int kind, float c) {
    if (kind == Z3_F32)
        return make_uint4(__float_as_uint(__fmul_rn(__uint_as_float(w.x), c)),
                          __float_as_uint(__fmul_rn(__uint_as_float(w.y), c)),
                          __float_as_uint(__fmul_rn(__uint_as_float(w.z), c)),
                          __float_as_uint(__fmul_rn(__uint_as_float(w.w), c)));
    float f[8];
    unpack8(w, f);
#pragma unroll
    for (int l = 0; l < 8; ++l) f[l] = __fmul_rn(f[l], c);
    return pack8(f);
}

constexpr int kClipU = 2;

// One product per element and one rounding to its type; each element is read
// and written once.  One tile per CTA, the last tiles first: what the norm
// read last is still in L2 (1.41 GB of fp32, norm and clipping: 628 us in the
// other order).  Alone, that clipping takes 398 us, 7.1 TB/s; 415 with one
// vector per thread, 399 with four, 476 with one contiguous share per CTA.
// Where coef is 1 the CTAs still start, look their tile up and leave: 175 us for
// those 172,609, 3.7 us for a d = 1024 layer in bf16 (8.9 with a coef).
template <typename TAB>
__global__ void __launch_bounds__(kListThreads, 8)
k_clip(const __grid_constant__ TAB tab, const float *clip) {
    using T = Tile<kClipU>;
    __shared__ StagedEntry staged[T::kVecs + 1];
    pdl_enter();
    const float c = clip[1];
    T tile{};
    const bool one = tile.locate(tab, (int64_t)gridDim.x - 1 - blockIdx.x);
    if (c == 1.0f || isnan(c)) return;  // nothing changes; no step to take
    if (one) {
        uint4 *p = reinterpret_cast<uint4 *>(tile.p) + threadIdx.x;
        const int n = (int)(tile.v1 - tile.v0) - (int)threadIdx.x;
        uint4 w[kClipU];
#pragma unroll
        for (int u = 0; u < kClipU; ++u)
            if (u * kListThreads < n) w[u] = p[u * kListThreads];
#pragma unroll
        for (int u = 0; u < kClipU; ++u)
            if (u * kListThreads < n) p[u * kListThreads] = scaled(w[u], tile.kind, c);
        return;
    }
    tile.stage(tab, staged);
    VecRef r[kClipU];
    uint4 w[kClipU];
#pragma unroll
    for (int u = 0; u < kClipU; ++u) {
        r[u] = tile.ref(staged, u);
        if (r[u].whole()) w[u] = *reinterpret_cast<const uint4 *>(r[u].p);
    }
#pragma unroll
    for (int u = 0; u < kClipU; ++u)
        if (r[u].whole()) *reinterpret_cast<uint4 *>(r[u].p) = scaled(w[u], r[u].kind, c);
#pragma unroll
    for (int u = 0; u < kClipU; ++u)
        if (r[u].partial()) store_partial(r[u], scaled(load_partial(r[u]), r[u].kind, c));
}

// --------------------------------------------------------------------------
// ReduceScatter that also leaves one sum of squares per tile
//
// In a warp, 8 multiply-adds and 5 additions of binary32 lie on a square's
// way: 13 roundings, as in a batch of the norm; binary64 from there on.
//
// z3_reduce_scatter's fold, tiles and stores; the squares are taken of the
// registers that are stored, so the norm costs no second read of the
// gradient (4 bytes per element) but the one barrier that joins a CTA's
// warps: 37.9 us instead of 36.6 for the d = 1024 layer over 8 ranks, 259
// instead of 256 for a [50257, 1024] embedding over 16.  At the 64 registers
// that keep eight CTAs on an SM the aligned form spills 16 bytes per thread.
// --------------------------------------------------------------------------

// A thread's share of its tile's sum of squares: s * 2^e, in binary32 where
// that is safe (e = 0).
struct TileSum {
    float s;
    int e;
    __device__ __forceinline__ double value() const {
        return (double)s * (e == 0 ? 1.0 : e < 0 ? 0x1p-200 : 0x1p+160);
    }
};

__device__ __forceinline__ TileSum tile_sum(const float g[8]) {
    float s = 0.0f;
#pragma unroll
    for (int l = 0; l < 8; ++l) s = __fmaf_rn(g[l], g[l], s);
    if (is_safe(s)) return {s, 0};
    const int e = s < kSafeLo ? -200 : 160;
    const float k = rescale(s);
    s = 0.0f;
#pragma unroll
    for (int l = 0; l < 8; ++l) s = __fmaf_rn(g[l] * k, g[l] * k, s);
    return {s, s == 0.0f ? 0 : e};
}

// The sum over the CTA, stored by one thread: in binary32 within each warp,
// unless one of its lanes could not hold its own share so.
__device__ __forceinline__ void store_tile_sum(const TileSum &t, double *out) {
    constexpr int WARPS = kReduceThreads / 32;
    __shared__ double warp_sum[WARPS];
    double w;
    if (__any_sync(0xffffffffu, t.e != 0)) {
        w = t.value();
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) w += __shfl_down_sync(0xffffffffu, w, d);
    } else {
        float s = t.s;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_down_sync(0xffffffffu, s, d);
        w = s;
    }
    if (threadIdx.x % 32 == 0) warp_sum[threadIdx.x / 32] = w;
    __syncthreads();
    if (threadIdx.x != 0) return;
    w = warp_sum[0];
#pragma unroll
    for (int i = 1; i < WARPS; ++i) w += warp_sum[i];
    *out = w;
}

template <int PHI, bool ACC, bool EARLY>
__device__ __forceinline__ TileSum reduce_norm_vector(const ReduceNormArgs &a, int n_ranks,
                                                     int64_t x0, int64_t delta) {
    float g[8];
    fold_vector<PHI>(a.grads, a.stride, a.scale, n_ranks, x0, delta, g);
    if constexpr (ACC) {
        float o[8];
        ld8f(a.grad_shards + x0, o);
#pragma unroll
        for (int l = 0; l < 8; ++l) g[l] = __fadd_rn(o[l], g[l]);
    }
    if constexpr (EARLY) pdl_enter();
    st8f(a.grad_shards + x0, g);
    return tile_sum(g);
}

template <bool ACC>
__device__ __noinline__ TileSum reduce_norm_edges(const ReduceNormArgs a, int n_ranks, int64_t x0,
                                                  int64_t delta, int64_t c0, int64_t c_end,
                                                  int64_t valid_end) {
    double s = 0.0;
    for (int l = 0; l < kVec; ++l) {
        const int64_t x = x0 + l;
        if (x < c0 || x >= c_end) continue;  // another chunk's element
        float g = 0.0f;
        if (x < valid_end) {
            g = fold_element(a.grads, a.stride, a.scale, n_ranks, x, delta);
            if constexpr (ACC) g = __fadd_rn(a.grad_shards[x], g);
        }
        a.grad_shards[x] = g;
        s += (double)g * (double)g;
    }
    if (s == 0.0 || is_safe((float)s)) return {(float)s, 0};
    return s < kSafeLo ? TileSum{(float)(s * 0x1p+200), -200} : TileSum{(float)(s * 0x1p-160), 160};
}

template <bool ALIGNED, bool ACC, bool EARLY>
__global__ void __launch_bounds__(kReduceThreads, 1024 / kReduceThreads)
k_reduce_norm(const __grid_constant__ Tab tab, const ReduceNormArgs a) {
    if constexpr (!EARLY) pdl_enter();
    const TileRef tr = locate<false>(tab, blockIdx.x);
    const TabEntry &e = tab.e[tr.p];
    const int64_t c0 = tr.r * tab.S + e.o;
    const int64_t c_end = c0 + e.s;
    const int64_t valid_end = c0 + min(e.s, max((int64_t)0, e.n - tr.r * e.s));
    const int64_t delta = e.F + tr.r * e.s - c0;
    const int64_t x0 = (c0 / kVec + tr.t * (int64_t)kReduceThreads + threadIdx.x) * kVec;
    const int n = tab.n_ranks;
    TileSum s;
    if (x0 >= c0 && x0 + kVec <= valid_end) {
        if constexpr (ALIGNED) {
            s = reduce_norm_vector<0, ACC, EARLY>(a, n, x0, delta);
        } else {
            switch ((int)(((delta % kVec) + kVec) % kVec)) {
                case 0: s = reduce_norm_vector<0, ACC, EARLY>(a, n, x0, delta); break;
                case 1: s = reduce_norm_vector<1, ACC, EARLY>(a, n, x0, delta); break;
                case 2: s = reduce_norm_vector<2, ACC, EARLY>(a, n, x0, delta); break;
                case 3: s = reduce_norm_vector<3, ACC, EARLY>(a, n, x0, delta); break;
                case 4: s = reduce_norm_vector<4, ACC, EARLY>(a, n, x0, delta); break;
                case 5: s = reduce_norm_vector<5, ACC, EARLY>(a, n, x0, delta); break;
                case 6: s = reduce_norm_vector<6, ACC, EARLY>(a, n, x0, delta); break;
                default: s = reduce_norm_vector<7, ACC, EARLY>(a, n, x0, delta); break;
            }
        }
    } else {
        if constexpr (EARLY) pdl_enter();
        s = x0 < c_end ? reduce_norm_edges<ACC>(a, n, x0, delta, c0, c_end, valid_end)
                       : TileSum{0.0f, 0};
    }
    store_tile_sum(s, a.sumsq + blockIdx.x);
}

// --------------------------------------------------------------------------
// Adam over the flat [N][S] shard buffers of one or several units, on coef *
// gradient
// --------------------------------------------------------------------------

// Bound by HBM: 16 bytes read and 14 written per element.  One launch for all
// units: the 25 updates of the 24-layer model took 1.57 ms as launches of
// their own, 1.51 ms as one.  Reading the state before the wait for the norm
// did not help (a d = 1024 layer's step: 113 us with it, 111 without).
template <typename UNITS>
__global__ void __launch_bounds__(kAdamThreads)
k_adam_clipped(const __grid_constant__ UNITS units, const float *clip) {
    pdl_enter();
    const float coef = clip[1];
    if (isnan(coef)) return;  // no step to take
    int i = 0;
    if constexpr (UNITS::kCap > 1) {
        int hi = units.count - 1;
        while (i < hi) {
            const int mid = (i + hi + 1) >> 1;
            if (units.block0[mid] <= blockIdx.x) i = mid; else hi = mid - 1;
        }
    }
    const AdamArgs &a = units.u[i];
    const int64_t x0 =
        ((int64_t)(blockIdx.x - units.block0[i]) * kAdamThreads + threadIdx.x) * kVec;
    if (x0 + kVec <= a.total) {
        float g[8], p[8], m[8], v[8];
        ld8f(a.grad + x0, g);
        ld8f(a.master + x0, p);
        ld8f(a.m + x0, m);
        ld8f(a.v + x0, v);
#pragma unroll
        for (int l = 0; l < 8; ++l) adam1(__fmul_rn(g[l], coef), p[l], m[l], v[l], a.k);
        st8f(a.master + x0, p);
        st8f(a.m + x0, m);
        st8f(a.v + x0, v);
        *reinterpret_cast<uint4 *>(a.shards + x0) = pack8(p);
    } else {
        for (int64_t x = x0; x < a.total; ++x) {
            float p = a.master[x], m = a.m[x], v = a.v[x];
            adam1(__fmul_rn(a.grad[x], coef), p, m, v, a.k);
            a.master[x] = p;
            a.m[x] = m;
            a.v[x] = v;
            a.shards[x] = f32_to_bf16(p);
        }
    }
}

// --------------------------------------------------------------------------
// launches over a tensor list
// --------------------------------------------------------------------------

// launch() for a kernel with a table, which it does not copy on its way to
// the runtime; cluster: the whole grid is one.
template <typename TAB, typename ARG>
void launch_list(void (*kernel)(TAB, ARG), int64_t grid, cudaStream_t stream, const TAB &tab,
                 const ARG &arg, bool cluster = false) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)kListThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)grid;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    void *args[2] = {const_cast<TAB *>(&tab), const_cast<ARG *>(&arg)};
    (void)cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(kernel), args);
}

template <int U, typename TAB>
int64_t tiles_of(const TAB &tab) {
    return (tab.vecs + U * kListThreads - 1) / (U * kListThreads);
}

template <typename TAB>
void norm_launches(const std::vector<TAB> &tabs, NormOut o, cudaStream_t stream) {
    for (const TAB &tab : tabs) {
        const int64_t tiles = std::max<int64_t>(1, tiles_of<kNormU>(tab));
        o.first = &tab == &tabs.front();
        o.last = &tab == &tabs.back();
        if (o.first && o.last && fits_cluster(tab, tiles)) {
            launch_list(k_grad_norm<TAB, true>, std::min<int64_t>(tiles, kNormCluster), stream,
                        tab, o, true);
            return;
        }
        const int64_t grid = std::min<int64_t>(kNormMaxGrid, tiles);
        launch_list(k_grad_norm<TAB, false>, grid, stream, tab, o);
        launch(k_norm_finish, 1, kFinishThreads, stream, o, (int)grid);
    }
}

template <typename TAB>
void clip_launches(const std::vector<TAB> &tabs, const float *clip, cudaStream_t stream) {
    for (const TAB &tab : tabs)
        if (tab.count > 0) launch_list(k_clip<TAB>, tiles_of<kClipU>(tab), stream, tab, clip);
}

}  // namespace

// --------------------------------------------------------------------------
// launchers
// --------------------------------------------------------------------------

cudaError_t launch_grad_norm(const z3_tensor_list *list, float max_norm, float *clip,
                             NormWorkspace *ws, cudaStream_t stream) {
    const NormOut o{clip, ws, max_norm, 0, 0};
    norm_launches(list->tabs4, o, stream);
    norm_launches(list->tabs8, o, stream);
    norm_launches(list->tabs16, o, stream);
    norm_launches(list->tabs32, o, stream);
    return cudaGetLastError();
}

cudaError_t launch_clip(const z3_tensor_list *list, const float *clip, cudaStream_t stream) {
    clip_launches(list->tabs4, clip, stream);
    clip_launches(list->tabs8, clip, stream);
    clip_launches(list->tabs16, clip, stream);
    clip_launches(list->tabs32, clip, stream);
    return cudaGetLastError();
}

template <bool ACC>
static void reduce_norm_launches(const z3_layout *L, ReduceNormArgs a, cudaStream_t stream,
                                 bool early) {
    for (const Tab &t : L->reduce_tabs) {
        if (t.phase0) {
            if (early) launch(k_reduce_norm<true, ACC, true>, t.tiles, kReduceThreads, stream, t, a);
            else launch(k_reduce_norm<true, ACC, false>, t.tiles, kReduceThreads, stream, t, a);
        } else {
            if (early) launch(k_reduce_norm<false, ACC, true>, t.tiles, kReduceThreads, stream, t, a);
            else launch(k_reduce_norm<false, ACC, false>, t.tiles, kReduceThreads, stream, t, a);
        }
        a.sumsq += t.tiles;
        // the next table's predecessor is this launch, which writes other
        // shard positions and other sums
        early = true;
    }
}

cudaError_t launch_reduce_norm(const z3_layout *L, const ReduceNormArgs &a, bool accumulate,
                               cudaStream_t stream, bool early) {
    if (accumulate) reduce_norm_launches<true>(L, a, stream, early);
    else reduce_norm_launches<false>(L, a, stream, early);
    return cudaGetLastError();
}

namespace {
template <typename UNITS>
void adam_launches(const AdamArgs *a, int32_t n, const float *clip, cudaStream_t stream) {
    UNITS t;
    for (int32_t i = 0; i < n;) {
        int64_t blocks = 0;
        for (t.count = 0; i < n && t.count < UNITS::kCap; ++i) {
            const int64_t b = flat_blocks(a[i].total, kAdamThreads);
            if (b == 0) continue;
            if (t.count > 0 && blocks + b > 0x7fffffff) break;
            t.block0[t.count] = (uint32_t)blocks;
            t.u[t.count++] = a[i];
            blocks += b;
        }
        if (t.count > 0) launch(k_adam_clipped<UNITS>, blocks, kAdamThreads, stream, t, clip);
    }
}
}  // namespace

cudaError_t launch_adam_clipped(const AdamArgs *a, int32_t n, const float *clip,
                                cudaStream_t stream) {
    if (n == 1) adam_launches<AdamUnits<1>>(a, n, clip, stream);
    else adam_launches<AdamUnits<40>>(a, n, clip, stream);
    return cudaGetLastError();
}

}  // namespace z3
