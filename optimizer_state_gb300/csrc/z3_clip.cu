// z3_clip.cu -- gradient clipping by the global norm: the norm over many
// tensors, clipping in place, the reduce-scatter that leaves its sums of
// squares, and the clipped shard Adam.
//
//   norm = sqrt(sum of g^2 over every element of every tensor)
//   coef = max_norm / norm where norm > max_norm, else 1; NaN where the norm
//          is not finite, and then nothing is written by what reads coef
//
// Sums of squares are held in binary64 across threads, in an order fixed by
// the sizes alone (no floating-point atomics): a call gives the same bits
// every time.  Every kernel is bound by HBM bandwidth; nothing contracts, so
// no tensor cores.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>

#include "z3_clip.h"
#include "z3_device.cuh"

namespace z3 {
namespace {

// --------------------------------------------------------------------------
// sums of squares
// --------------------------------------------------------------------------

// Squares are added in binary32 within one batch of a thread (at most 32
// elements in two chains), where they are exact to 2^-20, and in binary64
// beyond it: a binary64 addition for every element would bound the kernels
// by the few FP64 units (one clipped layer's reduce-scatter took 98 us that
// way, against 45 us).  A batch whose sum leaves [kSafeLo, kSafeHi] may have
// lost squares to underflow or overflow; it is summed again with its
// elements scaled by a power of two.  Above kSafeLo the squares that
// underflowed change the sum by under 2^-50 of it; scaled up from below
// kSafeLo, elements stay under 2^55 and the least subnormal's square is
// 2^-98; scaled down from above kSafeHi, what underflows is under 2^-60 of
// the sum.  Infinities and NaN stay what they are.
constexpr float kSafeLo = 0x1p-90f, kSafeHi = 0x1p+120f;

__device__ __forceinline__ bool is_safe(float s) { return s >= kSafeLo && s <= kSafeHi; }

// The scale for a sum that is not safe, and what undoes it on the squares.
__device__ __forceinline__ float rescale(float s) { return s < kSafeLo ? 0x1p+100f : 0x1p-100f; }
__device__ __forceinline__ double unscale(float s) { return s < kSafeLo ? 0x1p-200 : 0x1p+200; }

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

// --------------------------------------------------------------------------
// walking a list of tensors
// --------------------------------------------------------------------------

// One CTA's part of one tensor: n vectors from p, of which bytes
// [begin, end) belong to the tensor.  Vectors [lo, hi) are the tensor's
// whole; a partial one before or after them is handled by elements.
struct Segment {
    unsigned char *p;
    int64_t n, begin, end;
    int64_t lo, hi;
    int kind;
};

// The part of entry i that lies in vectors [v0, v1) of the run.
template <typename TAB>
__device__ __forceinline__ Segment segment(const TAB &tab, int i, int64_t v0, int64_t v1) {
    const ListEntry &e = tab.e[i];
    const int64_t a = (int64_t)(e.vec0_ends >> 8), b = (int64_t)(tab.e[i + 1].vec0_ends >> 8);
    const int64_t s = max(v0, a), t = min(v1, b);
    Segment g;
    g.kind = (int)(e.base_kind & 15);
    g.p = reinterpret_cast<unsigned char *>(e.base_kind & ~(uint64_t)15) + (s - a) * 16;
    g.n = t - s;
    const int head = (int)(e.vec0_ends >> 4) & 15, tail = (int)e.vec0_ends & 15;
    g.begin = s == a ? head : 0;
    g.end = t == b && tail != 0 ? g.n * 16 - 16 + tail : g.n * 16;
    g.lo = g.begin != 0 ? 1 : 0;
    g.hi = max(g.lo, g.end / 16);
    return g;
}

// The byte offset of the element of a partial vector that this thread
// handles, or -1: threads 0-7 take the first vector's, 8-15 the last's.
__device__ __forceinline__ int64_t edge_element(const Segment &g, int size) {
    const int l = threadIdx.x & 7;
    if (threadIdx.x >= 16 || l * size >= 16) return -1;
    const bool last = threadIdx.x >= 8;
    if (last ? g.hi * 16 >= g.end : g.lo == 0) return -1;  // no partial vector there
    const int64_t x = (last ? g.hi * 16 : 0) + l * size;
    return x >= g.begin && x < g.end ? x : -1;
}

// Vectors in flight per thread.
constexpr int kListBatch = 4;

// Sum of squares of the batch's elements times k.
template <bool SCALED>
__device__ __forceinline__ float squares(const uint4 (&w)[kListBatch], int kind, float k) {
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int u = 0; u < kListBatch; ++u) {
        if (kind == Z3_F32) {
            float f[4] = {__uint_as_float(w[u].x), __uint_as_float(w[u].y),
                          __uint_as_float(w[u].z), __uint_as_float(w[u].w)};
#pragma unroll
            for (int l = 0; l < 4; l += 2) {
                const float x = SCALED ? f[l] * k : f[l], y = SCALED ? f[l + 1] * k : f[l + 1];
                s0 = __fmaf_rn(x, x, s0);
                s1 = __fmaf_rn(y, y, s1);
            }
        } else {
            float f[8];
            unpack8(w[u], f);
#pragma unroll
            for (int l = 0; l < 8; l += 2) {
                const float x = SCALED ? f[l] * k : f[l], y = SCALED ? f[l + 1] * k : f[l + 1];
                s0 = __fmaf_rn(x, x, s0);
                s1 = __fmaf_rn(y, y, s1);
            }
        }
    }
    return s0 + s1;
}

// --------------------------------------------------------------------------
// the norm
// --------------------------------------------------------------------------

template <typename TAB>
__global__ void __launch_bounds__(kListThreads, kListCtas)
k_grad_norm(const __grid_constant__ TAB tab, const NormOut o) {
    pdl_enter();
    const int64_t v0 = tab.vecs * blockIdx.x / tab.grid;
    const int64_t v1 = tab.vecs * (blockIdx.x + 1) / tab.grid;
    double sum = 0.0;
    for (int i = tab.first[blockIdx.x]; i < tab.count; ++i) {
        if ((int64_t)(tab.e[i].vec0_ends >> 8) >= v1) break;
        const Segment g = segment(tab, i, v0, v1);
        if (g.kind == Z3_SUMSQ) {
            const double *d = reinterpret_cast<const double *>(g.p);
            for (int64_t x = g.begin / 8 + threadIdx.x; x < g.end / 8; x += kListThreads)
                sum += d[x];
            continue;
        }
        const uint4 *p = reinterpret_cast<const uint4 *>(g.p);
        for (int64_t q = g.lo + threadIdx.x; q < g.hi; q += kListBatch * kListThreads) {
            uint4 w[kListBatch];
#pragma unroll
            for (int u = 0; u < kListBatch; ++u)
                w[u] = q + u * kListThreads < g.hi ? __ldg(p + q + u * kListThreads)
                                                   : make_uint4(0, 0, 0, 0);
            const float s = squares<false>(w, g.kind, 1.0f);
            sum += is_safe(s) ? (double)s
                              : (double)squares<true>(w, g.kind, rescale(s)) * unscale(s);
        }
        const int64_t x = edge_element(g, g.kind == Z3_F32 ? 4 : 2);
        if (x >= 0) {
            const double f = g.kind == Z3_F32 ? *reinterpret_cast<const float *>(g.p + x)
                                              : bf16_to_f32(*reinterpret_cast<const uint16_t *>(g.p + x));
            sum += f * f;
        }
    }
    sum = block_sum<kListThreads>(sum);
    // the last CTA to store its partial adds them all, in CTA order
    __shared__ bool last;
    if (threadIdx.x == 0) {
        o.ws->partial[blockIdx.x] = sum;
        __threadfence();
        last = atomicInc(&o.ws->ticket, gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double all = 0.0;
    for (int b = threadIdx.x; b < (int)gridDim.x; b += kListThreads)
        all += __ldcg(&o.ws->partial[b]);
    all = block_sum<kListThreads>(all);
    if (threadIdx.x != 0) return;
    if (!o.first) all += __ldcg(&o.ws->carry);
    if (!o.last) {
        o.ws->carry = all;
        return;
    }
    const float norm = (float)sqrt(all);
    o.clip[0] = norm;
    o.clip[1] = !isfinite(norm) ? __int_as_float(0x7fc00000)
                                : norm > o.max_norm ? __fdiv_rn(o.max_norm, norm) : 1.0f;
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

// Each CTA walks its share backwards: what the norm read last is still in L2.
template <typename TAB>
__global__ void __launch_bounds__(kListThreads, kListCtas)
k_clip(const __grid_constant__ TAB tab, const float *clip) {
    pdl_enter();
    const float c = __ldcg(clip + 1);
    if (c == 1.0f || isnan(c)) return;  // nothing changes; no step to take
    const int b = blockIdx.x;
    const int64_t v0 = tab.vecs * b / tab.grid;
    const int64_t v1 = tab.vecs * (b + 1) / tab.grid;
    for (int i = b + 1 < tab.grid ? tab.first[b + 1] : tab.count - 1; i >= tab.first[b]; --i) {
        if ((int64_t)(tab.e[i].vec0_ends >> 8) >= v1) continue;
        const Segment g = segment(tab, i, v0, v1);
        uint4 *p = reinterpret_cast<uint4 *>(g.p);
        for (int64_t q = g.hi - 1 - threadIdx.x; q >= g.lo; q -= kListBatch * kListThreads) {
            uint4 w[kListBatch];
#pragma unroll
            for (int u = 0; u < kListBatch; ++u)
                if (q - u * kListThreads >= g.lo) w[u] = p[q - u * kListThreads];
#pragma unroll
            for (int u = 0; u < kListBatch; ++u)
                if (q - u * kListThreads >= g.lo) p[q - u * kListThreads] = scaled(w[u], g.kind, c);
        }
        const int64_t x = edge_element(g, g.kind == Z3_F32 ? 4 : 2);
        if (x >= 0 && g.kind == Z3_F32) {
            float *f = reinterpret_cast<float *>(g.p + x);
            *f = __fmul_rn(*f, c);
        } else if (x >= 0) {
            uint16_t *h = reinterpret_cast<uint16_t *>(g.p + x);
            *h = f32_to_bf16(__fmul_rn(bf16_to_f32(*h), c));
        }
    }
}

// --------------------------------------------------------------------------
// ReduceScatter that also leaves one sum of squares per tile
// --------------------------------------------------------------------------

// A thread's share of its tile's sum of squares: s * 2^e, in binary32 where
// that is safe (e = 0).
struct TileSum {
    float s;
    int e;
    __device__ __forceinline__ double value() const {
        return (double)s * (e == 0 ? 1.0 : e < 0 ? 0x1p-200 : 0x1p+200);
    }
};

__device__ __forceinline__ TileSum tile_sum(const float g[8]) {
    float s = 0.0f;
#pragma unroll
    for (int l = 0; l < 8; ++l) s = __fmaf_rn(g[l], g[l], s);
    if (is_safe(s)) return {s, 0};
    const int e = s < kSafeLo ? -200 : 200;
    const float k = e < 0 ? 0x1p+100f : 0x1p-100f;
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
    return s < kSafeLo ? TileSum{(float)(s * 0x1p+200), -200} : TileSum{(float)(s * 0x1p-200), 200};
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
// Adam over the flat [N][S] shard buffers on coef * gradient
// --------------------------------------------------------------------------

template <bool EARLY>
__global__ void __launch_bounds__(kAdamThreads) k_adam_clipped(const AdamClipArgs c) {
    if constexpr (!EARLY) pdl_enter();
    const AdamArgs &a = c.a;
    const int64_t x0 = ((int64_t)blockIdx.x * kAdamThreads + threadIdx.x) * kVec;
    const float coef = __ldcg(c.clip + 1);
    if (isnan(coef)) {  // no step to take
        if constexpr (EARLY) pdl_enter();
        return;
    }
    if (x0 >= a.total) return;
    if (x0 + kVec <= a.total) {
        float g[8], p[8], m[8], v[8];
        ld8f(a.grad + x0, g);
        ld8f(a.master + x0, p);
        ld8f(a.m + x0, m);
        ld8f(a.v + x0, v);
#pragma unroll
        for (int l = 0; l < 8; ++l) adam1(__fmul_rn(g[l], coef), p[l], m[l], v[l], a.k);
        if constexpr (EARLY) pdl_enter();
        st8f(a.master + x0, p);
        st8f(a.m + x0, m);
        st8f(a.v + x0, v);
        *reinterpret_cast<uint4 *>(a.shards + x0) = pack8(p);
    } else {
        if constexpr (EARLY) pdl_enter();
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
// launch tables of a tensor list
// --------------------------------------------------------------------------

// Fills tab from tensors[at...], as many as it holds; returns the next index.
template <typename TAB>
int32_t fill(TAB &tab, const z3_tensor *tensors, int32_t n, int32_t at) {
    tab.count = 0;
    int64_t vecs = 0;
    for (; at < n && tab.count < TAB::kCap; ++at) {
        const z3_tensor &t = tensors[at];
        if (t.numel == 0) continue;
        const uint64_t a = reinterpret_cast<uintptr_t>(t.data);
        const uint64_t z = a + (uint64_t)(t.numel * list_dtype_bytes(t.dtype));
        ListEntry &e = tab.e[tab.count++];
        e.base_kind = (a & ~(uint64_t)15) | (uint64_t)t.dtype;
        e.vec0_ends = (uint64_t)vecs << 8 | (a & 15) << 4 | (z & 15);
        vecs += (int64_t)((z + 15) / 16 - a / 16);
    }
    tab.e[tab.count].base_kind = 0;
    tab.e[tab.count].vec0_ends = (uint64_t)vecs << 8;
    tab.vecs = vecs;
    tab.grid = (int32_t)std::min<int64_t>(kListMaxGrid,
                                          std::max<int64_t>(1, vecs / (2 * kListThreads)));
    int32_t i = 0;
    for (int32_t b = 0; b < tab.grid; ++b) {
        const uint64_t v0 = (uint64_t)(vecs * b / tab.grid);
        while (i + 1 < tab.count && (tab.e[i + 1].vec0_ends >> 8) <= v0) ++i;
        tab.first[b] = (uint16_t)i;
    }
    return at;
}

template <typename TAB>
void norm_launches(const z3_tensor *tensors, int32_t n, NormOut o, cudaStream_t stream) {
    TAB tab;
    int32_t at = 0;
    o.first = 1;
    do {
        at = fill(tab, tensors, n, at);
        o.last = at == n;
        launch(k_grad_norm<TAB>, tab.grid, kListThreads, stream, tab, o);
        o.first = 0;
    } while (at < n);
}

template <typename TAB>
void clip_launches(const z3_tensor *tensors, int32_t n, const float *clip, cudaStream_t stream) {
    TAB tab;
    for (int32_t at = 0; at < n;) {
        at = fill(tab, tensors, n, at);
        if (tab.count > 0) launch(k_clip<TAB>, tab.grid, kListThreads, stream, tab, clip);
    }
}

}  // namespace

// --------------------------------------------------------------------------
// launchers
// --------------------------------------------------------------------------

cudaError_t launch_grad_norm(const z3_tensor *tensors, int32_t n, float max_norm, float *clip,
                             NormWorkspace *ws, cudaStream_t stream) {
    const NormOut o{clip, ws, max_norm, 0, 0};
    if (n <= ListSmall::kCap) norm_launches<ListSmall>(tensors, n, o, stream);
    else norm_launches<ListLarge>(tensors, n, o, stream);
    return cudaGetLastError();
}

cudaError_t launch_clip(const z3_tensor *tensors, int32_t n, const float *clip,
                        cudaStream_t stream) {
    if (n <= ListSmall::kCap) clip_launches<ListSmall>(tensors, n, clip, stream);
    else clip_launches<ListLarge>(tensors, n, clip, stream);
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

cudaError_t launch_adam_clipped(const AdamClipArgs &a, cudaStream_t stream, bool early) {
    const int64_t blocks = flat_blocks(a.a.total, kAdamThreads);
    if (early) launch(k_adam_clipped<true>, blocks, kAdamThreads, stream, a);
    else launch(k_adam_clipped<false>, blocks, kAdamThreads, stream, a);
    return cudaGetLastError();
}

}  // namespace z3
