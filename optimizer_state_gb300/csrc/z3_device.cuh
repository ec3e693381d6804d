// z3_device.cuh -- device code shared by the kernel translation units
// (z3_kernels.cu, z3_clip.cu): bf16 conversions, window shifting, the Adam
// arithmetic, the rank fold, the map from CTAs to tiles, and the launch with
// programmatic stream serialisation.  One definition of each keeps every
// kernel's numerics the same.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "z3_launch.h"

namespace z3 {


// --------------------------------------------------------------------------
// small device helpers
// --------------------------------------------------------------------------

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ float bf16_to_f32(uint16_t h) {
    return __uint_as_float(static_cast<uint32_t>(h) << 16);
}

__device__ __forceinline__ uint16_t f32_to_bf16(float x) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);  // .x (low half) = lo
    return *reinterpret_cast<uint32_t *>(&h);
}

__device__ __forceinline__ void unpack8(const uint4 &w, float f[8]) {
    f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x);
    f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
    f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z);
    f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
}

// Eight bf16 values from a 16-byte boundary.  A plain load: the kernel may have
// started while the one before it still writes them (pdl_enter), which is
// not what the non-coherent path is for; nor may the compiler move a plain
// load across the wait.  No const pointer is __restrict__ for the same reason.
__device__ __forceinline__ uint4 ld8b(const uint16_t *p) {
    return *reinterpret_cast<const uint4 *>(p);
}

// Elements [PHI, PHI+8) of the 16-element window (lo, hi) of bf16 values.
template <int PHI>
__device__ __forceinline__ uint4 window8(const uint4 &lo, const uint4 &hi) {
    if constexpr (PHI == 0) {
        return lo;
    } else {
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        constexpr int q = PHI >> 1;
        uint4 r;
        if constexpr ((PHI & 1) != 0) {
            r.x = __funnelshift_r(w[q], w[q + 1], 16);
            r.y = __funnelshift_r(w[q + 1], w[q + 2], 16);
            r.z = __funnelshift_r(w[q + 2], w[q + 3], 16);
            r.w = __funnelshift_r(w[q + 3], w[q + 4], 16);
        } else {
            r.x = w[q];
            r.y = w[q + 1];
            r.z = w[q + 2];
            r.w = w[q + 3];
        }
        return r;
    }
}

// Kingma & Ba, Algorithm 1, in the order fixed by include/z3.h.
__device__ __forceinline__ void adam1(float g, float &p, float &m, float &v, const AdamK &k) {
    const float m1 = __fadd_rn(__fmul_rn(k.b1, m), __fmul_rn(k.c1, g));
    const float v1 = __fadd_rn(__fmul_rn(k.b2, v), __fmul_rn(k.c2, __fmul_rn(g, g)));
    const float mh = __fmul_rn(m1, k.rb1);
    const float vh = __fmul_rn(v1, k.rb2);
    const float u = __fdiv_rn(mh, __fadd_rn(__fsqrt_rn(vh), k.eps));
    const float pd = __fsub_rn(p, __fmul_rn(k.lwd, p));
    p = __fsub_rn(pd, __fmul_rn(k.lr, u));
    m = m1;
    v = v1;
}

// Maps blockIdx.x to (table entry, rank, tile within the chunk).
struct TileRef {
    int p;
    int64_t r;
    int64_t t;
};

// The tiles of one launch number at most 2^31 - 1 (the layout starts a new
// launch table before that), and every entry has at least one tile per
// chunk, so the tile arithmetic fits unsigned 32 bits.  DIV32 divides by the
// tiles per chunk in 32 bits instead of an emulated 64-bit division: the
// copy kernels take it (their few instructions per element make the
// division a large share); the reduce kernels keep the 64-bit form, with
// which their fused modes fit 64 registers without spilling.
template <bool DIV32>
__device__ __forceinline__ TileRef locate(const Tab &tab, uint32_t g) {
    int lo = 0, hi = tab.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((uint32_t)tab.e[mid].tile0 <= g) lo = mid; else hi = mid - 1;
    }
    if constexpr (DIV32) {
        const uint32_t local = g - (uint32_t)tab.e[lo].tile0;
        const uint32_t tpc = (uint32_t)tab.e[lo].tpc;
        const uint32_t r = local / tpc;
        return TileRef{lo, (int64_t)r, (int64_t)(local - r * tpc)};
    } else {
        const int64_t local = (int64_t)g - tab.e[lo].tile0;
        const int64_t tpc = tab.e[lo].tpc;
        const int64_t r = local / tpc;
        return TileRef{lo, r, local - r * tpc};
    }
}

// Programmatic dependent launch.  Every kernel is launched so that it may
// start while the previous kernel of the stream (its primary) still runs.
// A thread first waits for the primary to complete -- memory included -- and
// only then lets the next kernel launch.  Because every kernel waits before
// it releases its dependent, a kernel that has started knows that everything
// enqueued before its primary has completed: only the primary may still be
// running.  So:
//   - a plain kernel waits before its first global memory access, and the
//     ordering between calls is exactly stream order;
//   - an EARLY variant (used only where the library itself enqueued the
//     primary, inside one call) may, before it waits, read buffers that the
//     primary does not write; it waits before its first store.  Its first
//     loads overlap the primary's tail.
// Without the launch attribute both instructions are no-ops.
__device__ __forceinline__ void pdl_enter() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Ranks whose 16-byte loads are issued together before they are folded.
constexpr int kRankBatch = 8;

__device__ __forceinline__ void ld8f(const float *p, float f[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    const float4 b = *reinterpret_cast<const float4 *>(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__device__ __forceinline__ void st8f(float *p, const float f[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

// The rank fold of one aligned shard vector: g[l] = scale * sum over k of the
// bf16 gradients grads[k][x0 + delta + l], l = 0..7, in ascending rank order
// from rank 0's value (8 ranks' 16-byte loads in flight per batch).
template <int PHI>
__device__ __forceinline__ void fold_vector(const uint16_t *grads, int64_t stride, float scale,
                                            int n_ranks, int64_t x0, int64_t delta, float g[8]) {
    const uint16_t *gp = grads + (x0 + delta - PHI);
    // a shifted window needs two 16-byte loads per rank: half the batch
    constexpr int RB = PHI == 0 ? kRankBatch : kRankBatch / 2;
    float acc[8];
    for (int k0 = 0; k0 < n_ranks; k0 += RB) {
        uint4 lo[RB], hi[RB];
#pragma unroll
        for (int u = 0; u < RB; ++u) {
            if (k0 + u < n_ranks) {
                const uint16_t *rp = gp + (int64_t)(k0 + u) * stride;
                lo[u] = ld8b(rp);
                hi[u] = PHI ? ld8b(rp + kVec) : lo[u];
            }
        }
#pragma unroll
        for (int u = 0; u < RB; ++u) {
            if (k0 + u < n_ranks) {
                float f[8];
                unpack8(window8<PHI>(lo[u], hi[u]), f);
                if (k0 + u == 0) {
#pragma unroll
                    for (int l = 0; l < 8; ++l) acc[l] = f[l];
                } else {
#pragma unroll
                    for (int l = 0; l < 8; ++l) acc[l] = __fadd_rn(acc[l], f[l]);
                }
            }
        }
    }
#pragma unroll
    for (int l = 0; l < 8; ++l) g[l] = __fmul_rn(acc[l], scale);
}

// The same fold of the one element at shard position x.
__device__ __forceinline__ float fold_element(const uint16_t *grads, int64_t stride, float scale,
                                              int n_ranks, int64_t x, int64_t delta) {
    const uint16_t *gp = grads + (x + delta);
    float s = bf16_to_f32(gp[0]);
    for (int k = 1; k < n_ranks; ++k) s = __fadd_rn(s, bf16_to_f32(gp[(int64_t)k * stride]));
    return __fmul_rn(s, scale);
}

// The eight bf16 roundings of p as one 16-byte vector.
__device__ __forceinline__ uint4 pack8(const float p[8]) {
    uint4 b;
    b.x = pack_bf16x2(p[0], p[1]);
    b.y = pack_bf16x2(p[2], p[3]);
    b.z = pack_bf16x2(p[4], p[5]);
    b.w = pack_bf16x2(p[6], p[7]);
    return b;
}

// Launches a kernel with programmatic stream serialisation allowed.
template <typename... KArgs, typename... Args>
void launch(void (*kernel)(KArgs...), int64_t grid, int block, cudaStream_t stream,
            Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    (void)cudaLaunchKernelEx(&cfg, kernel, args...);  // errors: cudaGetLastError below
}

}  // namespace z3
