// z3_check.h -- what the C-ABI entry points (z3_api.cpp, z3_head_api.cpp) share:
// buffer checks, launch-error reporting and NVTX ranges.  Not part of the
// public ABI.
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstdint>
#include <string>

#include "z3_internal.h"

namespace z3 {

struct Buf {
    const void *ptr;
    int64_t bytes;
    const char *name;
};

inline z3_status check_bufs(const char *fn, const Buf *bufs, int n) {
    for (int i = 0; i < n; ++i) {
        if (bufs[i].bytes == 0) continue;
        if (bufs[i].ptr == nullptr)
            return fail(Z3_ERR_INVALID_ARG, std::string(fn) + ": " + bufs[i].name + " is NULL");
        if (reinterpret_cast<uintptr_t>(bufs[i].ptr) % 16 != 0)
            return fail(Z3_ERR_ALIGNMENT,
                        std::string(fn) + ": " + bufs[i].name + " is not 16-byte aligned");
    }
    for (int i = 0; i < n; ++i) {
        for (int j = i + 1; j < n; ++j) {
            if (bufs[i].bytes == 0 || bufs[j].bytes == 0) continue;
            const uintptr_t a0 = reinterpret_cast<uintptr_t>(bufs[i].ptr);
            const uintptr_t b0 = reinterpret_cast<uintptr_t>(bufs[j].ptr);
            if (a0 < b0 + (uintptr_t)bufs[j].bytes && b0 < a0 + (uintptr_t)bufs[i].bytes)
                return fail(Z3_ERR_INVALID_ARG, std::string(fn) + ": " + bufs[i].name +
                                                    " overlaps " + bufs[j].name);
        }
    }
    return Z3_OK;
}

inline z3_status launched(const char *fn, cudaError_t err) {
    if (err != cudaSuccess)
        return fail(Z3_ERR_CUDA, std::string(fn) + ": " + cudaGetErrorString(err));
    return Z3_OK;
}

// Host-side NVTX range around the launches of one call, named after the
// collective it enqueues, so a trace shows the AllGather / ReduceScatter /
// update pattern of "The ZeRO-3 Diagram Most People Remember Is Wrong", s.6.
struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
    Range(const Range &) = delete;
    Range &operator=(const Range &) = delete;
};

}  // namespace z3
