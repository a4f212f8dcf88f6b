// entry.h -- what the C entry points share: pointer checks and the NVTX range
// around a call.
#pragma once

#include <stdint.h>

#include <initializer_list>

#include <nvtx3/nvToolsExt.h>

#include "llsa.h"

namespace llsa {

inline bool aligned(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

inline int check_ptrs(std::initializer_list<const void*> ptrs) {
    for (const void* q : ptrs) {
        if (!q) return LLSA_ERR_INVALID_ARG;
        if (!aligned(q)) return LLSA_ERR_ALIGN;
    }
    return LLSA_OK;
}

// An NVTX range around a C-ABI call (the call's name), so a profiler timeline
// shows each library call with the kernels it enqueued.
struct CallRange {
    explicit CallRange(const char* name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
};

}  // namespace llsa
