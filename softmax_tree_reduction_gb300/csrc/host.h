// Host-side helpers that api.cu shares with the other entry points' files:
// the device's set-up and the cache layout checks.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/tree_attn.h"

namespace ta {

struct DeviceInfo {
    int device;
    int num_sms;
    int* err;  // device address of the error word
};

// The current device's set-up (done on first use).  TA_OK or a negative status.
int device_info(DeviceInfo* out);

struct CacheLayout {
    int64_t stride_b, stride_h, stride_t;  // elements; stride_b is between pages for a pool
    int elem_bytes;
    int page_shift;                        // log2(page_size), 0 for dense caches
};

// Validate a cache's shape (and its pages, when given) and resolve its strides.
int cache_layout(const ta_shape* shape, const ta_paged_kv* paged, CacheLayout* out);

// A 4-bit cache's strides in bytes and the bytes up to the end of its last vector.
struct Int4Layout {
    int64_t code_b, code_h, code_t, step_b, step_h, step_t;
    size_t code_bytes, step_bytes;
    int page_shift;
};

// Validate a 4-bit cache and its shape, and resolve its strides.
int int4_layout(const ta_shape* shape, const ta_paged_kv* paged, const ta_int4_kv* cache, Int4Layout* out);

inline bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Launch attribute: the grid may start while the previous one on the stream
// ends (every kernel launched with it waits before it touches memory).
inline cudaLaunchAttribute programmatic_launch() {
    cudaLaunchAttribute a = {};
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    return a;
}

}  // namespace ta
