// Argument checks shared by the C ABI entry points (api.cu, layer_api.cu):
// device pointers, overlapping regions and the caller's workspace.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "kda_internal.h"

namespace kda {

// A pointer the kernels may dereference: device (or managed) memory of the
// current device `dev`, 16-byte aligned.
inline bool device_ptr_ok(const void* p, int dev)
{
    if (!p) return false;
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
    cudaPointerAttributes attr;
    if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
        cudaGetLastError();  // clear the sticky-free error state
        return false;
    }
    if (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged) return false;
    return attr.type == cudaMemoryTypeManaged || attr.device == dev;
}

inline bool device_ptr_ok(const void* p)
{
    int dev = -1;
    return p && cudaGetDevice(&dev) == cudaSuccess && device_ptr_ok(p, dev);
}

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb)
{
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}

inline size_t elem_size(kda_dtype d) { return d == KDA_DTYPE_BF16 ? 2 : 4; }

struct Region {
    const void* p;
    size_t n;
};

// The caller's workspace for a call that needs `need` bytes: device memory of
// the current device, 256-byte aligned, large enough, overlapping none of the
// call's tensors.  A call that needs none ignores it.
inline bool workspace_ok(const void* ws, size_t ws_bytes, size_t need, const Region* r, int nr)
{
    if (need == 0) return true;
    if (!ws || ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % 256 != 0) return false;
    if (!device_ptr_ok(ws)) return false;
    for (int i = 0; i < nr; ++i)
        if (overlaps(ws, need, r[i].p, r[i].n)) return false;
    return true;
}

}  // namespace kda
