// host.hpp -- what the host sides of the routed, grouped and layer operators
// share: checks of pointers and sizes, the compute-unit count, the workspace.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "gemm_coll.h"

namespace gc {
namespace host {

constexpr int kMaxDevices = 64;
inline std::atomic<int> g_cus[kMaxDevices];      // 0 = not queried yet

inline int cu_count(int &cus)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess)
        return GC_EIO;
    cus = dev < kMaxDevices ? g_cus[dev].load(std::memory_order_relaxed) : 0;
    if (cus == 0) {
        if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
            cus <= 0)
            return GC_EIO;
        if (dev < kMaxDevices)
            g_cus[dev].store(cus, std::memory_order_relaxed);
    }
    return GC_OK;
}

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool good16(const void *p) { return p && aligned(p, 16); }
inline bool good4(const void *p) { return p && aligned(p, 4); }

// Buffers are addressed through 32-bit byte offsets with an out-of-range
// sentinel at 2^31.
inline bool fits(int64_t rows, int64_t cols) { return cols == 0 || rows < ((int64_t)1 << 30) / cols; }

// Rows of weights past K are addressed too, and must read as zeros: up to 31
// rows past the buffer (127 for the adapters' up) the offset stays in 32 bits.
constexpr int64_t kMaxCols = (int64_t)1 << 24;

// Workspace: counters (4 KiB, zero between launches), then room for one of
// the partial tiles of the streaming kernel (two of at most kPartBytes per
// workgroup), the fp32 sums of products split along K, the counts of a
// many-block grouping, or lora_add's middle sums.
constexpr int64_t kCountBytes = 4096;
constexpr int64_t kPartBytes = 32768;
constexpr int64_t kSumBytes = (int64_t)64 << 20;
constexpr int kMaxWorkers = (int)(kCountBytes / 4);

inline int workers(int cus) { return std::min(cus, kMaxWorkers); }
inline int64_t base_bytes(int cus) { return kCountBytes + std::max(kSumBytes, 2 * kPartBytes * workers(cus)); }

inline int launched() { return hipGetLastError() == hipSuccess ? GC_OK : GC_EIO; }

}  // namespace host
}  // namespace gc
