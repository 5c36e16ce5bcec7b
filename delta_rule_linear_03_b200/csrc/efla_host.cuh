// efla_host.cuh - host helpers shared by the library's translation units:
// argument checks, NVTX ranges, the SM count.
#pragma once
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "../../include/efla.h"

namespace efla {
namespace host {

constexpr long long kMaxElems = (1LL << 46);  // sanity bound on any tensor's element count

// NVTX range around one C-ABI call (validation and launches), so a profiler
// timeline shows which library call enqueued which kernels.  Header-only
// NVTX: without an attached tool a push or pop is a test of a null pointer.
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

inline bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned16(const void *p) { return aligned_to(p, 16); }

inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

inline size_t esize(efla_dtype_t dt) { return dt == EFLA_F32 ? 4 : 2; }

inline bool known_dtype(efla_dtype_t dt) { return dt == EFLA_F32 || dt == EFLA_BF16; }

inline efla_status_t launched() { return cudaGetLastError() == cudaSuccess ? EFLA_OK : EFLA_ERR_CUDA; }

inline int num_sms() {
    static std::atomic<int> cached[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if ((n = cached[dev & 63].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    cached[dev & 63].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace host
}  // namespace efla
