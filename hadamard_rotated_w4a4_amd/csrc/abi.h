// Host-side helpers shared by the files that implement the C ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>

#include "w4a4.h"

namespace w4a4 {

inline thread_local char g_last_hip_error[256] = "";

inline w4a4_status hip_status(const char *what) {
    const hipError_t err = hipGetLastError();
    if (err == hipSuccess) return W4A4_OK;
    std::snprintf(g_last_hip_error, sizeof g_last_hip_error, "%s: %s", what, hipGetErrorString(err));
    return W4A4_ERR_HIP;
}

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }
inline unsigned blocks_for(int64_t work, int per) { return (unsigned)((work + per - 1) / per); }
inline size_t up256_bytes(int64_t b) { return (size_t)((b + 255) / 256 * 256); }

// Size bounds, so that every launch fits the hardware's grid limits and the
// kernels' 32-bit offsets: rows (m, or routed rows) within 65535 row tiles of
// 32 (the quantisers' grid.y); K and N well past any model's.  A 1-D launch
// must stay below 2^32 threads in all.
constexpr int64_t kMaxGridY = 65535;
constexpr int64_t kMaxRows = kMaxGridY * 32;
constexpr int64_t kMaxK = int64_t{1} << 24;
constexpr int64_t kMaxN = int64_t{1} << 26;
constexpr int64_t kMaxThreads = (int64_t{1} << 32) - 1;
inline bool grid_fits(int64_t threads) { return threads <= kMaxThreads; }
// m rows, n columns, k: inside the bounds above (sizes already known >= 0)
inline bool within_bounds(int64_t m, int64_t n, int64_t k) { return m <= kMaxRows && n <= kMaxN && k <= kMaxK; }

}  // namespace w4a4
