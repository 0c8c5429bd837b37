// host.hpp -- what the host side of every entry point shares: type and
// alignment checks, and the workspace of one call.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "igc.h"

namespace igc {

inline bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }
inline bool valid_type(igc_out_t t) { return t == IGC_OUT_F32 || t == IGC_OUT_BF16 || t == IGC_OUT_F16; }
inline int out_size(igc_out_t t) { return t == IGC_OUT_F32 ? 4 : 2; }
inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
// A launch has fewer than 2^32 threads.
inline bool launchable(int64_t blocks, int64_t threads) { return blocks <= 0x7fffffff && blocks * threads < (1ll << 32); }

// igc_lib.hip: the library's pool, and whether a stream is being captured into a graph.
void* workspace_alloc(size_t bytes, hipStream_t stream);
bool capturing(hipStream_t stream);

// The workspace of one call: the caller's where one is given, otherwise (when
// `bytes` > 0) taken stream-ordered from the library's pool and given back when
// this object goes, after the call's work is enqueued.
struct Workspace {
    void* ptr = nullptr;
    bool owned = false;
    hipStream_t stream = nullptr;

    igc_status_t take(int64_t bytes, void* user, int64_t user_bytes, hipStream_t st) {
        if (user && (user_bytes < bytes || (reinterpret_cast<uintptr_t>(user) & 255u))) return IGC_ERR_INVALID_VALUE;
        ptr = user;
        stream = st;
        if (user || bytes <= 0) return IGC_OK;
        if (capturing(st)) return IGC_ERR_UNSUPPORTED;
        ptr = workspace_alloc((size_t)bytes, st);
        owned = ptr != nullptr;
        return ptr ? IGC_OK : IGC_ERR_HIP;
    }
    Workspace() = default;
    Workspace(const Workspace&) = delete;
    Workspace& operator=(const Workspace&) = delete;
    ~Workspace() {
        if (owned) (void)hipFreeAsync(ptr, stream);
    }
};

}  // namespace igc
