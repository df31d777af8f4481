// linear_check.h -- argument checks, workspaces and launches shared by the
// checkpoint calls (act8.hip), the layer products (linear.hip) and the norms
// (norm.hip).  Host code only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "product_shape.h"
#include "tide.h"

namespace tide {

// Limits of the kernels' 32-bit arithmetic: a workgroup addresses at most 256
// rows from a 64-bit base, so 256 rows of bf16 have to stay within 2^31
// bytes; rows are counted in 31 bits, a grid's threads in 32.  Within these
// limits no launch of a call is refused for its grid, so that none is refused
// after the ones before it have run.
constexpr int64_t kMaxWidth = (int64_t)1 << 22;
constexpr int64_t kMaxThreads = UINT32_MAX;         // of a grid
constexpr int64_t kMaxRows = INT32_MAX;             // of a checkpoint
constexpr int64_t kMaxKept = (int64_t)1 << 36;      // its values (a lane packs 32 of them)
constexpr int64_t kMaxTokens = (int64_t)1 << 30;    // of a product (128 a workgroup of 256)
constexpr int64_t kMaxElements = (int64_t)1 << 33;  // of a product's matrices

// The bytes of a matrix: rows of `width` bytes, `pitch` apart.
struct Extent {
    uint64_t lo = 0, hi = 0, pitch = 0, width = 0;
};

inline Extent rows_extent(const void* p, int64_t ld, int64_t rows, int64_t cols,
                          int64_t elem_bytes = 2) {
    Extent e;
    if (!p || rows <= 0 || cols <= 0) return e;
    e.lo = reinterpret_cast<uintptr_t>(p);
    e.pitch = (uint64_t)(ld * elem_bytes);
    e.width = (uint64_t)(cols * elem_bytes);
    e.hi = e.lo + (uint64_t)(rows - 1) * e.pitch + e.width;
    return e;
}
inline Extent bytes_extent(const void* p, int64_t bytes) {
    return rows_extent(p, bytes, 1, bytes, 1);
}

// Whether two matrices share a byte.  Column ranges of one buffer (the same
// pitch) lie between each other without sharing any; otherwise interleaved
// rows count as sharing.
inline bool overlaps(const Extent& a, const Extent& b) {
    if (a.lo == a.hi || b.lo == b.hi || a.hi <= b.lo || b.hi <= a.lo) return false;
    if (a.pitch == b.pitch && a.pitch > 0) {
        const uint64_t d = (b.lo % a.pitch + a.pitch - a.lo % a.pitch) % a.pitch;
        if (d >= a.width && d + b.width <= a.pitch) return false;
    }
    return true;
}

// A matrix of bf16 rows: there, element-aligned, rows that do not run into
// each other, a row distance that the kernels can address.
inline tide_status check_rows(const void* p, int64_t ld, int64_t rows, int64_t cols) {
    if (rows == 0 || cols == 0) return TIDE_OK;
    if (!p || (rows > 1 && ld < cols)) return TIDE_EINVAL;
    if (rows > 1 && ld > kMaxWidth) return TIDE_EUNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(p) % 2) return TIDE_EALIGN;
    return TIDE_OK;
}

// The stream belongs to the current device (the null stream does).
inline tide_status check_stream_device(tide_stream_t stream) {
    if (!stream) return TIDE_OK;
    int dev = 0;
    hipDevice_t sdev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return TIDE_EHIP;
    if (hipStreamGetDevice(reinterpret_cast<hipStream_t>(stream), &sdev) != hipSuccess)
        return TIDE_EHIP;
    return sdev == dev ? TIDE_OK : TIDE_EINVAL;
}

inline tide_status check_kept(const void* p, int64_t rows, int64_t cols) {
    if (rows == 0 || cols == 0) return TIDE_OK;
    if (!p) return TIDE_EINVAL;
    return reinterpret_cast<uintptr_t>(p) % 16 ? TIDE_EALIGN : TIDE_OK;
}

// No output shares a byte with an input or another output.
inline tide_status check_apart(const Extent* in, int n_in, const Extent* out, int n_out) {
    for (int a = 0; a < n_out; ++a) {
        for (int b = 0; b < n_in; ++b)
            if (overlaps(out[a], in[b])) return TIDE_EOVERLAP;
        for (int b = 0; b < a; ++b)
            if (overlaps(out[a], out[b])) return TIDE_EOVERLAP;
    }
    return TIDE_OK;
}

inline tide_status check_workspace(void* ws, size_t have, int64_t need, const Extent* other, int n) {
    if (need == 0) return TIDE_OK;
    if (!ws || have < (size_t)need) return TIDE_ENOSPACE;
    if (reinterpret_cast<uintptr_t>(ws) % 16) return TIDE_EALIGN;
    const Extent e = bytes_extent(ws, need);
    for (int k = 0; k < n; ++k)
        if (overlaps(e, other[k])) return TIDE_EOVERLAP;
    return TIDE_OK;
}

#define TIDE_TRY(call)                                \
    do {                                              \
        const tide_status try_st = (call);            \
        if (try_st != TIDE_OK) return try_st;         \
    } while (0)

// The workspace's pieces, handed out in order, each on 256 bytes.
struct Carver {
    char* base;
    int64_t used = 0;
    template <typename T>
    T* take(int64_t count) {
        T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
        used += round_up(count * (int64_t)sizeof(T), 256);
        return p;
    }
};

template <typename... P, typename... A>
tide_status launch_lds(void (*kernel)(P...), int64_t grid, int threads, unsigned lds_bytes,
                       tide_stream_t stream, A... a) {
    if (grid <= 0) return TIDE_OK;
    if (grid > kMaxThreads / threads) return TIDE_EUNSUPPORTED;
    void* args[] = {&a...};
    static_assert(sizeof...(P) == sizeof...(A), "one argument for each parameter");
    static_assert((__is_same(P, A) && ...), "arguments of the parameters' own types");
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3((unsigned)grid),
                           dim3((unsigned)threads), args, lds_bytes,
                           reinterpret_cast<hipStream_t>(stream)) == hipSuccess
               ? TIDE_OK
               : TIDE_EHIP;
}
template <typename... P, typename... A>
tide_status launch(void (*kernel)(P...), int64_t grid, int threads, tide_stream_t stream, A... a) {
    return launch_lds(kernel, grid, threads, 0, stream, a...);
}

// tide_act8_unpack without its checks; once: x is not read again soon, so it
// needs no place in the caches.
tide_status act8_unpack_into(const void* kept, int64_t rows, int64_t cols, void* x, int64_t ldx,
                             bool once, tide_stream_t stream);

}  // namespace tide
