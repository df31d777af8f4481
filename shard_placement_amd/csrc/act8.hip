// act8.hip -- activations kept in 8 bits (format: act8.h), for gfx950.
//
// Pack reads a bf16 matrix once and writes its e4m3 values and block scales;
// unpack is the way back.  Both are bound by memory: 3 bytes and 1/32 for an
// element and a handful of operations.  A lane owns 8 consecutive columns
// (one 16-byte access on the bf16 side, one 8-byte access on the other, both
// contiguous over the wave), so the 4 lanes of a quad hold a block and its
// maximum takes two lane exchanges.  Rows are cut into units of 8 columns and
// the units of all rows dealt out in order, so that narrow and wide matrices
// fill the chip alike.  Nontemporal accesses measured (8192 x 8192): pack 35.4
// us with both, 40.0 with the loads only, 38.2 with the stores only, 43.8 with
// none; unpack 30.0 with the stores only, 36.0 with both, 39.6 with none.
#include <hip/hip_runtime.h>

#include "act8.h"
#include "bf16_io.h"
#include "linear_check.h"
#include "tide.h"

using namespace tide;

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;  // units of 8 columns for each lane
constexpr int64_t kUnitsPerGroup = (int64_t)kThreads * kUnits;

// The row and the unit in it of the workgroup's k-th unit for this lane.
struct UnitAt {
    int64_t row;
    int32_t unit;
};
__device__ __forceinline__ UnitAt unit_at(int64_t row0, uint32_t unit0, uint32_t per_row, int k) {
    const uint32_t n = unit0 + threadIdx.x + (uint32_t)k * kThreads;
    const uint32_t r = n / per_row;
    return {row0 + r, (int32_t)(n - r * per_row)};
}

__global__ __launch_bounds__(kThreads) void pack_kernel(const uint16_t* x, int64_t ldx,
                                                        int64_t rows, int64_t cols,
                                                        uint32_t per_row, uint8_t* out) {
    const int64_t first = (int64_t)blockIdx.x * kUnitsPerGroup;
    const int64_t row0 = first / per_row;
    const uint32_t unit0 = (uint32_t)(first - row0 * per_row);
    uint8_t* scales = out + act8_scale_offset(rows, cols);
    u32x4v w[kUnits];
    UnitAt at[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        at[k] = unit_at(row0, unit0, per_row, k);
        const int64_t c = (int64_t)at[k].unit * 8;
        w[k] = 0;
        if (at[k].row < rows && c + 8 <= cols) w[k] = load8_raw<true>(x + at[k].row * ldx + c);
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const int64_t c = (int64_t)at[k].unit * 8;
        float v[8];
        widen(w[k], v);
        if (at[k].row < rows && c < cols && c + 8 > cols)
            load8(x + at[k].row * ldx + c, cols - c, v);
        act8_u32x2 q;
        const int e = act8_pack8(v, &q);
        if (at[k].row >= rows) continue;
        const int64_t u = at[k].row * per_row + at[k].unit;
        __builtin_nontemporal_store(q, (TIDE_GLOBAL_AS u32x2*)(out + u * 8));
        if ((at[k].unit & 3) == 0) *(TIDE_GLOBAL_AS uint8_t*)(scales + u / 4) = (uint8_t)(e + 127);
    }
}

// ONCE: x is not read again soon.
template <bool ONCE>
__global__ __launch_bounds__(kThreads) void unpack_kernel(const uint8_t* in, int64_t rows,
                                                          int64_t cols, uint32_t per_row,
                                                          uint16_t* x, int64_t ldx) {
    const int64_t first = (int64_t)blockIdx.x * kUnitsPerGroup;
    const int64_t row0 = first / per_row;
    const uint32_t unit0 = (uint32_t)(first - row0 * per_row);
    const uint8_t* scales = in + act8_scale_offset(rows, cols);
    u32x2 q[kUnits];
    uint8_t s[kUnits];
    UnitAt at[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        at[k] = unit_at(row0, unit0, per_row, k);
        q[k] = 0;
        s[k] = 0;
        if (at[k].row >= rows) continue;
        const int64_t u = at[k].row * per_row + at[k].unit;
        q[k] = *(const TIDE_GLOBAL_AS u32x2*)(in + u * 8);
        s[k] = *(const TIDE_GLOBAL_AS uint8_t*)(scales + u / 4);
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        if (at[k].row >= rows) continue;
        const int64_t c = (int64_t)at[k].unit * 8;
        float v[8];
        act8_unpack8(q[k], act8_scale(s[k]), v);
        store8<ONCE>(x + at[k].row * ldx + c, cols - c, v);
    }
}

// Rows and columns of a checkpoint that the kernels can address: a row's
// units and a workgroup's units together stay below 2^31, a grid's threads
// below 2^32.
tide_status check_shape(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return TIDE_EINVAL;
    if (rows > kMaxRows || cols > kMaxWidth) return TIDE_EUNSUPPORTED;
    if (rows * act8_pitch(cols) > kMaxKept) return TIDE_EUNSUPPORTED;
    return TIDE_OK;
}

}  // namespace

extern "C" tide_status tide_act8_bytes(int64_t rows, int64_t cols, size_t* bytes) {
    if (!bytes) return TIDE_EINVAL;
    const tide_status st = check_shape(rows, cols);
    if (st != TIDE_OK) return st;
    *bytes = (size_t)act8_bytes(rows, cols);
    return TIDE_OK;
}

namespace {

// The checks of both directions; x is the bf16 side.
tide_status check_call(const void* x, int64_t ldx, const void* kept, int64_t rows, int64_t cols,
                       tide_stream_t stream) {
    tide_status st = check_shape(rows, cols);
    if (st != TIDE_OK) return st;
    if (rows == 0 || cols == 0) return TIDE_OK;
    st = check_rows(x, ldx, rows, cols);
    if (st != TIDE_OK) return st;
    if (!kept) return TIDE_EINVAL;
    if (reinterpret_cast<uintptr_t>(kept) % 16) return TIDE_EALIGN;
    if (overlaps(rows_extent(x, ldx, rows, cols),
                 bytes_extent(kept, act8_bytes(rows, cols)))) return TIDE_EOVERLAP;
    return check_stream_device(stream);
}

}  // namespace

extern "C" tide_status tide_act8_pack(const void* x, int64_t ldx, int64_t rows, int64_t cols,
                                      void* kept, tide_stream_t stream) {
    const tide_status st = check_call(x, ldx, kept, rows, cols, stream);
    if (st != TIDE_OK || rows == 0 || cols == 0) return st;
    const int64_t per_row = act8_pitch(cols) / 8;
    return launch(pack_kernel, (rows * per_row + kUnitsPerGroup - 1) / kUnitsPerGroup, kThreads,
                  stream, static_cast<const uint16_t*>(x), ldx, rows, cols, (uint32_t)per_row,
                  static_cast<uint8_t*>(kept));
}

tide_status tide::act8_unpack_into(const void* kept, int64_t rows, int64_t cols, void* x,
                                   int64_t ldx, bool once, tide_stream_t stream) {
    if (rows == 0 || cols == 0) return TIDE_OK;
    const int64_t per_row = act8_pitch(cols) / 8;
    return launch(once ? unpack_kernel<true> : unpack_kernel<false>,
                  (rows * per_row + kUnitsPerGroup - 1) / kUnitsPerGroup, kThreads, stream,
                  static_cast<const uint8_t*>(kept), rows, cols, (uint32_t)per_row,
                  static_cast<uint16_t*>(x), ldx);
}

extern "C" tide_status tide_act8_unpack(const void* kept, int64_t rows, int64_t cols, void* x,
                                        int64_t ldx, tide_stream_t stream) {
    const tide_status st = check_call(x, ldx, kept, rows, cols, stream);
    return st == TIDE_OK ? act8_unpack_into(kept, rows, cols, x, ldx, true, stream) : st;
}
