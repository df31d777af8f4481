// norm.hip -- rms and layer norm of a matrix's rows, with the 8-bit checkpoints
// of its input and output, and their gradients, for gfx950.
//
//   forward   n = (x - mu) r, y = n w + b; mu the row's mean (rms: 0),
//             r = 1 / sqrt(mean of (x - mu)^2 + eps)
//   backward  c = dy w, dx = r (c - mean(c) - n mean(c n)) + add (rms: without
//             mean(c)); dw = the sum of dy n over the rows, db = the sum of dy
//
// w is a full tensor as the all-gather placement writes it, dw and db are
// gradients as the reduce-scatter reads them.
//
// Memory bounds both directions: a row is read once, kept in registers as it
// lies in memory, and its statistics and results are worked out from there.
// 8192 x 8192 with rms: forward 46.4 us (5.8 TB/s), with both checkpoints 66.4 (6.1),
// backward from a checkpoint and onto a stream's gradient 80.0 (5.9); few rows are
// bound by launches (1 x 8192 forward 2.5 us) and by the second one backward.
// The backward pass works mu and r out again from x (or from its checkpoint)
// instead of keeping them: the row is in registers anyway.
//
// A row belongs to a group of lanes: 16 or 64 lanes of a wave for narrow rows, a
// workgroup of as many waves as hold it for wide ones (up to L lanes); a lane owns
// U units of 8 consecutive columns, the group's lanes apart, so every access is
// contiguous over the wave and the 4 lanes of a quad hold a checkpoint block.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "act8.h"
#include "bf16_io.h"
#include "linear_check.h"
#include "tide.h"

using namespace tide;

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) float lds_float;

constexpr int kThreads = 256;  // of a workgroup whose rows take fewer lanes

// ---- sums over a row's lanes -------------------------------------------------

template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float add_dpp(float v) {
    const int moved = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, ROWS == 0xf);
    return v + __builtin_bit_cast(float, moved);
}

// The sum over N <= 16 consecutive lanes, in all of them: pairs, pairs of pairs,
// then the mirrored half and the mirrored whole.
template <int N>
__device__ __forceinline__ float sum_lanes(float v) {
    v = add_dpp<0xB1>(v);
    v = add_dpp<0x4E>(v);
    if constexpr (N >= 8) v = add_dpp<0x141>(v);
    if constexpr (N >= 16) v = add_dpp<0x140>(v);
    return v;
}
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
// The sum over the wave, in its last lane: rows 1 and 3 take the sums of rows 0
// and 2, then rows 2 and 3 that of the first half.
__device__ __forceinline__ float sum64(float v) {
    v = sum_lanes<16>(v);
    v = add_dpp<0x142, 0xa>(v);
    return add_dpp<0x143, 0xc>(v);
}

// Every wave's LDS accesses before it are done.  (__syncthreads() would wait for
// the loads from memory too, the next row's among them: 2% of 8192 rows of 5120
// with layer norm.)
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// N sums over the L lanes of a row, in all of them, always added in the same
// order.  L > 64: `box` holds N * L / 64 floats that no wave still reads.
template <int L, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], lds_float* box) {
    if constexpr (L == 16) {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = sum_lanes<16>(v[k]);
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = sum64(v[k]);
    }
    if constexpr (L == 64) {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = lane_value(v[k], 63);
    }
    if constexpr (L > 64) {
        constexpr int kWaves = L / 64;
        if ((threadIdx.x & 63) == 63) {
#pragma unroll
            for (int k = 0; k < N; ++k) box[k * kWaves + (threadIdx.x >> 6)] = v[k];
        }
        lds_barrier();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t w = threadIdx.x & (kWaves - 1);
            v[k] = sum_lanes<kWaves>(w < blockDim.x / 64 ? box[k * kWaves + w] : 0.0f);
        }
    }
}

// ---- a lane's part of a row --------------------------------------------------

// The columns of a lane's unit u of L lanes, and how many of them exist.
template <int L>
__device__ __forceinline__ uint32_t column(int u, uint32_t thread) {
    if constexpr (L > 64) return (thread + (uint32_t)u * blockDim.x) * 8;
    return (thread % L + (uint32_t)u * L) * 8;
}

// The thread's number, to work out columns from where they are used: kept
// through the loop over rows, they and what is worked out from them take a
// third of the registers.
__device__ __forceinline__ uint32_t this_thread() {
    uint32_t t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

// Eight elements of which the first `less` are dropped, zeros moving in.
__device__ __forceinline__ u32x4v drop(u32x4v w, uint32_t less) {
    if (less & 4) w = u32x4v{w.z, w.w, 0u, 0u};
    if (less & 2) w = u32x4v{w.y, w.z, w.w, 0u};
    if (less & 1)
        w = u32x4v{w.x >> 16 | w.y << 16, w.y >> 16 | w.z << 16, w.z >> 16 | w.w << 16, w.w >> 16};
    return w;
}

// Eight elements from column c of a row of `cols`, as far as loading goes: every
// lane loads, where its eight columns pass the row's end the row's last eight,
// and settle() makes them its own with zeros behind, where they are used: here it
// would wait for them.  (Loading the elements before the end one by one, a wait
// for each, took 2 of 7 us for 4099 x 1001.)  ONCE: the row is read once.
template <bool ONCE = false>
__device__ __forceinline__ u32x4v load_unit(const uint16_t* row, uint32_t c, uint32_t cols) {
    if (cols >= 8) return load8_raw<ONCE>(row + min(c, cols - 8));
    u32x4v w = 0;
#pragma unroll
    for (int k = 0; k < 7; ++k)
        if (c + k < cols)
            w[k / 2] |= (uint32_t) * (const TIDE_GLOBAL_AS uint16_t*)(row + c + k) << (k % 2 * 16);
    return w;
}
__device__ __forceinline__ void settle(u32x4v& w, uint32_t c, uint32_t cols) {
    if (cols >= 8 && c + 8 > cols) w = c < cols ? drop(w, c + 8 - cols) : (u32x4v)0u;
}
// Of all of a lane's units.
template <int L, int U>
__device__ __forceinline__ void settle(u32x4v (&w)[U], uint32_t thread, uint32_t cols) {
#pragma unroll
    for (int u = 0; u < U; ++u) settle(w[u], column<L>(u, thread), cols);
}

// The units as they lie in memory are what stays in registers between the
// passes over a row: without this the compiler keeps their widened elements,
// twice the registers, which only lanes of one unit have.
template <int U>
__device__ __forceinline__ void forget(u32x4v (&w)[U]) {
    if constexpr (U > 1) {
#pragma unroll
        for (int u = 0; u < U; ++u) asm volatile("" : "+v"(w[u]));
    }
}

// v - mu where the element exists, else 0 (v is 0 there).  (A branch over several
// units keeps them all in registers.)
template <int U>
__device__ __forceinline__ void centre(float (&v)[8], float mu, uint32_t c, uint32_t cols) {
    mu = c < cols ? mu : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] -= mu;
    if (U > 4 || cols % 8) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = (int32_t)(cols - c) > k ? v[k] : 0.0f;
    }
}

// Layer norm takes off the mean's first 8 bits, and what is left of the mean (`off`,
// the mean of the differences) in a step of its own.  An element, of 8 bits, less a
// number of 8 bits is few bits long, so the differences are exact, and so, nearly, is
// their sum, be the mean large next to them or small.  (Differences from the mean in
// binary32 are rounded, equal ones alike, and what their sum shows is those roundings:
// n of elements near the mean was off by up to 4%, and 449 of 210 million y of 4096 x
// 5120 fell to the other side of a border in 8 bits, now 136, in the plain form 128.)
// Rounded to nearest, the mean of a row of one value is that value.
__device__ __forceinline__ float first_bits(float mean) {
    return __uint_as_float((uint32_t)to_bf16(mean) << 16);
}
// The sum of a lane's differences, from its sum of elements: one operation in the
// place of one for each.
template <int L, int U>
__device__ __forceinline__ float less_first_bits(float sum, float mu, uint32_t thread, uint32_t cols) {
    int n = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) n += min(max((int)cols - (int)column<L>(u, thread), 0), 8);
    return __builtin_fmaf(-(float)n, mu, sum);
}

// The mean square of the differences, less that of what is left of the mean.
__device__ __forceinline__ float variance(float mean_square, float off) {
    return fmaxf(__builtin_fmaf(-off, off, mean_square), 0.0f * mean_square);
}

// Within 0.87 of a step of 1 / sqrt(v), one in nine not the nearest number.  Rounded
// correctly, by one more step of Newton's, it is no nearer in what comes of it: of ten
// times 4096 x 8192 y in 8 bits 255 are on another side of a border than in 64 bits, 236
// so, 240 in the plain form.
__device__ __forceinline__ float inv_sqrt(float v) { return __builtin_amdgcn_rsqf(v); }

// ---- forward -------------------------------------------------------------------

struct NormForward {
    const uint16_t* x;
    int64_t ldx, rows;
    uint32_t cols;
    float eps, inv_cols;
    const uint16_t *w, *b;
    uint16_t* y;
    int64_t ldy;
    uint8_t *x_kept, *y_kept;
};

__device__ __forceinline__ void keep(uint8_t* kept, int64_t rows, int64_t row, uint32_t c,
                                     int64_t pitch, float (&v)[8]) {
    u32x2 q;
    const int e = act8_pack8(v, &q);
    const int64_t at = row * pitch + c;
    __builtin_nontemporal_store(q, (TIDE_GLOBAL_AS u32x2*)(kept + at));
    if (c % kActBlock == 0)
        *(TIDE_GLOBAL_AS uint8_t*)(kept + rows * pitch + at / kActBlock) = (uint8_t)(e + 127);
}

template <int L, int U, bool LAYER>
__global__ __launch_bounds__(L > kThreads ? L : kThreads) void norm_forward_kernel(NormForward p) {
    __shared__ float box[L > 64 ? 3 * (L / 64) : 1];
    constexpr int kRows = (L > kThreads ? L : kThreads) / L;
    const int64_t row = L > 64 ? blockIdx.x : (int64_t)blockIdx.x * kRows + threadIdx.x / L;
    if (row >= p.rows) return;  // the whole group of lanes; L > 64: never
    const uint16_t* from = p.x + row * p.ldx;
    u32x4v raw[U], w[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = load_unit<true>(from, column<L>(u, threadIdx.x), p.cols);
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = load_unit(p.w, column<L>(u, threadIdx.x), p.cols);
    if (p.b) {
#pragma unroll
        for (int u = 0; u < U; ++u) b[u] = load_unit(p.b, column<L>(u, threadIdx.x), p.cols);
    }
    settle<L>(raw, threadIdx.x, p.cols);
    float mu = 0.0f, left = 0.0f;
    if constexpr (LAYER) {
        float s[1] = {0.0f};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[8];
            widen(raw[u], v);
#pragma unroll
            for (int k = 0; k < 8; ++k) s[0] += v[k];
        }
        left = s[0];
        row_sums<L>(s, (lds_float*)box);
        mu = first_bits(s[0] * p.inv_cols);
        left = less_first_bits<L, U>(left, mu, threadIdx.x, p.cols);
        forget(raw);
    }
    float s[LAYER ? 2 : 1] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float v[8];
        widen(raw[u], v);
        if constexpr (LAYER) centre<U>(v, mu, column<L>(u, threadIdx.x), p.cols);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[0] = __builtin_fmaf(v[k], v[k], s[0]);
    }
    if constexpr (LAYER) s[1] = left;
    row_sums<L>(s, (lds_float*)box + (L > 64 ? L / 64 : 0));
    forget(raw);
    const float off = LAYER ? s[LAYER] * p.inv_cols : 0.0f;
    const float r = inv_sqrt(variance(s[0] * p.inv_cols, off) + p.eps);
    const int64_t pitch = act8_pitch(p.cols);
    settle<L>(w, threadIdx.x, p.cols);
    if (p.b) settle<L>(b, threadIdx.x, p.cols);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t c = column<L>(u, threadIdx.x);
        if (c >= pitch) break;  // the same in a quad, whose lanes pack together
        float v[8], f[8], y[8];
        widen(raw[u], v);
        widen(w[u], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = (LAYER ? v[k] - mu - off : v[k]) * r * f[k];
        if (p.b) {
            widen(b[u], f);
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] += f[k];
        }
        if (c < p.cols) store8(p.y + row * p.ldy + c, (int64_t)p.cols - c, y);
        if (p.x_kept) keep(p.x_kept, p.rows, row, c, pitch, v);
        if (p.y_kept) {
            if (c + 8 > p.cols) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (c + k >= p.cols) y[k] = 0.0f;
            }
            keep(p.y_kept, p.rows, row, c, pitch, y);
        }
    }
}

// ---- backward ------------------------------------------------------------------

struct NormBackward {
    const uint16_t* dy;
    int64_t lddy;
    const uint16_t* x;
    int64_t ldx;
    const uint8_t* x_kept;
    const uint16_t* w;
    const uint16_t* add;
    int64_t ldadd;
    uint16_t* dx;
    int64_t lddx;
    float *dw_sums, *db_sums;   // [workgroups][pitch], or NULL
    uint16_t *dweight, *dbias;  // the one workgroup's sums go there, or NULL
    int64_t rows, sums_pitch;
    uint32_t cols;
    float eps, inv_cols;
};

// What a lane reads of a row; of a kept x a unit is 8 bytes and its scale.
template <int U>
struct RowParts {
    u32x4v dy[U], x[U];
};

template <int L, int U>
__device__ __forceinline__ void load_row(const NormBackward& p, int64_t row, RowParts<U>& r) {
    const uint32_t t = this_thread();
#pragma unroll
    for (int u = 0; u < U; ++u) r.dy[u] = load_unit<true>(p.dy + row * p.lddy, column<L>(u, t), p.cols);
    if (p.x_kept) {
        const int64_t pitch = act8_pitch(p.cols);
        const uint8_t* scales = p.x_kept + p.rows * pitch;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t c = column<L>(u, t);
            const int64_t at = row * pitch + c;
            r.x[u] = 0;
            if (c < p.cols) {
                const u32x2 q = __builtin_nontemporal_load((const TIDE_GLOBAL_AS u32x2*)(p.x_kept + at));
                r.x[u].xy = q;
                r.x[u].z = *(const TIDE_GLOBAL_AS uint8_t*)(scales + at / kActBlock);
            }
        }
    } else if (p.x) {
#pragma unroll
        for (int u = 0; u < U; ++u) r.x[u] = load_unit<true>(p.x + row * p.ldx, column<L>(u, t), p.cols);
    } else {  // db alone needs no x
#pragma unroll
        for (int u = 0; u < U; ++u) r.x[u] = 0;
    }
}

template <int L, int U>
__device__ __forceinline__ void load_add(const NormBackward& p, int64_t row, u32x4v (&add)[U]) {
    if (p.add) {
        const uint32_t t = this_thread();
#pragma unroll
        for (int u = 0; u < U; ++u) add[u] = load_unit<true>(p.add + row * p.ldadd, column<L>(u, t), p.cols);
    }
}

// A kept unit's values as bf16, which holds them exactly (act8.h).
__device__ __forceinline__ u32x4v kept_unit(u32x4v x) {
    const float f = act8_scale(x.z);
    return u32x4v{act8_bf16x2<false>(x.x, f), act8_bf16x2<true>(x.x, f), act8_bf16x2<false>(x.y, f),
                  act8_bf16x2<true>(x.y, f)};
}

// A workgroup takes every gridDim-th row (kRows of them at a time), so that what
// the chip works on at a time is one piece of memory, and keeps its columns'
// sums of dy n and (DB) of dy in registers.  The next rows' loads are in flight
// while these are worked on, as far as the registers go: of wide rows w is read
// again for each row, `add` is not read ahead, and of the widest nothing is.
template <int L, int U, bool LAYER, bool DB>
__global__ __launch_bounds__(L > kThreads ? L : kThreads) void norm_backward_kernel(NormBackward p) {
    constexpr int kGroup = L > kThreads ? L : kThreads, kRows = kGroup / L;
    constexpr int kBox = L > 64 ? 4 * 3 * (L / 64) : 1;
    constexpr int kSums = kRows > 1 ? (kRows - 1) * L * U * 8 : 1;
    __shared__ __attribute__((aligned(16))) float lds[kBox > kSums ? kBox : kSums];
    lds_float* box = (lds_float*)lds;
    // what a lane holds, in registers, of the L = 1024 lanes' 128 or the others' 256
    constexpr int kHeld = 40 + (DB ? 32 : 24) * U, kMost = L == 1024 ? 124 : 248;
    constexpr bool kAhead = kHeld + 8 * U <= kMost, kAheadAdd = kHeld + 12 * U <= kMost;
    constexpr bool kKeepW = kAhead;
    int64_t row = L > 64 ? blockIdx.x : (int64_t)blockIdx.x * kRows + threadIdx.x / L;
    const int64_t stride = (int64_t)gridDim.x * kRows;
    u32x4v w[U];
    auto load_w = [&]() __attribute__((always_inline)) {
        const uint32_t t = this_thread();
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = p.w ? load_unit(p.w, column<L>(u, t), p.cols) : (u32x4v)0u;
        settle<L>(w, t, p.cols);
    };
    if (kKeepW) load_w();
    float dw[U][8] = {}, db[DB ? U : 1][8] = {};
    RowParts<U> next;
    u32x4v next_add[U], add[U];
    if (kAhead && row < p.rows) load_row<L, U>(p, row, next);
    if (kAheadAdd && row < p.rows) load_add<L, U>(p, row, next_add);
    int slot = 0;
#pragma unroll 1
    for (; row < p.rows; row += stride) {
        // A loop of 11 KB for waves in step takes longer at some places in memory than at
        // others: 8192 rows of 5120 with layer norm and a bias took 62 to 77 us with the
        // loop's start moved by a few instructions, 59.5 on 64 bytes.
        if constexpr (LAYER && L > 64 && U == 1) asm volatile(".p2align 6" ::: "memory");
        RowParts<U> now;
        if constexpr (kAhead)
            now = next;
        else
            load_row<L, U>(p, row, now);
        if constexpr (!kKeepW) load_w();
        if constexpr (kAheadAdd) {
#pragma unroll
            for (int u = 0; u < U; ++u) add[u] = next_add[u];
        } else if constexpr (kAhead) {
            load_add<L, U>(p, row, add);
        }
        if (kAhead && row + stride < p.rows) load_row<L, U>(p, row + stride, next);
        if (kAheadAdd && row + stride < p.rows) load_add<L, U>(p, row + stride, next_add);
        const uint32_t t0 = this_thread();
        settle<L>(now.dy, t0, p.cols);
        if (p.x_kept) {
#pragma unroll
            for (int u = 0; u < U; ++u) now.x[u] = kept_unit(now.x[u]);
        } else {
            settle<L>(now.x, t0, p.cols);
        }
        // a slot is written again two rows later, with a barrier in between
        lds_float* mine = box + (L > 64 ? slot * 6 * (L / 64) : 0);
        slot ^= 1;
        float mu = 0.0f, left = 0.0f, mean_c = 0.0f;
        if constexpr (LAYER) {
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float v[8], d[8], f[8];
                widen(now.x[u], v);
                widen(now.dy[u], d);
                widen(w[u], f);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    s[0] += v[k];
                    s[1] = __builtin_fmaf(d[k], f[k], s[1]);
                }
            }
            left = s[0];
            row_sums<L>(s, mine);
            forget(now.x);
            forget(now.dy);
            forget(w);
            mu = first_bits(s[0] * p.inv_cols);
            left = less_first_bits<L, U>(left, mu, this_thread(), p.cols);
            mean_c = s[1] * p.inv_cols;
            mine += L > 64 ? 2 * (L / 64) : 0;
        }
        float s[LAYER ? 3 : 2] = {};
        float held[U == 1 ? 8 : 1];  // x - mu of lanes of one unit
        const uint32_t t = this_thread();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[8], d[8], f[8];
            widen(now.x[u], v);
            if constexpr (LAYER) centre<U>(v, mu, column<L>(u, t), p.cols);
            widen(now.dy[u], d);
            widen(w[u], f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s[0] = __builtin_fmaf(v[k], v[k], s[0]);
                s[1] = __builtin_fmaf(d[k] * f[k], v[k], s[1]);
                if constexpr (U == 1) held[k] = v[k];
            }
        }
        if constexpr (LAYER) s[2] = left;
        row_sums<L>(s, mine);
        forget(now.x);
        forget(now.dy);
        if constexpr (kAhead) {
            forget(w);
        } else {
            load_add<L, U>(p, row, add);
            load_w();
        }
        // With d = x - mu still off by `off`, n = (d - off) r:
        //   dx = r c - (r^3 mean(c (d - off))) (d - off) - r mean(c)
        const float off = LAYER ? s[LAYER ? 2 : 0] * p.inv_cols : 0.0f;
        const float r = inv_sqrt(variance(s[0] * p.inv_cols, off) + p.eps);
        const float along = r * (r * __builtin_fmaf(-off, mean_c, s[1] * p.inv_cols));
        const float by_d = -r * along, rest = -r * __builtin_fmaf(-along, off, mean_c);
        const uint32_t t2 = this_thread();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t c = column<L>(u, t2);
            float v[8], d[8], f[8];
            if constexpr (U == 1) {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = held[k];
            } else {
                widen(now.x[u], v);
                if constexpr (LAYER) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] -= mu;
                }
            }
            widen(now.dy[u], d);
            if constexpr (DB) {
#pragma unroll
                for (int k = 0; k < 8; ++k) db[u][k] += d[k];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                d[k] *= r;
                dw[u][k] = __builtin_fmaf(d[k], LAYER ? v[k] - off : v[k], dw[u][k]);
            }
            if (p.dx && c < p.cols) {
                float g[8];
                widen(w[u], f);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    g[k] = __builtin_fmaf(d[k], f[k], LAYER ? __builtin_fmaf(by_d, v[k], rest) : by_d * v[k]);
                if (p.add) {
                    settle(add[u], c, p.cols);
                    widen(add[u], f);
#pragma unroll
                    for (int k = 0; k < 8; ++k) g[k] += f[k];
                }
                store8(p.dx + row * p.lddx + c, (int64_t)p.cols - c, g);
            }
        }
    }
    // the sums of the workgroup's other groups of lanes, then out
    auto finish = [&](auto& sum, float* sums, uint16_t* out) __attribute__((always_inline)) {
        const uint32_t t = threadIdx.x;
        if constexpr (kRows > 1) {
            __syncthreads();
            const int group = threadIdx.x / L, lane = threadIdx.x % L;
            if (group) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        box[(((group - 1) * U + u) * 8 + k) * L + lane] = sum[u][k];
            }
            __syncthreads();
            if (group) return;
            for (int o = 0; o < kRows - 1; ++o)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int k = 0; k < 8; ++k) sum[u][k] += box[((o * U + u) * 8 + k) * L + lane];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t c = column<L>(u, t);
            if (c >= p.cols) break;
            if (out) {
                store8(out + c, (int64_t)p.cols - c, sum[u]);
            } else {
                float* to = sums + (int64_t)blockIdx.x * p.sums_pitch + c;
#pragma unroll
                for (int k = 0; k < 8; k += 4)
                    *(TIDE_GLOBAL_AS f32x4*)(to + k) =
                        f32x4{sum[u][k], sum[u][k + 1], sum[u][k + 2], sum[u][k + 3]};
            }
        }
    };
    if (p.dw_sums || p.dweight) finish(dw, p.dw_sums, p.dweight);
    if constexpr (DB) finish(db, p.db_sums, p.dbias);
}

// dw and db from the workgroups' sums.  A workgroup takes 64 columns, 16 lanes of
// 4, and its 64 such sets of lanes a row of sums in turn, so that few workgroups
// (narrow rows) have many loads in flight; the sets' sums are added in order.
constexpr int kSumCols = 64, kSumSets = 64;
constexpr int kSumAhead = 8;  // rows whose loads are in flight together

__global__ __launch_bounds__(16 * kSumSets) void norm_sums_kernel(const float* dw_sums,
                                                                  const float* db_sums,
                                                                  int64_t rows, int64_t pitch,
                                                                  int64_t cols, uint16_t* dweight,
                                                                  uint16_t* dbias) {
    __shared__ __attribute__((aligned(16))) float part[kSumSets][kSumCols + 4];
    const int64_t groups = (cols + kSumCols - 1) / kSumCols;
    const bool second = blockIdx.x >= groups || !dw_sums;
    const float* sums = second ? db_sums : dw_sums;
    uint16_t* out = second ? dbias : dweight;
    const int64_t c0 = (blockIdx.x - (blockIdx.x >= groups ? groups : 0)) * kSumCols;
    const int set = threadIdx.x / 16, lane = threadIdx.x % 16;
    f32x4 s = 0.0f;
    if (c0 + lane * 4 < pitch) {
        const float* from = sums + c0 + lane * 4;
        for (int64_t k = set; k < rows; k += kSumSets * kSumAhead) {
            f32x4 v[kSumAhead];
#pragma unroll
            for (int a = 0; a < kSumAhead; ++a) {
                const int64_t at = k + a * kSumSets;
                v[a] = at < rows ? *(const TIDE_GLOBAL_AS f32x4*)(from + at * pitch) : (f32x4)0.0f;
            }
#pragma unroll
            for (int a = 0; a < kSumAhead; ++a) s += v[a];
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) part[set][lane * 4 + k] = s[k];
    __syncthreads();
    const int c = threadIdx.x % kSumCols, quarter = threadIdx.x / kSumCols;  // of 16
    float q = 0.0f;
#pragma unroll
    for (int k = 0; k < kSumSets / 16; ++k) q += part[quarter * (kSumSets / 16) + k][c];
    __syncthreads();
    part[quarter][c] = q;
    __syncthreads();
    if (threadIdx.x >= kSumCols || c0 + c >= cols) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) q += part[k][c];
    *(TIDE_GLOBAL_AS uint16_t*)(out + c0 + c) = to_bf16(q);
}

// ---- host ----------------------------------------------------------------------

constexpr int64_t kMaxNormCols = 32768;  // 4096 units: 1024 lanes of 4
constexpr int64_t kMaxNormRows = (int64_t)1 << 27;  // 16 lanes each in one grid
constexpr float kMinEps = 1e-30f;

// Lanes (at most) and units of a row: the first form that holds it is taken.
struct RowShape {
    int lanes, units;
};

using ForwardKernel = void (*)(NormForward);
using BackwardKernel = void (*)(NormBackward);

struct ForwardForm {
    RowShape shape;
    ForwardKernel rms, layer;
};
struct BackwardForm {
    RowShape shape;
    BackwardKernel rms, layer, rms_db, layer_db;
};

#define TIDE_FORWARD_FORM(L, U) \
    {{L, U}, norm_forward_kernel<L, U, false>, norm_forward_kernel<L, U, true>}
#define TIDE_BACKWARD_FORM(L, U)                                                    \
    {{L, U}, norm_backward_kernel<L, U, false, false>, norm_backward_kernel<L, U, true, false>, \
     norm_backward_kernel<L, U, false, true>, norm_backward_kernel<L, U, true, true>}

const ForwardForm kForwardForms[] = {
    TIDE_FORWARD_FORM(16, 1),  TIDE_FORWARD_FORM(64, 1),  TIDE_FORWARD_FORM(64, 2),
    TIDE_FORWARD_FORM(256, 1), TIDE_FORWARD_FORM(512, 2), TIDE_FORWARD_FORM(512, 3),
    TIDE_FORWARD_FORM(512, 4), TIDE_FORWARD_FORM(1024, 3), TIDE_FORWARD_FORM(1024, 4)};
// One unit a lane as far as 1024 lanes go, which keeps what the lane holds of the
// weight, the sums and the next row in few registers: us for 8192 rows of 5120 with
// rms and 640 lanes 56 (295 MB, 5.3 TB/s), with 256 lanes of 3 units 76.  Past 16384
// columns 512 lanes have the registers that 1024 have not (us with 512 lanes / with
// 1024 of 3 and 4 units, 2300 x 24576, 2300 x 28672 and 2000 x 32768): layer norm 82 / 94,
// 129 / 146, 132 / 162; with a bias 120 / 135, 151 / 243, 178 / 247, though with 7 units 9
// registers and with 8 units 57 of 256 are spilled to memory there (of 1024 lanes 34 and
// 96 of 128); rms 76 / 85, 110 / 103, 113 / 102, whose widest rows would be 7 to 10% faster
// the other way: one list serves all four.
const BackwardForm kBackwardForms[] = {
    TIDE_BACKWARD_FORM(16, 1),   TIDE_BACKWARD_FORM(64, 1),  TIDE_BACKWARD_FORM(64, 2),
    TIDE_BACKWARD_FORM(1024, 1), TIDE_BACKWARD_FORM(1024, 2), TIDE_BACKWARD_FORM(512, 5),
    TIDE_BACKWARD_FORM(512, 6),  TIDE_BACKWARD_FORM(512, 7), TIDE_BACKWARD_FORM(512, 8)};

template <typename Form, size_t N>
const Form& form_of(const Form (&forms)[N], int64_t cols) {
    const int64_t units = act8_pitch(cols) / 8;
    for (size_t k = 0; k + 1 < N; ++k)
        if (forms[k].shape.lanes * forms[k].shape.units >= units) return forms[k];
    return forms[N - 1];
}

// Threads of a workgroup: of wide rows, whole waves that hold one.  (Lanes that
// hold nothing work all the same: 8192 rows of 5120 with layer norm took 84 us with
// 1024 lanes, 76 with 640, 60 as the loop is now.  Its vector pipes are busy 56% of the
// time, 30% for 777 rows; the rest the waves of a row wait for each other, twice a row.)
int threads_of(const RowShape& s, int64_t cols) {
    return s.lanes <= 64 ? kThreads : (int)round_up(ceil_div(act8_pitch(cols) / 8, s.units), 64);
}

// Rows of a workgroup at a time.
int64_t rows_of(const RowShape& s) { return s.lanes <= 64 ? kThreads / s.lanes : 1; }

// Workgroups of the backward pass at most.  Each writes a row of sums that another
// launch reads, so wide rows take no more than the compute units: us at 256 and
// 512 workgroups for 2300 x 28672 with rms 112 and 125, 8192 x 8192 73 and 78, 512 x
// 4096 11.2 and 12.1.  Narrower ones take twice as many: 8192 x 2048 39.9 and 29.5
// (1024: 29.3), 65536 x 128 23.3 and 19.2 (1024: 17.9, which is not taken: one number
// serves all narrow rows).
// So does layer norm, whose waves wait for each other twice a row, where two of its
// workgroups fit a compute unit's registers: 8192 rows of 4096 with a bias 54 and 47,
// without 53 and 44, of 5120 without 71 and 57, of 6144 without 75 and 64; of 5120 with
// a bias, whose 10 waves of 85 registers do not fit twice, 59.5 and 65, of 7168 without
// 88 and 93.  (From 2048 rows on, four for each: 777 of 4096 with a bias 14 and 15; of
// lanes with one unit: 2300 x 28672 148 and 172.)
int64_t most_groups(const RowShape& s, int threads, int64_t rows, bool layer, bool db) {
    const bool two = layer && s.units == 1 && threads <= (db ? 512 : 768);
    return threads < 512 || (two && rows >= 2048) ? 512 : 256;
}

tide_status check_norm(int64_t rows, int64_t cols, int32_t kind, float eps) {
    if (rows < 0 || cols < 0 || (kind != TIDE_NORM_RMS && kind != TIDE_NORM_LAYER)) return TIDE_EINVAL;
    if (!(eps >= kMinEps) || !std::isfinite(eps)) return TIDE_EINVAL;
    if (rows > kMaxNormRows || cols > kMaxNormCols || rows * cols > kMaxElements)
        return TIDE_EUNSUPPORTED;
    return TIDE_OK;
}

}  // namespace

extern "C" tide_status tide_norm_forward(const tide_norm_forward_args* args, tide_stream_t stream) {
    if (!args) return TIDE_EINVAL;
    const tide_norm_forward_args& a = *args;
    const int64_t T = a.rows, C = a.cols;
    TIDE_TRY(check_norm(T, C, a.kind, a.eps));
    if (T == 0 || C == 0) return TIDE_OK;
    TIDE_TRY(check_rows(a.x, a.ldx, T, C));
    TIDE_TRY(check_rows(a.weight, C, 1, C));
    if (a.bias) TIDE_TRY(check_rows(a.bias, C, 1, C));
    TIDE_TRY(check_rows(a.y, a.ldy, T, C));
    if (a.x_kept) TIDE_TRY(check_kept(a.x_kept, T, C));
    if (a.y_kept) TIDE_TRY(check_kept(a.y_kept, T, C));
    const Extent in[] = {rows_extent(a.x, a.ldx, T, C), rows_extent(a.weight, C, 1, C),
                         rows_extent(a.bias, C, 1, C)};
    const Extent out[] = {rows_extent(a.y, a.ldy, T, C), bytes_extent(a.x_kept, act8_bytes(T, C)),
                          bytes_extent(a.y_kept, act8_bytes(T, C))};
    TIDE_TRY(check_apart(in, 3, out, 3));
    TIDE_TRY(check_stream_device(stream));
    NormForward p = {};
    p.x = static_cast<const uint16_t*>(a.x);
    p.ldx = a.ldx;
    p.rows = T;
    p.cols = (uint32_t)C;
    p.eps = a.eps;
    p.inv_cols = 1.0f / (float)C;
    p.w = static_cast<const uint16_t*>(a.weight);
    p.b = static_cast<const uint16_t*>(a.bias);
    p.y = static_cast<uint16_t*>(a.y);
    p.ldy = a.ldy;
    p.x_kept = static_cast<uint8_t*>(a.x_kept);
    p.y_kept = static_cast<uint8_t*>(a.y_kept);
    const ForwardForm& f = form_of(kForwardForms, C);
    const int threads = threads_of(f.shape, C);
    return launch(a.kind == TIDE_NORM_LAYER ? f.layer : f.rms, ceil_div(T, rows_of(f.shape)), threads,
                  stream, p);
}

namespace {

struct NormBackwardPlan {
    const BackwardForm* form;
    int threads;
    int64_t groups, pitch;  // workgroups; columns of their sums
    float *dw = nullptr, *db = nullptr;
    int64_t bytes;
};

tide_status check_backward(const tide_norm_backward_args& a) {
    const int64_t T = a.rows, C = a.cols;
    TIDE_TRY(check_norm(T, C, a.kind, a.eps));
    if (!a.dx && !a.dweight && !a.dbias) return TIDE_OK;
    TIDE_TRY(check_rows(a.dy, a.lddy, T, C));
    if (a.x && a.x_kept) return TIDE_EINVAL;
    if (a.dx || a.dweight) {
        if (a.x)
            TIDE_TRY(check_rows(a.x, a.ldx, T, C));
        else
            TIDE_TRY(check_kept(a.x_kept, T, C));
    }
    if (a.dx) {
        TIDE_TRY(check_rows(a.weight, C, 1, C));
        TIDE_TRY(check_rows(a.dx, a.lddx, T, C));
        if (a.add) TIDE_TRY(check_rows(a.add, a.ldadd, T, C));
    }
    if (a.dweight) TIDE_TRY(check_rows(a.dweight, C, 1, C));
    if (a.dbias) TIDE_TRY(check_rows(a.dbias, C, 1, C));
    return TIDE_OK;
}

NormBackwardPlan plan_backward(const tide_norm_backward_args& a, void* ws) {
    NormBackwardPlan b;
    Carver c{static_cast<char*>(ws)};
    b.form = &form_of(kBackwardForms, a.cols);
    b.threads = threads_of(b.form->shape, a.cols);
    const int64_t at_once = rows_of(b.form->shape);
    const int64_t most = most_groups(b.form->shape, b.threads, a.rows, a.kind == TIDE_NORM_LAYER,
                                     a.dbias != nullptr);
    const int64_t each = std::max<int64_t>(1, ceil_div(a.rows, most * at_once));
    b.groups = ceil_div(a.rows, each * at_once);
    b.pitch = round_up(a.cols, 8);
    if (b.groups > 1) {
        if (a.dweight) b.dw = c.take<float>(b.groups * b.pitch);
        if (a.dbias) b.db = c.take<float>(b.groups * b.pitch);
    }
    b.bytes = c.used;
    return b;
}

}  // namespace

extern "C" tide_status tide_norm_backward_workspace(const tide_norm_backward_args* args,
                                                    size_t* bytes) {
    if (!args || !bytes) return TIDE_EINVAL;
    TIDE_TRY(check_backward(*args));
    *bytes = args->rows && args->cols ? (size_t)plan_backward(*args, nullptr).bytes : 0;
    return TIDE_OK;
}

extern "C" tide_status tide_norm_backward(const tide_norm_backward_args* args, void* workspace,
                                          size_t workspace_bytes, tide_stream_t stream) {
    if (!args) return TIDE_EINVAL;
    const tide_norm_backward_args& a = *args;
    TIDE_TRY(check_backward(a));
    const int64_t T = a.rows, C = a.cols;
    if ((!a.dx && !a.dweight && !a.dbias) || C == 0) return TIDE_OK;
    const bool in_place = a.add == a.dx && (T <= 1 || a.ldadd == a.lddx);
    const Extent ext[] = {
        rows_extent(a.dy, a.lddy, T, C),
        a.dx || a.dweight ? rows_extent(a.x, a.ldx, T, C) : Extent(),
        a.dx || a.dweight ? bytes_extent(a.x_kept, act8_bytes(T, C)) : Extent(),
        a.dx ? rows_extent(a.weight, C, 1, C) : Extent(),
        a.dx && !in_place ? rows_extent(a.add, a.ldadd, T, C) : Extent(),
        rows_extent(a.dx, a.lddx, T, C),
        rows_extent(a.dweight, C, 1, C),
        rows_extent(a.dbias, C, 1, C)};
    TIDE_TRY(check_apart(ext, 5, ext + 5, 3));
    const NormBackwardPlan b = plan_backward(a, workspace);
    TIDE_TRY(check_workspace(workspace, workspace_bytes, T ? b.bytes : 0, ext, 8));
    TIDE_TRY(check_stream_device(stream));
    NormBackward p = {};
    p.dy = static_cast<const uint16_t*>(a.dy);
    p.lddy = a.lddy;
    const bool need_x = a.dx || a.dweight;
    if (need_x) {
        p.x = static_cast<const uint16_t*>(a.x);
        p.ldx = a.ldx;
        p.x_kept = static_cast<const uint8_t*>(a.x_kept);
    }
    p.dx = static_cast<uint16_t*>(a.dx);
    p.lddx = a.lddx;
    if (a.dx) {
        p.w = static_cast<const uint16_t*>(a.weight);
        p.add = static_cast<const uint16_t*>(a.add);
        p.ldadd = a.ldadd;
    }
    p.dw_sums = b.dw;
    p.db_sums = b.db;
    if (b.groups <= 1) {
        p.dweight = static_cast<uint16_t*>(a.dweight);
        p.dbias = static_cast<uint16_t*>(a.dbias);
    }
    p.rows = T;
    p.sums_pitch = b.pitch;
    p.cols = (uint32_t)C;
    p.eps = a.eps;
    p.inv_cols = 1.0f / (float)C;
    const bool layer = a.kind == TIDE_NORM_LAYER;
    const BackwardForm& f = *b.form;
    auto k = layer ? a.dbias ? f.layer_db : f.layer : a.dbias ? f.rms_db : f.rms;
    // without rows one workgroup writes the empty sums
    const int64_t grid = T ? b.groups : a.dweight || a.dbias ? 1 : 0;
    TIDE_TRY(launch(k, grid, b.threads, stream, p));
    if (b.groups <= 1 || !(b.dw || b.db)) return TIDE_OK;
    return launch(norm_sums_kernel, ceil_div(C, kSumCols) * ((b.dw ? 1 : 0) + (b.db ? 1 : 0)),
                  16 * kSumSets, stream, (const float*)b.dw, (const float*)b.db, b.groups, b.pitch, C,
                  static_cast<uint16_t*>(a.dweight), static_cast<uint16_t*>(a.dbias));
}
