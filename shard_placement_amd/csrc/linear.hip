// linear.hip -- a layer's product on a placed weight, with bias, activation
// and residual in its epilogue, and its gradients from 8-bit checkpoints, for
// gfx950.
//
//   forward   z = x W^T + bias, y = act(z) + residual
//   backward  dz = dy act'(z), dx = dz W, dW = dz^T x, dbias = column sums of dz
//
// W is a full tensor as the all-gather placement writes it, dW and dbias are
// gradients as the reduce-scatter reads them.  All three products run
// through one tile loop (tile_product.h); the epilogue works on the
// accumulators in registers, so z is never written in more than 8 bits.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "act8.h"
#include "bf16_io.h"
#include "linear_check.h"
#include "product_shape.h"
#include "tide.h"
#include "tile_product.h"

using namespace tide;

namespace {

// ---- activation functions ------------------------------------------------

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kLog2E = 1.4426950408889634f;
// 2 sqrt(2 / pi) (z + 0.044715 z^3) = z (kTanhC + kTanhA z^2)
constexpr float kTanhC = 1.5957691216057308f;
constexpr float kTanhA = kTanhC * 0.044715f;

// 1 / (1 + exp(-u)), off by a few binary32 steps; 0.5 (1 + tanh(v)) is this at
// u = 2 v, so the tanh form of gelu is z * sigmoid(z (kTanhC + kTanhA z^2)).
// The exponential's and the reciprocal's instructions are within one step; a
// division written out would be most of the epilogue's work.
__device__ __forceinline__ float sigmoid(float u) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2E * u));
}

// exp(-z^2 / 2) and the normal distribution's Phi(z).  Its lower tail is
// erfc(x) / 2, x = |z| / sqrt(2), and erfc(x) = t Q(t) exp(-x^2) with t = 1 / (1 +
// 0.375 x).  Q is fitted to the least relative error over 0 <= x <= 10 (6.4e-7;
// from x = 9.3 on exp(-x^2) is below binary32's normal numbers and 0 here), so
// gelu is a bf16 rounding off in its far negative tail too, where a formula of
// small absolute error is percents off.  A library erff took 55 us in the
// gradient of 2048 x 13824 elements, which reads and writes 141 MB, where this
// takes 39; a forward of 4096 x 16384 x 1024 with gelu takes 157 us, 154 with
// a shorter polynomial of small absolute error, 2% off at z = -10.
__device__ __forceinline__ float normal_cdf(float z, float* bell) {
    const float g = __builtin_amdgcn_exp2f(-0.5f * kLog2E * (z * z));
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.375f * kSqrtHalf, fabsf(z), 1.0f));
    float poly = __builtin_fmaf(-0.1350946333f, t, 0.3879334708f);
    poly = __builtin_fmaf(poly, t, -0.1295913167f);
    poly = __builtin_fmaf(poly, t, 0.2830573515f);
    poly = __builtin_fmaf(poly, t, 0.1666661391f);
    poly = __builtin_fmaf(poly, t, 0.2156888808f);
    poly = __builtin_fmaf(poly, t, 0.2113394712f);
    const float tail = 0.5f * poly * t * g;
    *bell = g;
    return z < 0.0f ? tail : 1.0f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == TIDE_ACT_RELU) return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    if constexpr (ACT == TIDE_ACT_GELU) {
        float bell;
        return z * normal_cdf(z, &bell);
    }
    if constexpr (ACT == TIDE_ACT_GELU_TANH)
        return z * sigmoid(z * __builtin_fmaf(kTanhA, z * z, kTanhC));
    if constexpr (ACT == TIDE_ACT_SILU) return z * sigmoid(z);
    return z;
}

// z may be infinite where a finite one was kept (act8.h: values that round up
// to 2^128), and infinity times the 0 that bounds it would be NaN: a factor z is
// held within what changes nothing, the other factor being 0 outside.  (NaN
// reaches the result through the other terms.)
__device__ __forceinline__ float within(float z) { return __builtin_amdgcn_fmed3f(z, -256.0f, 256.0f); }

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == TIDE_ACT_RELU) return z > 0.0f ? 1.0f : z < 0.0f ? 0.0f : 0.0f * z;
    if constexpr (ACT == TIDE_ACT_GELU) {
        float bell;
        const float cdf = normal_cdf(z, &bell);
        return __builtin_fmaf(within(z) * kInvSqrt2Pi, bell, cdf);
    }
    if constexpr (ACT == TIDE_ACT_GELU_TANH) {
        const float t = z * z;
        const float s = sigmoid(z * __builtin_fmaf(kTanhA, t, kTanhC));
        // where the sigmoid is 0 or 1 the polynomial may be infinite already
        const float q = __builtin_fmaf(-s, s, s);
        return q > 0.0f ? __builtin_fmaf(z * q, __builtin_fmaf(3.0f * kTanhA, t, kTanhC), s) : s;
    }
    if constexpr (ACT == TIDE_ACT_SILU) {
        const float s = sigmoid(z);
        return s * __builtin_fmaf(within(z), 1.0f - s, 1.0f);
    }
    return 1.0f;
}

// v to act(v), eight at a time: the choice is made once for all of them.
template <int ACT>
__device__ __forceinline__ void apply_act(float (&v)[8]) {
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] = act_value<ACT>(v[r]);
}
__device__ __forceinline__ void apply_act(float (&v)[8], int act) {
    switch (act) {
        case TIDE_ACT_RELU: return apply_act<TIDE_ACT_RELU>(v);
        case TIDE_ACT_GELU: return apply_act<TIDE_ACT_GELU>(v);
        case TIDE_ACT_GELU_TANH: return apply_act<TIDE_ACT_GELU_TANH>(v);
        case TIDE_ACT_SILU: return apply_act<TIDE_ACT_SILU>(v);
        default: return;
    }
}

// v times act'(z).
template <int ACT>
__device__ __forceinline__ void apply_slope(const float (&z)[8], float (&v)[8]) {
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] *= act_slope<ACT>(z[r]);
}

// ---- epilogue ------------------------------------------------------------

// What happens to a finished sum at output column i of row j.
struct Epilogue {
    int64_t I, J;
    uint16_t* out;
    int64_t ldo;
    const uint16_t* bias;
    const uint16_t* res;
    int64_t ldr;
    uint8_t* kept;  // the checkpoint of z
    int32_t act;
};

// Eight sums at columns i .. i + 7 of row j through the epilogue.  A
// checkpoint's block of 32 columns lies in four consecutive lanes, all of
// which call this (`there`: the lane's row and columns exist).
__device__ __forceinline__ void finish(const Epilogue& e, int64_t i, int64_t j, bool there,
                                       float (&v)[8]) {
    const int64_t n = there ? e.I - i : 0;
    if (e.bias) {
        float b[8];
        load8(e.bias + i, n, b);
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] += b[r];
    }
    if (e.kept) {
        float z[8];
        if (n >= 8) {
#pragma unroll
            for (int r = 0; r < 8; ++r) z[r] = v[r];
        } else {
#pragma unroll
            for (int r = 0; r < 8; ++r) z[r] = r < n ? v[r] : 0.0f;
        }
        u32x2 q;
        const int x = act8_pack8(z, &q);
        const int64_t pitch = act8_pitch(e.I);
        if (j < e.J && i < pitch) {
            *(TIDE_GLOBAL_AS u32x2*)(e.kept + j * pitch + i) = q;
            if (i % kActBlock == 0)
                *(TIDE_GLOBAL_AS uint8_t*)(e.kept + e.J * pitch + (j * pitch + i) / kActBlock) =
                    (uint8_t)(x + 127);
        }
    }
    if (n <= 0) return;
    apply_act(v, e.act);
    if (e.res) {
        float x[8];
        load8(e.res + j * e.ldr + i, n, x);
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] += x[r];
    }
    store8(e.out + j * e.ldo + i, n, v);
}

// ---- products ------------------------------------------------------------

struct Product {
    Operand A, B;
    int64_t depth;        // contraction elements
    int64_t split_depth;  // of one split (a multiple of kSplitUnit)
    int32_t tiles_i, tiles_j, splits;
    float* partial;       // [splits][J][pitch] sums where splits > 1
    int64_t partial_pitch;
    Epilogue e;
};

// Workgroup -> (tile, split).  Consecutive workgroups go to the 8 XCDs in
// turn, so each XCD is given a run of consecutive tiles of its own, and tiles
// are numbered in bands of kBand tiles of j (all of i inside a band): the
// tiles an XCD works on together share rows of both operands in its L2.
constexpr int kXcdCount = 8;
constexpr int kBand = 4;

__device__ __forceinline__ void tile_at(const Product& p, uint32_t b, uint32_t total, int* ti,
                                        int* tj, int* sp) {
    const uint32_t each = total / kXcdCount, extra = total % kXcdCount;
    const uint32_t x = b % kXcdCount, n = b / kXcdCount;
    b = x * each + min(x, extra) + n;
    const uint32_t tiles = (uint32_t)p.tiles_i * (uint32_t)p.tiles_j;
    const uint32_t s = b / tiles;
    b -= s * tiles;
    const uint32_t band = b / (uint32_t)(kBand * p.tiles_i);
    const uint32_t width = min((uint32_t)kBand, p.tiles_j - band * kBand);
    b -= band * kBand * p.tiles_i;
    // the same in all lanes: scalar registers, of which the tile loop needs fewer
    *sp = __builtin_amdgcn_readfirstlane(s);
    *ti = __builtin_amdgcn_readfirstlane(b / width);
    *tj = __builtin_amdgcn_readfirstlane(band * kBand + b % width);
}

// A wave's LDS writes have arrived before its reads, and its reads have
// returned before it writes again.
__device__ __forceinline__ void wave_lds_order() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// LDS of a workgroup: two staged tiles, which the epilogue reuses.
template <int BI, int BJ, int K>
constexpr int kProductLds = 2 * (BI + BJ) * K * 2;

// The tile of workgroup `block` of `blocks`.  H = 2: the contraction in two
// halves, each by WI * WJ waves with tiles in LDS of their own, whose sums are
// added in LDS; each set of waves then finishes half of the tile.
template <int BI, int BJ, int K, int WI, int WJ, Layout CA, Layout CB, int H = 1>
__device__ __forceinline__ void product_tile(const Product& p, uint32_t block, uint32_t blocks,
                                             TIDE_LDS char* lds) {
    constexpr int TI = BI / WI / 16, TJ = BJ / WJ / 16;
    static_assert(TI % 2 == 0, "a wave holds whole checkpoint blocks");
    int ti, tj, sp;
    tile_at(p, block, blocks, &ti, &tj, &sp);
    const int64_t i0 = (int64_t)ti * BI, j0 = (int64_t)tj * BJ;
    f32x4v acc[TI][TJ];
    tile_loop<BI, BJ, K, WI, WJ, CA, CB, H>(p.A, p.B, p.depth, sp * p.split_depth,
                                            min(p.depth, (sp + 1) * p.split_depth), i0, j0, lds, acc);

    // The accumulators pass through LDS, 16 rows of a wave at a time, so that
    // each lane ends with 8 consecutive columns and a row's stores are whole
    // lines.  The row pitch's extra 4 floats keep the writes off each other's
    // banks.
    constexpr int kRow = TI * 16, kPitch = kRow + 4, kLanes = kRow / 8;
    constexpr int kStaging = WI * WJ * H * 16 * kPitch * 4;
    constexpr int kDone = H == 2 && TJ > 1 ? TJ / 2 : TJ;  // 16-row pieces that a wave finishes
    static_assert(H == 1 || TJ == 1 || TJ % 2 == 0, "the halves share the tile");
    static_assert(kStaging <= kProductLds<BI, BJ, K> * H, "the staging fits");
    tile_barrier(lds, lds);
    // (what follows from the thread is worked out here, not kept in registers
    // through the loop)
    int thread = threadIdx.x;
    asm volatile("" : "+v"(thread));
    const int half = H == 2 ? __builtin_amdgcn_readfirstlane(thread >> 6) / (WI * WJ) : 0;
    const int lane = thread & 63, wave = (thread >> 6) - half * WI * WJ;
    if constexpr (H == 2) {
        // what the other half's wave finishes goes to it; staging lies behind
        constexpr int kPiece = 64 * 16, kWave = TI * kDone * kPiece;
        static_assert(kStaging + 2 * WI * WJ * kWave <= 2 * kProductLds<BI, BJ, K>, "both fit");
        TIDE_LDS char* box = lds + kStaging + wave * kWave + lane * 16;
        constexpr int kOther = WI * WJ * kWave;
        if (half) {
#pragma unroll
            for (int x = 0; x < TI; ++x)
#pragma unroll
                for (int y = 0; y < kDone; ++y)
                    *(TIDE_LDS f32x4v*)(box + (x * kDone + y) * kPiece) = acc[x][y];
        } else if (TJ > 1) {
#pragma unroll
            for (int x = 0; x < TI; ++x)
#pragma unroll
                for (int y = 0; y < kDone; ++y)
                    *(TIDE_LDS f32x4v*)(box + kOther + (x * kDone + y) * kPiece) = acc[x][TJ - kDone + y];
        }
        tile_barrier(lds, lds);
        if (half && TJ == 1) return;
        if (half) {
#pragma unroll
            for (int x = 0; x < TI; ++x)
#pragma unroll
                for (int y = 0; y < kDone; ++y)
                    acc[x][y] = acc[x][TJ - kDone + y] +
                                *(const TIDE_LDS f32x4v*)(box + kOther + (x * kDone + y) * kPiece);
        } else {
#pragma unroll
            for (int x = 0; x < TI; ++x)
#pragma unroll
                for (int y = 0; y < kDone; ++y)
                    acc[x][y] += *(const TIDE_LDS f32x4v*)(box + (x * kDone + y) * kPiece);
        }
    }
    TIDE_LDS float* mine = (TIDE_LDS float*)lds + (thread >> 6) * 16 * kPitch;
    const int64_t iw = i0 + (wave / WJ) * kRow + (lane % kLanes) * 8;
    const int64_t jw = j0 + ((wave % WJ) * TJ + half * kDone) * 16 + lane / kLanes;
#pragma unroll
    for (int y = 0; y < kDone; ++y) {
#pragma unroll
        for (int x = 0; x < TI; ++x)
            *(TIDE_LDS f32x4v*)(mine + (lane & 15) * kPitch + x * 16 + (lane >> 4) * 4) = acc[x][y];
        wave_lds_order();
#pragma unroll 1
        for (int r = 0; r < 16; r += 64 / kLanes) {
            const int64_t j = jw + 16 * y + r;
            const TIDE_LDS float* row = mine + (r + lane / kLanes) * kPitch + (lane % kLanes) * 8;
            const f32x4v lo = *(const TIDE_LDS f32x4v*)row, hi = *(const TIDE_LDS f32x4v*)(row + 4);
            const bool there = j < p.e.J && iw < p.e.I;
            if (p.splits > 1) {
                if (!there) continue;
                float* to = p.partial + (sp * p.e.J + j) * p.partial_pitch + iw;
                *(TIDE_GLOBAL_AS f32x4v*)to = lo;
                *(TIDE_GLOBAL_AS f32x4v*)(to + 4) = hi;
                continue;
            }
            float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            finish(p.e, iw, j, there, v);
        }
        wave_lds_order();
    }
}

template <int BI, int BJ, int K, int WI, int WJ, Layout CA, Layout CB, int H = 1>
__global__ __launch_bounds__(WI* WJ * 64 * H, BI == 256 ? 2 : 1) void product_kernel(Product p) {
    __shared__ __attribute__((aligned(1024))) char lds[kProductLds<BI, BJ, K> * H];
    product_tile<BI, BJ, K, WI, WJ, CA, CB, H>(p, blockIdx.x, gridDim.x, (TIDE_LDS char*)lds);
}

// dx and dW in one launch, for shapes too small to fill the chip one after the
// other (77 x 768 x 2048: 13.2 us for both, 7.6, 3.0 and 8.0 for dx, its join
// and dW): the first `n_w` workgroups take dW's tiles, the others dx's.  H = 2
// where each has a compute unit to itself (the same call 14.7 us with dz's
// launch, 16.0 with one set of waves; 300 x 1024 x 1024 16.3, 18.5).
template <int BJ, int WI, int WJ, int H>
__global__ __launch_bounds__(256 * H) void pair_kernel(Product w, Product x, int32_t n_w) {
    __shared__ __attribute__((aligned(1024))) char lds[kProductLds<128, 128, 64> * H];
    if ((int)blockIdx.x < n_w)
        product_tile<128, 128, 64, 2, 2, kKept, kColumns, H>(w, blockIdx.x, n_w,
                                                             (TIDE_LDS char*)lds);
    else
        product_tile<128, BJ, 64, WI, WJ, kColumns, kRows, H>(x, blockIdx.x - n_w, gridDim.x - n_w,
                                                              (TIDE_LDS char*)lds);
}

// The same with 256-wide tiles, one workgroup a compute unit, the product of the
// longer tiles first: where its tiles do not fill whole rounds of the chip the
// other's fill the gaps (2048 x 13824 x 5120: 160 tiles of dx of 342 us and 1080 of
// dW of 57 on 256 compute units, 460 us for both, 570 one after the other).
template <int BJW, int BJX>
__global__ __launch_bounds__(512, 2) void wide_pair_kernel(Product w, Product x, int32_t first_w,
                                                           int32_t first_x) {
    constexpr int kBj = BJW > BJX ? BJW : BJX;
    __shared__ __attribute__((aligned(1024))) char lds[kProductLds<256, kBj, 64>];
    const int block = blockIdx.x, blocks = gridDim.x;
    // one of the two starts at 0, the other where that one ends
    const bool of_x = first_x ? block >= first_x : block < first_w;
    if (of_x)
        product_tile<256, BJX, 64, 2, 4, kColumns, kRows>(
            x, block - first_x, first_x ? blocks - first_x : first_w, (TIDE_LDS char*)lds);
    else
        product_tile<256, BJW, 64, 2, 4, kColumns, kColumns>(
            w, block - first_w, first_w ? blocks - first_w : first_x, (TIDE_LDS char*)lds);
}

// The sums of a split contraction added up in the splits' order, then the
// epilogue.  Bound by the partial sums' bytes and a launch: 3 splits of 2048 x
// 5120 sums (126 MB) 23 us, 10 of 24 x 5120 (5 MB) 4.2.
constexpr int kJoinThreads = 256;
constexpr int kJoinAhead = 8;  // splits whose loads are in flight together

__global__ __launch_bounds__(kJoinThreads) void join_kernel(Product p) {
    const int64_t per_row = p.partial_pitch / 8;
    const int64_t u = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
    const int64_t j = u / per_row, i = (u - j * per_row) * 8;
    const bool there = j < p.e.J && i < p.e.I;
    float v[8] = {};
    if (there) {
        const float* from = p.partial + j * p.partial_pitch + i;
        const int64_t next = p.e.J * p.partial_pitch;
        for (int s = 0; s < p.splits; s += kJoinAhead) {
            f32x4v lo[kJoinAhead], hi[kJoinAhead];
#pragma unroll
            for (int u = 0; u < kJoinAhead; ++u) {
                const bool have = s + u < p.splits;
                lo[u] = have ? *(const TIDE_GLOBAL_AS f32x4v*)from : (f32x4v)0.0f;
                hi[u] = have ? *(const TIDE_GLOBAL_AS f32x4v*)(from + 4) : (f32x4v)0.0f;
                from += next;
            }
#pragma unroll
            for (int u = 0; u < kJoinAhead; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    v[r] += lo[u][r];
                    v[r + 4] += hi[u][r];
                }
        }
    }
    finish(p.e, i, j, there, v);
}

// ---- forward for one to four tokens -----------------------------------------

// The weight's bytes bound this product, and how fast they come depends on how
// they are asked for: of W's rows of 16 KB, reads of 64 bytes of 16 rows an
// instruction reach 4.7 TB/s, 1 KB of one row an instruction in runs of 1 KB a
// row 5.3, in runs of 4 KB 6.6 (nontemporal; plain loads 0.5 less).  So a
// workgroup takes 8 rows, its 4 waves side by side 4 KB of each at a time; a
// lane multiplies its 8 elements of every row by its 8 elements of each
// token in binary32 and the lanes' sums are added at the end.  28672 x 8192:
// 72 us for one token (6.5 TB/s), 74 for two, 85 for four.  Rows may start
// anywhere.
struct Gemv {
    const uint16_t* x;
    int64_t ldx;
    const uint16_t* w;
    int64_t K;
    Epilogue e;  // I = N, J = T
};

constexpr int kGemvRows = 8;
constexpr int kGemvThreads = 256;

template <int T>
__global__ __launch_bounds__(kGemvThreads, 4) void gemv_kernel(Gemv p) {
    __shared__ float part[kGemvThreads / 64][T][kGemvRows];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n0 = (int64_t)blockIdx.x * kGemvRows;
    const int64_t c = (int64_t)threadIdx.x * 8;
    const uint16_t* w[kGemvRows];
#pragma unroll
    for (int r = 0; r < kGemvRows; ++r) w[r] = p.w + min(n0 + r, p.e.I - 1) * p.K + c;
    const uint16_t* x[T];
#pragma unroll
    for (int t = 0; t < T; ++t) x[t] = p.x + min((int64_t)t, p.e.J - 1) * p.ldx + c;
    float acc[kGemvRows][T] = {};
    // elements k .. k + 7 of the lane's piece, of which the first `seen` do not count
    auto step = [&](int64_t k, int seen) __attribute__((always_inline)) {
        u32x4v wv[kGemvRows], xv[T];
#pragma unroll
        for (int r = 0; r < kGemvRows; ++r) wv[r] = load8_raw<true>(w[r] + k);
#pragma unroll
        for (int t = 0; t < T; ++t) xv[t] = load8_raw(x[t] + k);
#pragma unroll
        for (int r = 0; r < kGemvRows; ++r) {
            float v[8];
            widen(wv[r], v);
#pragma unroll
            for (int t = 0; t < T; ++t) {
                float u[8];
                widen(xv[t], u);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    acc[r][t] = __builtin_fmaf(q < seen ? 0.0f : v[q], q < seen ? 0.0f : u[q], acc[r][t]);
            }
        }
    };
    int64_t k = 0;
#pragma unroll 1
    for (; k + c + 8 <= p.K; k += kGemvThreads * 8) step(k, 0);
    // the one lane whose piece ends inside: the row's last 8 elements, those
    // that the lane before it has had left out
    if (k + c < p.K) step(p.K - 8 - c, (int)(k + c + 8 - p.K));
#pragma unroll
    for (int r = 0; r < kGemvRows; ++r)
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float s = acc[r][t];
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
            if (lane == 0) part[wave][t][r] = s;
        }
    __syncthreads();
    if (threadIdx.x >= T) return;
    float v[kGemvRows];
#pragma unroll
    for (int r = 0; r < kGemvRows; ++r) {
        v[r] = part[0][threadIdx.x][r];
#pragma unroll
        for (int u = 1; u < kGemvThreads / 64; ++u) v[r] += part[u][threadIdx.x][r];
    }
    finish(p.e, n0, threadIdx.x, threadIdx.x < p.e.J, v);
}

// ---- operand preparation -------------------------------------------------

// Rows of `cols` elements copied to rows of `width` (a multiple of 8), the
// rest 0: operands whose rows do not start on 16 bytes, or whose length is
// not a multiple of 8.  (Reading such a weight straight into the matrix
// instructions' registers, without the copy, took 58 us against 22 for 24
// tokens and 1001 x 5121, 401 against 293 for 32 and 28672 x 8191.)
constexpr int kPadThreads = 256;

__global__ __launch_bounds__(kPadThreads) void pad_kernel(const uint16_t* in, int64_t ld,
                                                          int64_t rows, int64_t cols,
                                                          uint16_t* out, int64_t width) {
    const int64_t per_row = width / 8;
    const int64_t u = (int64_t)blockIdx.x * kPadThreads + threadIdx.x;
    const int64_t r = u / per_row, c = (u - r * per_row) * 8;
    if (r >= rows) return;
    float v[8];
    load8(in + r * ld + c, cols - c, v);
    store8(out + r * width + c, 8, v);
}

// dz = dy act'(z) rounded to bf16, rows of `width` elements with zeros behind
// the N-th, and the column sums of dz before the rounding over each chunk of
// rows (one row of `sums` for each chunk).  A lane keeps its 8 columns through
// a quarter of the chunk's rows, so a workgroup reads runs of up to 4 KB of a
// row, and has the loads of kDzRows rows in flight; the quarters' sums meet in
// LDS.  (2048 x 13824 with relu: 29 us, 4.9 TB/s; 33 without
// the quarters, two waves a SIMD.)
//
// The rounding is the matrix instructions': they take bf16.  It makes dx and dW
// off by 2.3e-3 of themselves, root mean square, where the one rounding of their
// own leaves 1.7e-3.  dz in two bf16 parts would keep it and double the products'
// work (2048 x 13824 x 5120: 387 us at the least); dbias, which needs no product,
// sums dz before it.
constexpr int kDzLanes = 256;    // of 8 columns
constexpr int kDzQuarters = 4;
constexpr int kDzRows = 4;
constexpr int64_t kDzOneChunk = 64;

struct DzArgs {
    const uint16_t* dy;
    int64_t ld;
    const uint8_t* z;  // its checkpoint, or NULL (act none)
    uint16_t* dz;      // or NULL: sums only
    int64_t width;
    float* sums;       // or NULL
    uint16_t* dbias;   // the one chunk's sums go there, or NULL
    int64_t T, N, chunk;
    int32_t col_groups;
};

// One lane's columns c .. c + 7 through a chunk; WHOLE: all of them exist.
template <int ACT, bool WHOLE>
__device__ __forceinline__ void dz_lane(const DzArgs& p, int64_t c, int64_t t0, int64_t t1,
                                        float (&sum)[8]) {
    const int64_t pitch = act8_pitch(p.N);
    const uint8_t* scales = p.z + p.T * pitch;
    for (; t0 < t1; t0 += kDzRows) {
        u32x4v y[kDzRows];
        float v[kDzRows][8];
        u32x2 q[kDzRows];
        uint32_t s[kDzRows];
#pragma unroll
        for (int u = 0; u < kDzRows; ++u) {
            const int64_t t = min(t0 + u, t1 - 1);
            const uint16_t* from = p.dy + t * p.ld + c;
            if constexpr (WHOLE)
                y[u] = load8_raw(from);
            else
                load8(from, p.N - c, v[u]);
            if constexpr (ACT != TIDE_ACT_NONE) {
                q[u] = *(const TIDE_GLOBAL_AS u32x2*)(p.z + t * pitch + c);
                s[u] = *(const TIDE_GLOBAL_AS uint8_t*)(scales + (t * pitch + c) / kActBlock);
            }
        }
#pragma unroll
        for (int u = 0; u < kDzRows; ++u) {
            const int64_t t = t0 + u;
            if (t >= t1) break;
            if constexpr (WHOLE) widen(y[u], v[u]);
            if constexpr (ACT != TIDE_ACT_NONE) {
                float z[8];
                act8_unpack8(q[u], act8_scale(s[u]), z);
                apply_slope<ACT>(z, v[u]);
            }
            if constexpr (!WHOLE) {
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (c + r >= p.N) v[u][r] = 0.0f;
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) sum[r] += v[u][r];
            if (p.dz) store8(p.dz + t * p.width + c, 8, v[u]);
        }
    }
}

template <int ACT>
__global__ __launch_bounds__(kDzLanes* kDzQuarters) void dz_kernel(DzArgs p) {
    extern __shared__ __attribute__((aligned(16))) float part[];  // [quarters - 1][lanes * 8]
    const int lanes = blockDim.x / kDzQuarters;
    const int quarter = threadIdx.x / lanes, lane = threadIdx.x - quarter * lanes;
    const int64_t cg = blockIdx.x % p.col_groups, ch = blockIdx.x / p.col_groups;
    const int64_t c = (cg * lanes + lane) * 8;
    const int64_t each = p.chunk / kDzQuarters;
    const int64_t t0 = ch * p.chunk + quarter * each, t1 = min(p.T, t0 + each);
    float sum[8] = {};
    if (c + 8 <= p.N)
        dz_lane<ACT, true>(p, c, t0, t1, sum);
    else if (c < p.N)
        dz_lane<ACT, false>(p, c, t0, t1, sum);
    if (!p.sums && !p.dbias) return;
    if (quarter) {
#pragma unroll
        for (int r = 0; r < 8; ++r) part[((quarter - 1) * 8 + r) * lanes + lane] = sum[r];
    }
    __syncthreads();
    if (quarter) return;
#pragma unroll
    for (int u = 0; u < kDzQuarters - 1; ++u)
#pragma unroll
        for (int r = 0; r < 8; ++r) sum[r] += part[(u * 8 + r) * lanes + lane];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        if (c + r >= p.N) continue;
        if (p.dbias)
            *(TIDE_GLOBAL_AS uint16_t*)(p.dbias + c + r) = to_bf16(sum[r]);
        else
            p.sums[ch * p.N + c + r] = sum[r];
    }
}

// dbias from the chunks' sums: a wave's lane takes a column, the workgroup's
// waves every kDbWaves-th chunk.
constexpr int kDbWaves = 8;

__global__ __launch_bounds__(64 * kDbWaves) void dbias_kernel(const float* sums, int64_t chunks,
                                                              int64_t N, uint16_t* out) {
    __shared__ float part[kDbWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (c < N) {
#pragma unroll 4
        for (int64_t k = wave; k < chunks; k += kDbWaves) s += sums[k * N + c];
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave || c >= N) return;
#pragma unroll
    for (int w = 1; w < kDbWaves; ++w) s += part[w][lane];
    *(TIDE_GLOBAL_AS uint16_t*)(out + c) = to_bf16(s);
}

// ---- host ----------------------------------------------------------------

int64_t partial_floats(const Shape& s, int64_t I, int64_t J) {
    return s.splits > 1 ? s.splits * J * round_up(I, kActBlock) : 0;
}

using ProductKernel = void (*)(Product);

template <int BI, int BJ, int K, int WI, int WJ, int H = 1>
ProductKernel of_kind(Kind k) {
    switch (k) {
        case kForward: return product_kernel<BI, BJ, K, WI, WJ, kRows, kRows, H>;
        case kGradInput: return product_kernel<BI, BJ, K, WI, WJ, kColumns, kRows, H>;
        default: return product_kernel<BI, BJ, K, WI, WJ, BI == 256 ? kColumns : kKept, kColumns, H>;
    }
}

void set_shape(Product* p, const Shape& s, float* partial) {
    p->tiles_i = s.tiles_i;
    p->tiles_j = s.tiles_j;
    p->splits = s.splits;
    p->split_depth = s.split_depth;
    p->partial = partial;
    p->partial_pitch = round_up(p->e.I, kActBlock);
}

tide_status run_join(const Product& p, tide_stream_t stream) {
    if (p.splits == 1) return TIDE_OK;
    return launch(join_kernel, ceil_div(p.e.J * p.partial_pitch / 8, kJoinThreads), kJoinThreads,
                  stream, p);
}

tide_status run_product(Kind kind, Product p, const Shape& s, float* partial,
                        tide_stream_t stream) {
    if (p.e.I == 0 || p.e.J == 0) return TIDE_OK;
    set_shape(&p, s, partial);
    ProductKernel k;
    int threads = 256;
    if (s.bi == 256) {
        k = s.bj == 256   ? of_kind<256, 256, 64, 2, 4>(kind)
            : s.bj == 192 ? of_kind<256, 192, 64, 2, 4>(kind)
                          : of_kind<256, 128, 64, 2, 4>(kind);
        threads = 512;
    } else if (s.bj == 128) {
        k = s.halves == 2 ? of_kind<128, 128, 64, 2, 2, 2>(kind) : of_kind<128, 128, 64, 2, 2>(kind);
        threads = 256 * s.halves;
    } else if (s.bj == 64) {
        k = s.halves == 2 ? of_kind<128, 64, 64, 2, 2, 2>(kind) : of_kind<128, 64, 64, 2, 2>(kind);
        threads = 256 * s.halves;
    } else if (s.bj == 32) {
        k = s.bk == 256     ? product_kernel<128, 32, 256, 4, 1, kRows, kRows>
            : s.halves == 2 ? of_kind<128, 32, 64, 4, 1, 2>(kind)
                            : of_kind<128, 32, 64, 4, 1>(kind);
        threads = 256 * s.halves;
    } else {
        k = s.bk == 256 ? product_kernel<128, 16, 256, 4, 1, kRows, kRows> : of_kind<128, 16, 64, 4, 1>(kind);
    }
    const tide_status st = launch(k, grid_of(s), threads, stream, p);
    return st == TIDE_OK ? run_join(p, stream) : st;
}

// Whether the kernels can read rows of this matrix where they lie.
bool direct(const void* p, int64_t ld, int64_t rows, int64_t cols) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && cols % 8 == 0 && (rows <= 1 || ld % 8 == 0);
}

tide_status pad(const void* in, int64_t ld, int64_t rows, int64_t cols, uint16_t* out,
                tide_stream_t stream) {
    const int64_t width = round_up(cols, 8);
    return launch(pad_kernel, ceil_div(rows * (width / 8), kPadThreads), kPadThreads, stream,
                  static_cast<const uint16_t*>(in), ld, rows, cols, out, width);
}

// An operand: the matrix itself, or its copy in the workspace.
struct Source {
    const void* p;
    int64_t ld, rows, cols;
    uint16_t* copy = nullptr;
    bool copied = false;
    void plan(Carver& c) {
        copied = rows > 0 && cols > 0 && !direct(p, ld, rows, cols);
        if (copied) copy = c.take<uint16_t>(rows * round_up(cols, 8));
    }
    tide_status fill(tide_stream_t stream) const {
        return copied ? pad(p, ld, rows, cols, copy, stream) : TIDE_OK;
    }
    // `count` is what the tile loop calls it: the rows, or the columns
    Operand operand(bool columns) const {
        const int64_t width = round_up(cols, 8);
        Operand o;
        o.p = copied ? copy : p;
        o.ld = copied || rows <= 1 ? width : ld;
        o.count = columns ? width : rows;
        o.depth = columns ? rows : width;
        return o;
    }
};

tide_status check_dims(int64_t T, int64_t N, int64_t K, int32_t act, int32_t reserved) {
    if (T < 0 || N < 0 || K < 0 || act < TIDE_ACT_NONE || act > TIDE_ACT_SILU || reserved != 0)
        return TIDE_EINVAL;
    if (T > kMaxTokens || N > kMaxWidth || K > kMaxWidth) return TIDE_EUNSUPPORTED;
    if (T * N > kMaxElements || T * K > kMaxElements || N * K > kMaxElements)
        return TIDE_EUNSUPPORTED;
    return TIDE_OK;
}

// ---- forward -------------------------------------------------------------

struct ForwardPlan {
    bool gemv;
    Source x, w;
    Shape shape;
    float* partial;
    int64_t bytes;
};

tide_status check_forward(const tide_linear_forward_args& a) {
    TIDE_TRY(check_dims(a.tokens, a.out_features, a.in_features, a.act, a.reserved));
    const int64_t T = a.tokens, N = a.out_features, K = a.in_features;
    if (T == 0 || N == 0) return TIDE_OK;
    TIDE_TRY(check_rows(a.x, a.ldx, T, K));
    TIDE_TRY(check_rows(a.weight, K, N, K));
    if (a.bias) TIDE_TRY(check_rows(a.bias, N, 1, N));
    if (a.residual) TIDE_TRY(check_rows(a.residual, a.ldr, T, N));
    TIDE_TRY(check_rows(a.y, a.ldy, T, N));
    if (a.z_kept) TIDE_TRY(check_kept(a.z_kept, T, N));
    return TIDE_OK;
}

int forward_extents(const tide_linear_forward_args& a, Extent* in, Extent* out) {
    const int64_t T = a.tokens, N = a.out_features, K = a.in_features;
    const bool in_place = a.residual == a.y && (T <= 1 || a.ldr == a.ldy);
    in[0] = rows_extent(a.x, a.ldx, T, K);
    in[1] = rows_extent(a.weight, K, N, K);
    in[2] = rows_extent(a.bias, N, 1, N);
    in[3] = in_place ? Extent() : rows_extent(a.residual, a.ldr, T, N);
    out[0] = rows_extent(a.y, a.ldy, T, N);
    out[1] = bytes_extent(a.z_kept, act8_bytes(T, N));
    return 4;
}

ForwardPlan plan_forward(const tide_linear_forward_args& a, void* ws) {
    ForwardPlan f;
    Carver c{static_cast<char*>(ws)};
    const int64_t T = a.tokens, N = a.out_features, K = a.in_features;
    f.gemv = forward_by_rows(T, N, K, a.z_kept != nullptr,
                             direct(a.x, a.ldx, T, K) && direct(a.weight, K, N, K));
    f.bytes = 0;
    if (f.gemv) return f;
    f.x = {a.x, a.ldx, T, K};
    f.w = {a.weight, K, N, K};
    f.x.plan(c);
    f.w.plan(c);
    f.shape = choose(kForward, N, T, round_up(K, 8));
    f.partial = c.take<float>(partial_floats(f.shape, N, T));
    f.bytes = c.used;
    return f;
}

}  // namespace

extern "C" tide_status tide_linear_forward_workspace(const tide_linear_forward_args* args,
                                                     size_t* bytes) {
    if (!args || !bytes) return TIDE_EINVAL;
    TIDE_TRY(check_forward(*args));
    *bytes = args->tokens && args->out_features ? (size_t)plan_forward(*args, nullptr).bytes : 0;
    return TIDE_OK;
}

extern "C" tide_status tide_linear_forward(const tide_linear_forward_args* args, void* workspace,
                                           size_t workspace_bytes, tide_stream_t stream) {
    if (!args) return TIDE_EINVAL;
    const tide_linear_forward_args& a = *args;
    TIDE_TRY(check_forward(a));
    const int64_t T = a.tokens, N = a.out_features, K = a.in_features;
    if (T == 0 || N == 0) return TIDE_OK;
    Extent ext[6];
    const int n_in = forward_extents(a, ext, ext + 4);
    TIDE_TRY(check_apart(ext, n_in, ext + 4, 2));
    const ForwardPlan f = plan_forward(a, workspace);
    TIDE_TRY(check_workspace(workspace, workspace_bytes, f.bytes, ext, 6));
    TIDE_TRY(check_stream_device(stream));
    Epilogue e = {};
    e.I = N;
    e.J = T;
    e.out = static_cast<uint16_t*>(a.y);
    e.ldo = a.ldy;
    e.bias = static_cast<const uint16_t*>(a.bias);
    e.res = static_cast<const uint16_t*>(a.residual);
    e.ldr = a.ldr;
    e.kept = static_cast<uint8_t*>(a.z_kept);
    e.act = a.act;
    if (f.gemv) {
        const Gemv gemv = {static_cast<const uint16_t*>(a.x), T > 1 ? a.ldx : K,
                           static_cast<const uint16_t*>(a.weight), K, e};
        return launch(T == 1 ? gemv_kernel<1> : T == 2 ? gemv_kernel<2> : gemv_kernel<4>,
                      ceil_div(N, kGemvRows), kGemvThreads, stream, gemv);
    }
    TIDE_TRY(f.x.fill(stream));
    TIDE_TRY(f.w.fill(stream));
    Product p = {};
    p.A = f.w.operand(false);
    p.B = f.x.operand(false);
    p.depth = round_up(K, 8);
    p.e = e;
    return run_product(kForward, p, f.shape, f.partial, stream);
}

// ---- backward ------------------------------------------------------------

namespace {

struct BackwardPlan {
    bool make_dz;       // dz is written (to the workspace), not dy itself
    bool pair = false;  // dx and dW share a launch
    bool in_first = false;
    int64_t width;      // of dz's rows there
    int dz_lanes;
    int64_t dz_groups, chunk, chunks;
    Source w;
    uint16_t* dz = nullptr;
    float* sums = nullptr;
    uint16_t* x = nullptr;
    Shape in_shape, w_shape;
    float* partial = nullptr;
    int64_t bytes;
};

tide_status check_backward(const tide_linear_backward_args& a) {
    TIDE_TRY(check_dims(a.tokens, a.out_features, a.in_features, a.act, a.reserved));
    const int64_t T = a.tokens, N = a.out_features, K = a.in_features;
    if (!a.dx && !a.dweight && !a.dbias) return TIDE_OK;
    TIDE_TRY(check_rows(a.dy, a.lddy, T, N));
    if (a.act != TIDE_ACT_NONE) TIDE_TRY(check_kept(a.z_kept, T, N));
    if (a.dx) {
        TIDE_TRY(check_rows(a.weight, K, N, K));
        TIDE_TRY(check_rows(a.dx, a.lddx, T, K));
    }
    if (a.dweight) {
        TIDE_TRY(check_kept(a.x_kept, T, K));
        TIDE_TRY(check_rows(a.dweight, K, N, K));
    }
    if (a.dbias) TIDE_TRY(check_rows(a.dbias, N, 1, N));
    return TIDE_OK;
}

using PairKernel = void (*)(Product, Product, int32_t);

template <int H>
PairKernel pair_of(int bj) {
    return bj == 128  ? pair_kernel<128, 2, 2, H>
           : bj == 64 ? pair_kernel<64, 2, 2, H>
           : bj == 32 ? pair_kernel<32, 4, 1, H>
                      : pair_kernel<16, 4, 1, H>;
}

using DzKernel = void (*)(DzArgs);

DzKernel dz_kernel_of(int32_t act) {
    switch (act) {
        case TIDE_ACT_RELU: return dz_kernel<TIDE_ACT_RELU>;
        case TIDE_ACT_GELU: return dz_kernel<TIDE_ACT_GELU>;
        case TIDE_ACT_GELU_TANH: return dz_kernel<TIDE_ACT_GELU_TANH>;
        case TIDE_ACT_SILU: return dz_kernel<TIDE_ACT_SILU>;
        default: return dz_kernel<TIDE_ACT_NONE>;
    }
}

BackwardPlan plan_backward(const tide_linear_backward_args& a, void* ws) {
    BackwardPlan b;
    Carver c{static_cast<char*>(ws)};
    const int64_t T = a.tokens, N = a.out_features, K = a.in_features;
    const bool products = (a.dx && T && K) || (a.dweight && N && K);
    b.make_dz = products && T && N && (a.act != TIDE_ACT_NONE || !direct(a.dy, a.lddy, T, N));
    b.width = round_up(N, 8);
    if (b.make_dz) b.dz = c.take<uint16_t>(T * b.width);
    // Chunks of rows: about 512 workgroups of 16 waves, but where the column
    // sums are wanted at least 32 rows, so that the partial sums stay few
    const int64_t n = std::max<int64_t>(N, 1);
    b.dz_lanes = (int)std::min<int64_t>(kDzLanes, round_up(ceil_div(n, 8), 64));
    b.dz_groups = ceil_div(n, 8 * b.dz_lanes);
    b.chunk = std::max<int64_t>(a.dbias ? 32 : kDzQuarters,
                                ceil_div(T, std::max<int64_t>(1, 512 / b.dz_groups)));
    b.chunk = round_up(b.chunk, kDzQuarters);
    // few rows are one chunk, whose sums are dbias
    if (a.dbias && T <= kDzOneChunk) b.chunk = round_up(std::max<int64_t>(T, 1), kDzQuarters);
    b.chunks = ceil_div(T, b.chunk);
    if (a.dbias && b.chunks != 1) b.sums = c.take<float>(b.chunks * N);
    b.w = {a.weight, K, a.dx && T ? N : 0, K};
    b.w.plan(c);
    const Gradients g = choose_gradients(T, N, K, a.dx && T && N && K, a.dweight && T && N && K);
    b.in_shape = g.in;
    b.w_shape = g.weight;
    b.pair = g.pair;
    b.in_first = g.in_first;
    // the 256-wide tiles read x from here, widened (tile_product.h)
    if (a.dweight && N && b.w_shape.bi == 256) b.x = c.take<uint16_t>(T * act8_pitch(K));
    int64_t floats = 0;
    if (a.dx) floats = std::max(floats, partial_floats(b.in_shape, K, T));
    if (a.dweight) floats = std::max(floats, partial_floats(b.w_shape, K, N));
    b.partial = c.take<float>(floats);
    b.bytes = c.used;
    return b;
}

}  // namespace

extern "C" tide_status tide_linear_backward_workspace(const tide_linear_backward_args* args,
                                                      size_t* bytes) {
    if (!args || !bytes) return TIDE_EINVAL;
    TIDE_TRY(check_backward(*args));
    *bytes = (size_t)plan_backward(*args, nullptr).bytes;
    return TIDE_OK;
}

extern "C" tide_status tide_linear_backward(const tide_linear_backward_args* args, void* workspace,
                                            size_t workspace_bytes, tide_stream_t stream) {
    if (!args) return TIDE_EINVAL;
    const tide_linear_backward_args& a = *args;
    TIDE_TRY(check_backward(a));
    if (!a.dx && !a.dweight && !a.dbias) return TIDE_OK;
    const int64_t T = a.tokens, N = a.out_features, K = a.in_features;
    Extent ext[7] = {rows_extent(a.dy, a.lddy, T, N),
                     a.dx ? rows_extent(a.weight, K, N, K) : Extent(),
                     a.dweight ? bytes_extent(a.x_kept, act8_bytes(T, K)) : Extent(),
                     a.act != TIDE_ACT_NONE ? bytes_extent(a.z_kept, act8_bytes(T, N)) : Extent(),
                     rows_extent(a.dx, a.lddx, T, K),
                     rows_extent(a.dweight, K, N, K),
                     rows_extent(a.dbias, N, 1, N)};
    TIDE_TRY(check_apart(ext, 4, ext + 4, 3));
    const BackwardPlan b = plan_backward(a, workspace);
    TIDE_TRY(check_workspace(workspace, workspace_bytes, b.bytes, ext, 7));
    TIDE_TRY(check_stream_device(stream));

    if (T && N && (b.make_dz || a.dbias)) {
        DzArgs d = {};
        d.dy = static_cast<const uint16_t*>(a.dy);
        d.ld = a.lddy;
        d.z = a.act != TIDE_ACT_NONE ? static_cast<const uint8_t*>(a.z_kept) : nullptr;
        d.dz = b.make_dz ? b.dz : nullptr;
        d.width = b.width;
        d.sums = b.sums;
        d.dbias = b.chunks == 1 ? static_cast<uint16_t*>(a.dbias) : nullptr;
        d.T = T;
        d.N = N;
        d.chunk = b.chunk;
        d.col_groups = (int32_t)b.dz_groups;
        const int threads = b.dz_lanes * kDzQuarters;
        const unsigned lds = a.dbias ? (kDzQuarters - 1) * b.dz_lanes * 8 * sizeof(float) : 0;
        TIDE_TRY(launch_lds(dz_kernel_of(a.act), b.dz_groups * b.chunks, threads, lds, stream, d));
    }
    if (a.dbias && N && b.chunks != 1)
        TIDE_TRY(launch(dbias_kernel, ceil_div(N, 64), 64 * kDbWaves, stream,
                        static_cast<const float*>(b.sums), b.chunks, N,
                        static_cast<uint16_t*>(a.dbias)));
    if (K == 0) return TIDE_OK;

    Source dz = {b.make_dz ? b.dz : a.dy, b.make_dz ? b.width : a.lddy, T, b.make_dz ? b.width : N};
    Product x = {}, w = {};
    if (a.dx && T) {
        TIDE_TRY(b.w.fill(stream));
        x.A = b.w.operand(true);
        x.B = dz.operand(false);
        x.depth = b.width;  // dz's columns behind the N-th are 0
        x.e.I = K;
        x.e.J = T;
        x.e.out = static_cast<uint16_t*>(a.dx);
        x.e.ldo = a.lddx;
    }
    if (a.dweight && N) {
        w.A = {a.x_kept, act8_pitch(K), act8_pitch(K), T};
        if (b.w_shape.bi == 256) {
            TIDE_TRY(act8_unpack_into(a.x_kept, T, K, b.x, act8_pitch(K), false, stream));
            w.A.p = b.x;
        }
        w.B = dz.operand(true);
        w.depth = T;
        w.e.I = K;
        w.e.J = N;
        w.e.out = static_cast<uint16_t*>(a.dweight);
        w.e.ldo = K;
    }
    if (b.pair) {
        set_shape(&w, b.w_shape, nullptr);
        set_shape(&x, b.in_shape, b.partial);
        const int64_t n_w = grid_of(b.w_shape), n_x = grid_of(b.in_shape);
        if (b.w_shape.bi == 256) {
            const bool x_first = b.in_first;
            auto wide = b.w_shape.bj == 256
                            ? b.in_shape.bj == 256 ? wide_pair_kernel<256, 256> : wide_pair_kernel<256, 192>
                            : b.in_shape.bj == 256 ? wide_pair_kernel<192, 256> : wide_pair_kernel<192, 192>;
            return launch(wide, n_w + n_x, 512, stream, w, x, (int32_t)(x_first ? n_x : 0),
                          (int32_t)(x_first ? 0 : n_w));
        }
        const int halves = n_w + n_x <= kCus ? 2 : 1;
        auto k = halves == 2 ? pair_of<2>(b.in_shape.bj) : pair_of<1>(b.in_shape.bj);
        TIDE_TRY(launch(k, n_w + n_x, 256 * halves, stream, w, x, (int32_t)n_w));
        return run_join(x, stream);
    }
    if (a.dx && T) TIDE_TRY(run_product(kGradInput, x, b.in_shape, b.partial, stream));
    if (a.dweight && N) TIDE_TRY(run_product(kGradWeight, w, b.w_shape, b.partial, stream));
    return TIDE_OK;
}
