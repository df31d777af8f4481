// product.h -- a layer product around its tile loop (tile_product.h): workgroup
// to tile, split contractions, epilogues, the form for few tokens, operands
// copied to padded rows, and the launches.  Shared by linear.hip and gated.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "act8.h"
#include "activation.h"
#include "bf16_io.h"
#include "linear_check.h"
#include "product_shape.h"
#include "tide.h"
#include "tile_product.h"

namespace tide {
namespace {

// ---- epilogue ------------------------------------------------------------

// What happens to a finished sum at output column i of row j.
struct Epilogue {
    static constexpr bool kPairs = false;  // A is two matrices' rows in turn
    static constexpr bool kNarrow = true;  // J may be 64 or less
    int64_t I, J;
    uint16_t* out;
    int64_t ldo;
    const uint16_t* bias;
    const uint16_t* res;
    int64_t ldr;
    uint8_t* kept;  // the checkpoint of z
    int32_t act;
    __device__ __forceinline__ int64_t columns() const { return I; }
};

// A lane's 8 of 32 consecutive columns, i .. i + 7 of row j, of which the first n
// exist, into a checkpoint of J rows of I columns; the four lanes of a block
// together.
__device__ __forceinline__ void keep_unit(uint8_t* kept, int64_t I, int64_t J, int64_t i, int64_t j,
                                          int64_t n, const float (&v)[8]) {
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
    const int64_t pitch = act8_pitch(I);
    if (j < J && i < pitch) {
        *(TIDE_GLOBAL_AS u32x2*)(kept + j * pitch + i) = q;
        if (i % kActBlock == 0)
            *(TIDE_GLOBAL_AS uint8_t*)(kept + J * pitch + (j * pitch + i) / kActBlock) =
                (uint8_t)(x + 127);
    }
}

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
    if (e.kept) keep_unit(e.kept, e.I, e.J, i, j, n, v);
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

// E: what becomes of the finished sums; OA: what the operand A is.
template <typename E, typename OA = Operand>
struct Product {
    OA A;
    Operand B;
    int64_t depth;        // contraction elements
    int64_t split_depth;  // of one split (a multiple of kSplitUnit)
    int32_t tiles_i, tiles_j, splits;
    float* partial;       // [splits][J][pitch] sums where splits > 1
    int64_t partial_pitch;
    E e;
};

template <typename P>
constexpr bool kPairOfA = std::is_same<decltype(P::A), PairOperand>::value;
template <typename P>
constexpr bool kPairsOut = decltype(P::e)::kPairs;

// Workgroup -> (tile, split).  Consecutive workgroups go to the 8 XCDs in
// turn, so each XCD is given a run of consecutive tiles of its own, and tiles
// are numbered in bands of kBand tiles of j (all of i inside a band): the
// tiles an XCD works on together share rows of both operands in its L2.
constexpr int kXcdCount = 8;
constexpr int kBand = 4;

template <typename P>
__device__ __forceinline__ void tile_at(const P& p, uint32_t b, uint32_t total, int* ti,
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

// Forms whose tiles are a ring (tile_product.h), and how many: as many as 160 KB
// hold.
constexpr bool in_ring(Layout a, int h) { return h == 2 && (a == kPairRows || a == kPairRowsOnce); }
template <int BI, int BJ, int K>
constexpr int kRing = (160 << 10) / ((BI + BJ) * K * 2);
template <int BI, int BJ, int K, Layout CA, int H>
constexpr int kTileLds = in_ring(CA, H) ? kRing<BI, BJ, K> * (BI + BJ) * K * 2 : kProductLds<BI, BJ, K> * H;

// The tile of workgroup `block` of `blocks`.  H = 2: the contraction in two
// halves, each by WI * WJ waves with tiles in LDS of their own (in a ring: half of
// each tile, which they share), whose sums are added in
// LDS; each set of waves then finishes half of the tile.
template <int BI, int BJ, int K, int WI, int WJ, Layout CA, Layout CB, int H, typename P>
__device__ __forceinline__ void product_tile(const P& p, uint32_t block, uint32_t blocks,
                                             TIDE_LDS char* lds) {
    constexpr int TI = BI / WI / 16, TJ = BJ / WJ / 16;
    static_assert(TI % (kPairsOut<P> ? 4 : 2) == 0, "a wave holds whole checkpoint blocks");
    int ti, tj, sp;
    tile_at(p, block, blocks, &ti, &tj, &sp);
    const int64_t i0 = (int64_t)ti * BI, j0 = (int64_t)tj * BJ;
    f32x4v acc[TI][TJ];
    const int64_t k0 = sp * p.split_depth, k1 = min(p.depth, (sp + 1) * p.split_depth);
    constexpr int kLds = kTileLds<BI, BJ, K, CA, H>;
    if constexpr (in_ring(CA, H))
        ring_loop<BI, BJ, K, WI, WJ, CA, CB, kRing<BI, BJ, K>>(p.A, p.B, p.depth, k0, k1, i0, j0, lds, acc);
    else
        tile_loop<BI, BJ, K, WI, WJ, CA, CB, H>(p.A, p.B, p.depth, k0, k1, i0, j0, lds, acc);

    // The accumulators pass through LDS, 16 rows of a wave at a time, so that
    // each lane ends with 8 consecutive columns and a row's stores are whole
    // lines.  The row pitch's extra 4 floats keep the writes off each other's
    // banks.
    constexpr int kRow = TI * 16, kPitch = kRow + 4, kLanes = kRow / 8;
    constexpr int kStaging = WI * WJ * H * 16 * kPitch * 4;
    constexpr int kDone = H == 2 && TJ > 1 ? TJ / 2 : TJ;  // 16-row pieces that a wave finishes
    static_assert(H == 1 || TJ == 1 || TJ % 2 == 0, "the halves share the tile");
    static_assert(kStaging <= kLds, "the staging fits");
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
        static_assert(kStaging + 2 * WI * WJ * kWave <= kLds, "both fit");
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
        for (int r = 0; r < (kPairsOut<P> && p.splits == 1 ? 0 : 16); r += 64 / kLanes) {
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
            if constexpr (!kPairsOut<P>) {
                float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                finish(p.e, iw, j, there, v);
            }
        }
        if constexpr (kPairsOut<P>) {
            // 16 columns of the first matrix lie before the same 16 of the second
            constexpr int kUnits = kRow / 16;
            const int unit = lane % kUnits;
            const int64_t n = (i0 + (wave / WJ) * kRow) / 2 + unit * 8;
            const int64_t j1 = j0 + ((wave % WJ) * TJ + half * kDone + y) * 16 + lane / kUnits;
#pragma unroll 1
            for (int r = 0; r < (p.splits == 1 ? 16 : 0); r += 64 / kUnits) {
                const TIDE_LDS float* row = mine + (r + lane / kUnits) * kPitch + (unit / 2) * 32 + unit % 2 * 8;
                float a[8], b[8];
#pragma unroll
                for (int k = 0; k < 8; k += 4) {
                    const f32x4v va = *(const TIDE_LDS f32x4v*)(row + k);
                    const f32x4v vb = *(const TIDE_LDS f32x4v*)(row + 16 + k);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        a[k + q] = va[q];
                        b[k + q] = vb[q];
                    }
                }
                finish(p.e, n, j1 + r, a, b);
            }
        }
        wave_lds_order();
    }
}

template <int BI, int BJ, int K, int WI, int WJ, Layout CA, Layout CB, int H, typename P>
__global__ __launch_bounds__(WI* WJ * 64 * H, BI == 256 ? 2 : 1) void product_kernel(P p) {
    __shared__ __attribute__((aligned(1024))) char lds[kTileLds<BI, BJ, K, CA, H>];
    product_tile<BI, BJ, K, WI, WJ, CA, CB, H>(p, blockIdx.x, gridDim.x, (TIDE_LDS char*)lds);
}

// dx and dW in one launch, for shapes too small to fill the chip one after the
// other (77 x 768 x 2048: 13.2 us for both, 7.6, 3.0 and 8.0 for dx, its join
// and dW): the first `n_w` workgroups take dW's tiles, the others dx's.  H = 2
// where each has a compute unit to itself (the same call 14.7 us with dz's
// launch, 16.0 with one set of waves; 300 x 1024 x 1024 16.3, 18.5).
template <int BJ, int WI, int WJ, int H, typename PW, typename PX>
__global__ __launch_bounds__(256 * H) void pair_kernel(PW w, PX x, int32_t n_w) {
    __shared__ __attribute__((aligned(1024))) char lds[kProductLds<128, 128, 64> * H];
    if ((int)blockIdx.x < n_w)
        product_tile<128, 128, 64, 2, 2, kKept, kColumns, H>(w, blockIdx.x, n_w,
                                                             (TIDE_LDS char*)lds);
    else
        product_tile<128, BJ, 64, WI, WJ, kPairOfA<PX> ? kPairColumns : kColumns, kRows, H>(x, blockIdx.x - n_w, gridDim.x - n_w,
                                                              (TIDE_LDS char*)lds);
}

// The same with 256-wide tiles, one workgroup a compute unit, the product of the
// longer tiles first: where its tiles do not fill whole rounds of the chip the
// other's fill the gaps (2048 x 13824 x 5120: 160 tiles of dx of 342 us and 1080 of
// dW of 57 on 256 compute units, 460 us for both, 570 one after the other).
template <int BJW, int BJX, typename PW, typename PX>
__global__ __launch_bounds__(512, 2) void wide_pair_kernel(PW w, PX x, int32_t first_w,
                                                           int32_t first_x) {
    constexpr int kBj = BJW > BJX ? BJW : BJX;
    __shared__ __attribute__((aligned(1024))) char lds[kProductLds<256, kBj, 64>];
    const int block = blockIdx.x, blocks = gridDim.x;
    // one of the two starts at 0, the other where that one ends
    const bool of_x = first_x ? block >= first_x : block < first_w;
    if (of_x)
        product_tile<256, BJX, 64, 2, 4, kPairOfA<PX> ? kPairColumns : kColumns, kRows, 1>(
            x, block - first_x, first_x ? blocks - first_x : first_w, (TIDE_LDS char*)lds);
    else
        product_tile<256, BJW, 64, 2, 4, kColumns, kColumns, 1>(
            w, block - first_w, first_w ? blocks - first_w : first_x, (TIDE_LDS char*)lds);
}

// The sums of a split contraction added up in the splits' order, then the
// epilogue.  Bound by the partial sums' bytes and a launch: 3 splits of 2048 x
// 5120 sums (126 MB) 23 us, 10 of 24 x 5120 (5 MB) 4.2.
constexpr int kJoinThreads = 256;
constexpr int kJoinAhead = 8;  // splits whose loads are in flight together

// Eight columns of the splits' sums of a row.
template <typename P>
__device__ __forceinline__ void join_sums(const P& p, int64_t j, int64_t i, float (&v)[8]) {
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

template <typename P>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(P p) {
    if constexpr (kPairsOut<P>) {
        const int64_t per_row = act8_pitch(p.e.N) / 8;
        const int64_t u = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
        const int64_t j = u / per_row, n = (u - j * per_row) * 8;
        float a[8] = {}, b[8] = {};
        if (j < p.e.J && n < p.e.N) {
            const int64_t i = n / 16 * 32 + n % 16;
            join_sums(p, j, i, a);
            join_sums(p, j, i + 16, b);
        }
        finish(p.e, n, j, a, b);
    } else {
        const int64_t per_row = p.partial_pitch / 8;
        const int64_t u = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
        const int64_t j = u / per_row, i = (u - j * per_row) * 8;
        const bool there = j < p.e.J && i < p.e.I;
        float v[8] = {};
        if (there) join_sums(p, j, i, v);
        finish(p.e, i, j, there, v);
    }
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
//
// Of two matrices a workgroup takes four rows each.
template <typename E>
struct Gemv {
    const uint16_t* x;
    int64_t ldx;
    const uint16_t *w, *w2;  // w2: of two matrices
    int64_t K;
    E e;  // I = N, J = T
};

constexpr int kGemvRows = 8;
constexpr int kGemvThreads = 256;

template <int T, typename E>
__global__ __launch_bounds__(kGemvThreads, 4) void gemv_kernel(Gemv<E> p) {
    constexpr int kColumns = E::kPairs ? kGemvRows / 2 : kGemvRows;  // of the output
    __shared__ float part[kGemvThreads / 64][T][kGemvRows];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n0 = (int64_t)blockIdx.x * kColumns;
    const int64_t c = (int64_t)threadIdx.x * 8;
    const uint16_t* w[kGemvRows];
#pragma unroll
    for (int r = 0; r < kGemvRows; ++r)
        w[r] = (r < kColumns ? p.w : p.w2) + min(n0 + r % kColumns, p.e.columns() - 1) * p.K + c;
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
    if constexpr (E::kPairs)
        finish4(p.e, n0, threadIdx.x, v);
    else
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

// ---- host ----------------------------------------------------------------

inline int64_t partial_floats(const Shape& s, int64_t I, int64_t J) {
    return s.splits > 1 ? s.splits * J * round_up(I, kActBlock) : 0;
}

template <Kind KIND, typename P, int BI, int BJ, int K, int WI, int WJ, int H = 1>
void (*kernel_of())(P) {
    if constexpr (KIND == kForward)
        return product_kernel<BI, BJ, K, WI, WJ, kPairOfA<P> ? kPairRows : kRows, kRows, H, P>;
    else if constexpr (KIND == kGradInput)
        return product_kernel<BI, BJ, K, WI, WJ, kPairOfA<P> ? kPairColumns : kColumns, kRows, H, P>;
    else
        return product_kernel<BI, BJ, K, WI, WJ, BI == 256 ? kColumns : kKept, kColumns, H, P>;
}

// The forms of 128 rows of two matrices' rows in turn: a wave takes 64 of them, so
// that it holds whole blocks of the output's checkpoints.
template <typename P, int BJ, int K, int WJ>
void (*ring_of(bool once))(P) {
    return once ? product_kernel<128, BJ, K, 2, WJ, kPairRowsOnce, kRows, 2, P>
                : product_kernel<128, BJ, K, 2, WJ, kPairRows, kRows, 2, P>;
}
template <typename P>
void (*pairs_of(const Shape& s, bool once, int* threads))(P) {
    *threads = 512;
    if (s.bj == 128 && s.halves == 2) return ring_of<P, 128, 64, 2>(once);
    if (s.bj == 64) return ring_of<P, 64, 128, 2>(once);
    if (s.bj == 32 && s.halves == 2) return ring_of<P, 32, 128, 2>(once);
    *threads = 256;
    if (s.bj == 128) return kernel_of<kForward, P, 128, 128, 64, 2, 2>();
    if (s.bj == 32) return kernel_of<kForward, P, 128, 32, 256, 2, 2>();
    return ring_of<P, 16, 128, 1>(once);
}

template <typename P>
void set_shape(P* p, const Shape& s, float* partial) {
    p->tiles_i = s.tiles_i;
    p->tiles_j = s.tiles_j;
    p->splits = s.splits;
    p->split_depth = s.split_depth;
    p->partial = partial;
    p->partial_pitch = round_up(p->e.I, kActBlock);
}

template <typename P>
tide_status run_join(const P& p, tide_stream_t stream) {
    if (p.splits == 1) return TIDE_OK;
    int64_t per_row;
    if constexpr (kPairsOut<P>)
        per_row = act8_pitch(p.e.N) / 8;
    else
        per_row = p.partial_pitch / 8;
    return launch(join_kernel<P>, ceil_div(p.e.J * per_row, kJoinThreads), kJoinThreads, stream, p);
}

template <Kind KIND, typename P>
tide_status run_product(P p, const Shape& s, float* partial, tide_stream_t stream) {
    if (p.e.I == 0 || p.e.J == 0) return TIDE_OK;
    set_shape(&p, s, partial);
    void (*k)(P);
    int threads = 256 * s.halves;
    if (s.bi == 256) {
        k = s.bj == 256   ? kernel_of<KIND, P, 256, 256, 64, 2, 4>()
            : s.bj == 192 ? kernel_of<KIND, P, 256, 192, 64, 2, 4>()
                          : kernel_of<KIND, P, 256, 128, 64, 2, 4>();
        threads = 512;
    } else if constexpr (kPairsOut<P>) {
        k = pairs_of<P>(s, past_the_cache(p.e.I, p.depth) && s.tiles_j == 1, &threads);
    } else if (s.bj == 128) {
        k = s.halves == 2 ? kernel_of<KIND, P, 128, 128, 64, 2, 2, 2>()
                          : kernel_of<KIND, P, 128, 128, 64, 2, 2>();
    } else if constexpr (!decltype(P::e)::kNarrow) {
        return TIDE_EINVAL;  // choose() takes no such tile
    } else if (s.bj == 64) {
        k = s.halves == 2 ? kernel_of<KIND, P, 128, 64, 64, 2, 2, 2>()
                          : kernel_of<KIND, P, 128, 64, 64, 2, 2>();
    } else if (s.bj == 32) {
        k = s.halves == 2 ? kernel_of<KIND, P, 128, 32, 64, 4, 1, 2>()
                          : kernel_of<KIND, P, 128, 32, 64, 4, 1>();
        if constexpr (KIND == kForward)
            if (s.bk == 256) k = kernel_of<KIND, P, 128, 32, 256, 4, 1>();
    } else {
        k = kernel_of<KIND, P, 128, 16, 64, 4, 1>();
        if constexpr (KIND == kForward)
            if (s.bk == 256) k = kernel_of<KIND, P, 128, 16, 256, 4, 1>();
    }
    const tide_status st = launch(k, grid_of(s), threads, stream, p);
    return st == TIDE_OK ? run_join(p, stream) : st;
}

// dx and dW, x and w, as their shapes say: in one launch or one after the other.
template <int H, typename PW, typename PX>
void (*pair_of(int bj))(PW, PX, int32_t) {
    return bj == 128  ? pair_kernel<128, 2, 2, H, PW, PX>
           : bj == 64 ? pair_kernel<64, 2, 2, H, PW, PX>
           : bj == 32 ? pair_kernel<32, 4, 1, H, PW, PX>
                      : pair_kernel<16, 4, 1, H, PW, PX>;
}

template <typename PW, typename PX>
tide_status run_gradients(const Gradients& g, PW w, bool want_w, PX x, bool want_x, float* partial,
                          tide_stream_t stream) {
    if (g.pair) {
        set_shape(&w, g.weight, nullptr);
        set_shape(&x, g.in, partial);
        const int64_t n_w = grid_of(g.weight), n_x = grid_of(g.in);
        if (g.weight.bi == 256) {
            const bool x_first = g.in_first;
            auto wide = g.weight.bj == 256 ? g.in.bj == 256 ? wide_pair_kernel<256, 256, PW, PX>
                                                            : wide_pair_kernel<256, 192, PW, PX>
                        : g.in.bj == 256   ? wide_pair_kernel<192, 256, PW, PX>
                                           : wide_pair_kernel<192, 192, PW, PX>;
            TIDE_TRY(launch(wide, n_w + n_x, 512, stream, w, x, (int32_t)(x_first ? n_x : 0),
                            (int32_t)(x_first ? 0 : n_w)));
            return run_join(x, stream);
        }
        const int halves = n_w + n_x <= kCus ? 2 : 1;
        auto k = halves == 2 ? pair_of<2, PW, PX>(g.in.bj) : pair_of<1, PW, PX>(g.in.bj);
        TIDE_TRY(launch(k, n_w + n_x, 256 * halves, stream, w, x, (int32_t)n_w));
        return run_join(x, stream);
    }
    if (want_x) TIDE_TRY(run_product<kGradInput>(x, g.in, partial, stream));
    if (want_w) TIDE_TRY(run_product<kGradWeight>(w, g.weight, partial, stream));
    return TIDE_OK;
}

// Whether the kernels can read rows of this matrix where they lie.
inline bool direct(const void* p, int64_t ld, int64_t rows, int64_t cols) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && cols % 8 == 0 && (rows <= 1 || ld % 8 == 0);
}

inline tide_status pad(const void* in, int64_t ld, int64_t rows, int64_t cols, uint16_t* out,
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

}  // namespace
}  // namespace tide
