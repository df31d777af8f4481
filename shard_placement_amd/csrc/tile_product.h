// tile_product.h -- the matrix-core tile loop behind the layer products
// (linear.hip), for gfx950.
//
// One workgroup computes D[i, j] = sum over k of A[i, k] B[j, k] for a BI x BJ
// tile.  i is always the index along which the product's output is
// contiguous: the 16x16x32 matrix instruction leaves 4 consecutive rows of D
// in a lane, so with A's index as the row a lane ends with 4 consecutive
// output elements.  The layer's three products are this
// one, with operands whose contraction index runs along memory ("rows": A[i]
// is a row) or across it ("columns": row k of memory holds A[., k]):
//   forward  y[t, n]:  A = W rows,       B = x rows
//   dx[t, k]:          A = W columns,    B = dz rows
//   dW[n, k]:          A = x columns,    B = dz columns
//
// Operands go from memory to LDS without passing registers (16 bytes a lane);
// the LDS side of such a load is contiguous over the wave, so the bank
// swizzle is put on the memory side: a lane fetches the 16-byte chunk that
// belongs at its place.  A "rows" tile holds 64 k of each index as 8 chunks,
// chunk c of row r at place c ^ (r & 7), read with 16-byte LDS reads.  A
// "columns" tile holds BI (BJ) indices of each k, 16 indices (32 bytes) at a
// time at place p ^ swizzle(k); the transposing LDS read gives each lane 4
// consecutive k of its index, and the 8 rows of k that two 16-lane groups
// read together lie in 8 different 32-byte places.
//
// Loads go through buffer descriptors that end at the operand's last
// element: rows past the end read as 0 and need no branch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act8.h"
#include "bf16_io.h"

namespace tide {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4v __attribute__((ext_vector_type(4)));

#define TIDE_LDS __attribute__((address_space(3)))


// An operand as the kernel reads it: 16-byte aligned, ld % 8 == 0, and either
// (rows) `count` rows of `depth` contraction elements, or (columns) `depth`
// rows of `count` elements; the contiguous length is a multiple of 8.  Of two
// operands one may be up to 7 contraction elements longer than the other,
// whose missing elements read as 0 (the longer one's then have to be finite).
//
// A "kept" operand is the columns of a checkpoint (act8.h): `depth` rows of
// `count` = ld = its pitch.
//
// Two matrices of one shape are one operand A in two ways.  "Pair rows": rows,
// 16 of the first and the same 16 of the second in turn, so that a lane ends
// with the same element of both products.  "Pair columns": columns, the
// contraction going through the first and then, from element `turn` (a multiple
// of 64, `depth` or more; what lies between reads as 0) on, through the second.
// "Pair rows once": pair rows that no other workgroup reads and that come past the
// caches.
enum Layout { kRows, kColumns, kKept, kPairRows, kPairColumns, kPairRowsOnce };

// The contraction index runs across memory.
constexpr bool across(Layout l) { return l == kColumns || l == kKept || l == kPairColumns; }

struct Operand {
    const void* p;
    int64_t ld;
    int64_t count;
    int64_t depth;
};

struct PairOperand {
    const void *p, *p2;
    int64_t ld;
    int64_t count;  // of one matrix
    int64_t depth;  // of one matrix
    int64_t turn;   // pair columns
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* base, int64_t bytes) {
    const int64_t most = (int64_t)1 << 31;
    const int32_t n = (int32_t)(uint32_t)(bytes < 0 ? 0 : bytes > most ? most : bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, n, 0x00020000);
}

constexpr uint32_t kNowhere = 0xf0000000u;  // an offset past every descriptor's end

// The swizzles: a "rows" tile's chunk c of row r lies at c ^ row_swizzle(r), a
// "columns" tile's 32-byte pair p of row k at p ^ column_swizzle(k).
__device__ __forceinline__ constexpr int row_swizzle(int r) {
    return r & 7;
}
template <int N>
__device__ __forceinline__ constexpr int column_swizzle(int k) {
    constexpr int kPairs = N / 16;
    return ((k & 3) | ((k >> 1) & 4)) & (kPairs % 8 == 0 ? 7 : kPairs % 4 == 0 ? 3 : kPairs - 1);
}

// 16 bytes a lane from memory to LDS, contiguous over the wave there.  (The
// compiler's host pass checks the size against the host's features, not
// gfx950's, takes 16 for an error and the functions that use it for unusable.)
constexpr int kNonTemporal = 2;
template <int AUX>
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, TIDE_LDS char* lds,
                                            uint32_t offset) {
#ifdef __HIP_DEVICE_COMPILE__
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds, 16, offset, 0, 0, AUX);
#endif
}

// A tile of N indices and K contraction elements from `first` on, staged by
// WAVES waves.  ONCE: no other workgroup reads the operand's elements.
template <int N, int K, int WAVES, bool COLUMNS, bool ONCE = false>
struct Stager {
    static constexpr int kBytes = N * K * 2;
    static constexpr int kLoads = kBytes / 1024;                       // of a whole wave
    static constexpr int kMine = (kLoads + WAVES - 1) / WAVES;
    static constexpr int kRowChunks = COLUMNS ? N / 8 : K / 8;    // 16-byte chunks of a row

    // a lane's chunk is the same in all its loads: they are a multiple of the
    // swizzle's period of rows apart
    static_assert(COLUMNS || kMine == 1 || WAVES * 64 / kRowChunks % 8 == 0, "");

    const char* base;
    int64_t step;        // bytes from one k tile to the next
    int64_t left;        // bytes from base to the operand's end
    uint32_t offset[kMine];
    int wave;
    int chunk_k;         // rows: first contraction element of the lane's chunk

    __device__ __forceinline__ void init(const Operand& o, int64_t first, int64_t k0, int lane,
                                         int wave_) {
        wave = wave_;
        chunk_k = 0;
        if constexpr (COLUMNS) {
            base = static_cast<const char*>(o.p) + 2 * (k0 * o.ld + first);
            left = 2 * ((o.depth - k0 - 1) * o.ld + o.count - first);
            step = 2 * K * o.ld;
        } else {
            base = static_cast<const char*>(o.p) + 2 * (first * o.ld + k0);
            left = 2 * ((o.count - first - 1) * o.ld + o.depth - k0);
            step = 2 * K;
        }
#pragma unroll
        for (int q = 0; q < kMine; ++q) {
            const int place = (q * WAVES + wave) * 64 + lane;
            const int row = place / kRowChunks, at = place % kRowChunks;
            int c;
            if constexpr (COLUMNS) {
                c = at ^ (column_swizzle<N>(row) << 1);
            } else {
                c = at ^ row_swizzle(row);
                chunk_k = c * 8;
            }
            offset[q] = (uint32_t)((int64_t)row * o.ld * 2 + c * 16);
        }
    }

    __device__ __forceinline__ void prime() {}

    // Stage the current k tile into `lds` and move on to the next.  valid:
    // contraction elements left from the tile's first on.
    __device__ __forceinline__ void stage(TIDE_LDS char* lds, int64_t valid) {
        const __amdgpu_buffer_rsrc_t r = resource(base, left);
        // a "columns" tile's rows past the end are past the descriptor's end
        const bool none = !COLUMNS && valid < K && chunk_k >= valid;
#pragma unroll
        for (int q = 0; q < kMine; ++q) {
            const int load = q * WAVES + wave;
            if (kLoads % WAVES && load >= kLoads) break;
            load_to_lds<ONCE ? kNonTemporal : 0>(r, lds + load * 1024, none ? kNowhere : offset[q]);
        }
        base += step;
        left -= step;
    }
};

// The same for a "columns" tile whose operand is kept in 8 bits: it passes
// registers, where it is widened to bf16 (exactly).  A lane takes 16 columns
// of a row of k, half a block: 16 bytes, one scale, and 32 bytes in LDS.  The
// next tile's bytes are loaded while this one is multiplied.  For tiles of
// four waves, where it saves writing and reading x in bf16: dW of 1003 x 1001
// x 8192 31.4 us against 39.1, of 77 x 768 x 2048 8.9 against 12.7.  256 x 256
// tiles, power-bound, pay more for widening x once in every row of tiles:
// 4096 x 28672 x 8192 1553 us against 1467 with x widened beforehand.
template <int N, int K, int WAVES>
struct KeptStager {
    static constexpr int kBytes = N * K * 2;
    static constexpr int kRowPairs = N / 16;
    static constexpr int kMine = N * K / 16 / (WAVES * 64);
    static_assert(kMine * WAVES * 64 * 16 == N * K, "every lane has as many pieces");

    const char *base, *scales;
    int64_t step, left;
    uint32_t offset[kMine], place[kMine];
    u32x4v bytes[kMine];
    uint32_t scale[kMine];

    __device__ __forceinline__ void init(const Operand& o, int64_t first, int64_t k0, int lane,
                                         int wave) {
        base = static_cast<const char*>(o.p) + k0 * o.ld + first;
        scales = static_cast<const char*>(o.p) + o.depth * o.ld + (k0 * o.ld + first) / kActBlock;
        left = (o.depth - k0) * o.ld - first;
        step = K * o.ld;
#pragma unroll
        for (int q = 0; q < kMine; ++q) {
            const int piece = (q * WAVES + wave) * 64 + lane;
            const int row = piece / kRowPairs, pair = piece % kRowPairs;
            offset[q] = (uint32_t)((int64_t)row * o.ld + pair * 16);
            place[q] = (uint32_t)(row * 2 * N + (pair ^ column_swizzle<N>(row)) * 32);
        }
    }

    // Rows past the end read as zeros with a scale of zero.
    __device__ __forceinline__ void prime() {
        const __amdgpu_buffer_rsrc_t r = resource(base, left);
        const __amdgpu_buffer_rsrc_t s = resource(scales, left / kActBlock);
#pragma unroll
        for (int q = 0; q < kMine; ++q) {
            bytes[q] = __builtin_amdgcn_raw_buffer_load_b128(r, offset[q], 0, 0);
            scale[q] = __builtin_amdgcn_raw_buffer_load_b8(s, offset[q] / kActBlock, 0, 0);
        }
        base += step;
        scales += step / kActBlock;
        left -= step;
    }

    __device__ __forceinline__ void stage(TIDE_LDS char* lds, int64_t) {
#pragma unroll
        for (int q = 0; q < kMine; ++q) {
            const float f = act8_scale(scale[q]);
            u32x4v lo, hi;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                lo[2 * w] = act8_bf16x2<false>(bytes[q][w], f);
                lo[2 * w + 1] = act8_bf16x2<true>(bytes[q][w], f);
                hi[2 * w] = act8_bf16x2<false>(bytes[q][w + 2], f);
                hi[2 * w + 1] = act8_bf16x2<true>(bytes[q][w + 2], f);
            }
            *(TIDE_LDS u32x4v*)(lds + place[q]) = lo;
            *(TIDE_LDS u32x4v*)(lds + place[q] + 16) = hi;
        }
        prime();
    }
};

// "Pair rows": tile row r is row r / 32 * 16 + r % 16 of matrix r / 16 % 2.
template <int N, int K, int WAVES, bool ONCE>
struct PairRowsStager {
    static constexpr int kBytes = N * K * 2;
    static constexpr int kLoads = kBytes / 1024;
    static constexpr int kMine = kLoads / WAVES;
    static constexpr int kRowChunks = K / 8;
    static constexpr int kLoadRows = 64 / kRowChunks;  // of a wave's load
    static_assert(kMine * WAVES == kLoads && WAVES * kLoadRows % 8 == 0, "");
    // a wave's loads are of one matrix, or of both in the same order in every wave
    static constexpr bool kOne = WAVES * kLoadRows % 32 == 0;
    static_assert(kOne || WAVES * kLoadRows <= 16, "");

    const char *base, *base2;  // kOne: the wave's matrix, in `base`
    int64_t left;
    uint32_t offset[kMine];
    int wave;
    int chunk_k;

    __device__ __forceinline__ void init(const PairOperand& o, int64_t first, int64_t k0, int lane,
                                         int wave_) {
        wave = wave_;
        const int64_t at = 2 * (first / 2 * o.ld + k0);
        const bool second = kOne && wave * kLoadRows / 16 % 2;
        base = static_cast<const char*>(second ? o.p2 : o.p) + at;
        base2 = static_cast<const char*>(o.p2) + at;
        left = 2 * ((o.count - first / 2 - 1) * o.ld + o.depth - k0);
#pragma unroll
        for (int q = 0; q < kMine; ++q) {
            const int place = (q * WAVES + wave) * 64 + lane;
            const int row = place / kRowChunks, c = place % kRowChunks ^ row_swizzle(row);
            chunk_k = c * 8;
            offset[q] = (uint32_t)((int64_t)(row / 32 * 16 + row % 16) * o.ld * 2 + c * 16);
        }
    }

    __device__ __forceinline__ void prime() {}

    __device__ __forceinline__ void stage(TIDE_LDS char* lds, int64_t valid) {
        const __amdgpu_buffer_rsrc_t r = resource(base, left), r2 = resource(base2, left);
        const bool none = valid < K && chunk_k >= valid;
#pragma unroll
        for (int q = 0; q < kMine; ++q) {
            const bool second = !kOne && q * WAVES * kLoadRows / 16 % 2;
            load_to_lds<ONCE ? kNonTemporal : 0>(second ? r2 : r, lds + (q * WAVES + wave) * 1024,
                                                 none ? kNowhere : offset[q]);
        }
        base += 2 * K;
        base2 += 2 * K;
        left -= 2 * K;
    }
};

// "Pair columns": a "columns" tile that goes on in the second matrix.
template <int N, int K, int WAVES>
struct PairColumnsStager : Stager<N, K, WAVES, true> {
    using Base = Stager<N, K, WAVES, true>;
    const char* base2;  // the second matrix's first tile
    int64_t left2;
    int64_t until;      // contraction elements up to it

    __device__ __forceinline__ void init(const PairOperand& o, int64_t first, int64_t k0, int lane,
                                         int wave) {
        const bool second = k0 >= o.turn;
        Base::init(Operand{second ? o.p2 : o.p, o.ld, o.count, o.depth}, first,
                   second ? k0 - o.turn : k0, lane, wave);
        base2 = static_cast<const char*>(o.p2) + 2 * first;
        left2 = 2 * ((o.depth - 1) * o.ld + o.count - first);
        until = o.turn - k0;  // none left of it where the second is under way
    }

    __device__ __forceinline__ void stage(TIDE_LDS char* lds, int64_t valid) {
        Base::stage(lds, valid);
        until -= K;
        if (until == 0) {
            this->base = base2;
            this->left = left2;
        }
    }
};

template <int N, int K, int WAVES, Layout L, bool ONCE>
struct StagerOf {
    using type = Stager<N, K, WAVES, L == kColumns, ONCE>;
};
template <int N, int K, int WAVES, bool ONCE>
struct StagerOf<N, K, WAVES, kKept, ONCE> {
    using type = KeptStager<N, K, WAVES>;
};
template <int N, int K, int WAVES, bool ONCE>
struct StagerOf<N, K, WAVES, kPairRows, ONCE> {
    using type = PairRowsStager<N, K, WAVES, ONCE>;
};
template <int N, int K, int WAVES, bool ONCE>
struct StagerOf<N, K, WAVES, kPairRowsOnce, ONCE> {
    using type = PairRowsStager<N, K, WAVES, true>;
};
template <int N, int K, int WAVES, bool ONCE>
struct StagerOf<N, K, WAVES, kPairColumns, ONCE> {
    using type = PairColumnsStager<N, K, WAVES>;
};

// The 16 x 32 piece of a staged tile that a matrix instruction takes: index
// m0 + (lane & 15), contraction k = 32 * s + 8 * (lane >> 4) .. + 7.
template <int N, int K, Layout L>
struct Reader {
    template <int S>
    __device__ __forceinline__ static bf16x8 read(const TIDE_LDS char* lds, int m0, int lane) {
        return read(lds, m0, lane, S);
    }
    __device__ __forceinline__ static bf16x8 read(const TIDE_LDS char* lds, int m0, int lane, int S) {
        if constexpr (across(L)) {
            constexpr int kRow = 2 * N;
            const int g = lane >> 4, i = lane & 15;
            const int k = 32 * S + 8 * g + (i >> 2);
            const int pair = (m0 >> 4) ^ column_swizzle<N>(k);
            const TIDE_LDS char* p = lds + k * kRow + pair * 32 + (i & 3) * 8;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TIDE_LDS s16x4*)p);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TIDE_LDS s16x4*)(p + 4 * kRow));
            const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(bf16x8, v);
        } else {
            const int row = m0 + (lane & 15);
            const int c = (4 * S + (lane >> 4)) ^ row_swizzle(lane & 15);
            return *(const TIDE_LDS bf16x8*)(lds + row * (2 * K) + c * 16);
        }
    }
};

// Every load into LDS has landed and every LDS read has returned, in every
// wave: the staged tile can be read and the other one overwritten.
// The two tiles' addresses are operands so that, __restrict__ or not, the
// compiler takes it to use that memory and moves no access across.
__device__ __forceinline__ void tile_barrier(const TIDE_LDS char* a, const TIDE_LDS char* b) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::"s"(a), "s"(b) : "memory");
}

// The S-th 32 contraction elements of a staged tile of K: their reads, and
// their matrix instructions.
template <int BI, int BJ, int K, int TI, int TJ, Layout CA, Layout CB, int S>
__device__ __forceinline__ void read_part(const TIDE_LDS char* la, const TIDE_LDS char* lb, int i0,
                                          int j0, int lane, bf16x8 (&a)[TI], bf16x8 (&b)[TJ]) {
#pragma unroll
    for (int t = 0; t < TI; ++t) a[t] = Reader<BI, K, CA>::template read<S>(la, i0 + 16 * t, lane);
#pragma unroll
    for (int t = 0; t < TJ; ++t) b[t] = Reader<BJ, K, CB>::template read<S>(lb, j0 + 16 * t, lane);
}

template <int TI, int TJ>
__device__ __forceinline__ void multiply_part(const bf16x8 (&a)[TI], const bf16x8 (&b)[TJ],
                                              f32x4v (&acc)[TI][TJ]) {
#pragma unroll
    for (int x = 0; x < TI; ++x)
#pragma unroll
        for (int y = 0; y < TJ; ++y)
            acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[x], b[y], acc[x][y], 0, 0, 0);
}

// Deals READS LDS reads out between the matrix instructions of their block,
// one to one.
template <int READS>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int k = 0; k < READS; ++k) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
}

// One k tile, for tiles that have a compute unit to themselves (8 waves, two
// on each SIMD).  The first half is in registers (a0, b0) already; while it is
// multiplied the second half is read.  Then, after the barrier, all waves
// have done reading this tile (`now`) and the next one (`next`) has landed:
// the tile after the next goes where this one was, and while the second half
// is multiplied the first half of the next tile is read.  A load has a whole
// step to arrive, a read half a step, and there is one barrier a step.  The
// two tiles lie in different halves of LDS, and saying so (__restrict__)
// keeps the compiler from making reads of one wait for loads into the other.
//
// Measured with 256 x 256 tiles on 4096 x 28672 x 8192: 1370 TFLOP/s, against
// 1265 with the plain step below and 1335 without the dealing-out; two groups
// of four waves in opposite phases (four barriers a step) 1175, 32x32x16
// instructions 1300.  The matrix pipes are busy 66% of the cycles then, and the
// clock is down to 1.75 GHz: what bounds it is power.
template <int BI, int BJ, int K, int TI, int TJ, Layout CA, Layout CB, typename SA, typename SB>
__device__ __forceinline__ void deep_step(TIDE_LDS char* __restrict__ next,
                                          TIDE_LDS char* __restrict__ now, bool more, bool more2,
                                          SA& sa, SB& sb, int64_t valid, int wi, int wj, int lane,
                                          bf16x8 (&a0)[TI], bf16x8 (&b0)[TJ],
                                          f32x4v (&acc)[TI][TJ]) {
    constexpr int kReads = TI * (across(CA) ? 2 : 1) + TJ * (across(CB) ? 2 : 1);
    bf16x8 a1[TI], b1[TJ];
    read_part<BI, BJ, K, TI, TJ, CA, CB, 1>(now, now + SA::kBytes, wi, wj, lane, a1, b1);
    multiply_part<TI, TJ>(a0, b0, acc);
    interleave<kReads>();
    __builtin_amdgcn_sched_barrier(0);
    tile_barrier(now, next);
    __builtin_amdgcn_sched_barrier(0);
    if (more) read_part<BI, BJ, K, TI, TJ, CA, CB, 0>(next, next + SA::kBytes, wi, wj, lane, a0, b0);
    if (more2) {
        sa.stage(now, valid);
        sb.stage(now + SA::kBytes, valid);
    }
    multiply_part<TI, TJ>(a1, b1, acc);
    if constexpr (across(CB)) {
        // many short reads: the loads are issued before them
        __builtin_amdgcn_sched_group_barrier(0x020, SA::kMine + SB::kMine, 0);
        interleave<kReads>();
    }
    __builtin_amdgcn_sched_barrier(0);
}

template <int S>
struct Part {
    static constexpr int value = S;
};

// One k tile, plainly: the next tile's loads, this tile's reads and matrix
// instructions half by half.  For the smaller tiles, of which a compute unit
// holds several: other workgroups fill the gaps, and fewer registers let more
// of them in (the step above on 128 x 128 tiles: 8% slower on 1003 x 1001 x
// 8192, 15% on 2048 x 5120 x 13824).
template <int BI, int BJ, int K, int TI, int TJ, Layout CA, Layout CB, typename SA, typename SB>
__device__ __forceinline__ void plain_step(TIDE_LDS char* __restrict__ next,
                                           const TIDE_LDS char* __restrict__ now, bool more, SA& sa,
                                           SB& sb, int64_t valid, int wi, int wj, int lane,
                                           f32x4v (&acc)[TI][TJ]) {
    if (more) {
        sa.stage(next, valid);
        sb.stage(next + SA::kBytes, valid);
    }
    bf16x8 a[TI], b[TJ];
    auto part = [&](auto s) __attribute__((always_inline)) {
        read_part<BI, BJ, K, TI, TJ, CA, CB, decltype(s)::value>(now, now + SA::kBytes, wi, wj, lane,
                                                                a, b);
        multiply_part<TI, TJ>(a, b, acc);
    };
    part(Part<0>());
    part(Part<1>());
    if constexpr (K == 256) {
        part(Part<2>());
        part(Part<3>());
        part(Part<4>());
        part(Part<5>());
        part(Part<6>());
        part(Part<7>());
    }
}

// The loop over the contraction elements [k0, k1) of `depth` (the longer
// operand's) of the tile at (i0, j0), with two tiles of K of them in LDS.
// H = 2: the elements in two halves of as many steps, each by WI * WJ waves
// with tiles of their own in LDS.  (Only where k1 = depth can the number of
// steps be odd, and behind `depth` the operands read as 0.)
template <int BI, int BJ, int K, int WI, int WJ, Layout CA, Layout CB, int H, typename OA>
__device__ __forceinline__ void tile_loop(const OA& A, const Operand& B, int64_t depth,
                                          int64_t k0, int64_t k1, int64_t i0, int64_t j0,
                                          TIDE_LDS char* lds,
                                          f32x4v (&acc)[BI / WI / 16][BJ / WJ / 16]) {
    constexpr int kWaves = WI * WJ, TI = BI / WI / 16, TJ = BJ / WJ / 16;
    using SA = typename StagerOf<BI, K, kWaves, CA, (K > 64)>::type;
    using SB = typename StagerOf<BJ, K, kWaves, CB, false>::type;
    constexpr int kTile = SA::kBytes + SB::kBytes;
    const int lane = threadIdx.x & 63;
    int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int steps = (int)((k1 - k0 + K - 1) / K);
    if constexpr (H == 2) {
        const int half = wave / kWaves;
        wave -= half * kWaves;
        steps = (steps + 1) / 2;
        k0 += (int64_t)half * steps * K;
        lds += half * 2 * kTile;
    }
    const int wi = (wave / WJ) * TI * 16, wj = (wave % WJ) * TJ * 16;
    SA sa;
    SB sb;
    sa.init(A, i0, k0, lane, wave);
    sb.init(B, j0, k0, lane, wave);
#pragma unroll
    for (int x = 0; x < TI; ++x)
#pragma unroll
        for (int y = 0; y < TJ; ++y) acc[x][y] = 0;
    if (steps == 0) return;
    int64_t valid = depth - k0;
    int at = 0;
    sa.prime();
    sb.prime();
    sa.stage(lds, valid);
    sb.stage(lds + SA::kBytes, valid);
    if constexpr (kWaves == 8) {
        tile_barrier(lds, lds + kTile);
        valid -= K;
        if (steps > 1) {
            sa.stage(lds + kTile, valid);
            sb.stage(lds + kTile + SA::kBytes, valid);
        }
        bf16x8 a0[TI], b0[TJ];
        read_part<BI, BJ, K, TI, TJ, CA, CB, 0>(lds, lds + SA::kBytes, wi, wj, lane, a0, b0);
        auto step = [&](bool more, bool more2) __attribute__((always_inline)) {
            valid -= K;
            deep_step<BI, BJ, K, TI, TJ, CA, CB>(lds + (at ^ kTile), lds + at, more, more2, sa, sb,
                                              valid, wi, wj, lane, a0, b0, acc);
            at ^= kTile;
        };
#pragma unroll 1
        for (int s = 0; s < steps - 2; ++s) step(true, true);
        if (steps > 1) step(true, false);
        step(false, false);
    } else {
        for (int s = 0; s < steps; ++s) {
            tile_barrier(lds + at, lds + (at ^ kTile));
            valid -= K;
            plain_step<BI, BJ, K, TI, TJ, CA, CB>(lds + (at ^ kTile), lds + at, s + 1 < steps, sa, sb,
                                               valid, wi, wj, lane, acc);
            at ^= kTile;
        }
    }
}

// All but the latest N loads of this wave have landed.
template <int N>
__device__ __forceinline__ void wait_loads(const TIDE_LDS char* tile) {
    static_assert(N < 64, "the counter has 6 bits");
    asm volatile("s_waitcnt vmcnt(%1)" ::"s"(tile), "n"(N) : "memory");
}
// Every LDS read of every wave has returned, and what each has waited for is
// there for all.
__device__ __forceinline__ void ring_barrier(const TIDE_LDS char* a, const TIDE_LDS char* b) {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::"s"(a), "s"(b) : "memory");
}

// A step of a ring: loads into one tile, the set's half of another.
template <int BI, int BJ, int K, int TI, int TJ, Layout CA, Layout CB, typename SA, typename SB>
__device__ __forceinline__ void ring_step(TIDE_LDS char* __restrict__ next,
                                          const TIDE_LDS char* __restrict__ now, SA& sa, SB& sb,
                                          int64_t valid, int wi, int wj, int lane, int set,
                                          f32x4v (&acc)[TI][TJ]) {
    sa.stage(next, valid);
    sb.stage(next + SA::kBytes, valid);
#pragma unroll
    for (int k = 0; k < K / 64; ++k) {
        bf16x8 a[TI], b[TJ];
#pragma unroll
        for (int t = 0; t < TI; ++t)
            a[t] = Reader<BI, K, CA>::read(now, wi + 16 * t, lane, set * (K / 64) + k);
#pragma unroll
        for (int t = 0; t < TJ; ++t)
            b[t] = Reader<BJ, K, CB>::read(now + SA::kBytes, wj + 16 * t, lane, set * (K / 64) + k);
        multiply_part<TI, TJ>(a, b, acc);
    }
}

// The same loop with R tiles in LDS, R - 1 of them under way: a step waits for the
// oldest only, so the loads never run dry.  Two sets of WI * WJ waves share the
// tiles, each with half of a tile's contraction.  Loads are issued to the last step,
// so that every step has as many to wait for: behind the contraction's end they lie
// outside the operands' descriptors (they read as 0), behind the end of another
// split they are the next one's first R - 1 tiles, which it reads too (a third more
// bytes for 16 x 1001 x 8192 in 8 splits, a tenth for 16 x 4096 x 4096 in 2).  The
// barrier behind the loop waits for them before LDS is used again.
//
// For rows of two matrices (the gated block's forward product, where the plain
// step's pair of tiles leaves a compute unit waiting for memory): us with the
// ring and, before it, with tiles in pairs, T x N x K: 16 x 4096 x 4096 17.4 and
// 27.8, 16 x 1001 x 8192 15.2 and 25.4, 64 x 13824 x 5120 51.0 and 69.9, 1003 x 768 x
// 2048 18.4 and 22.5.  Tiles of 128 contraction elements against 64: 49.8 and
// 51.3 for 16 x 13824 x 5120.  Operands across memory gain nothing (dx of 64 x
// 4096 x 4096 25.1, in pairs 24.3): their reads from LDS are twice as many.
template <int BI, int BJ, int K, int WI, int WJ, Layout CA, Layout CB, int R, typename OA>
__device__ __forceinline__ void ring_loop(const OA& A, const Operand& B, int64_t depth, int64_t k0,
                                          int64_t k1, int64_t i0, int64_t j0, TIDE_LDS char* lds,
                                          f32x4v (&acc)[BI / WI / 16][BJ / WJ / 16]) {
    constexpr int kSet = WI * WJ, kWaves = 2 * kSet, TI = BI / WI / 16, TJ = BJ / WJ / 16;
    using SA = typename StagerOf<BI, K, kWaves, CA, false>::type;
    using SB = typename StagerOf<BJ, K, kWaves, CB, false>::type;
    constexpr int kTile = SA::kBytes + SB::kBytes;
    // every wave's loads of a step are as many, which is what it waits by
    constexpr int kLoads = SA::kMine + SB::kMine;
    static_assert(SA::kBytes / 1024 % kWaves == 0 && SB::kBytes / 1024 % kWaves == 0, "");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int set = wave / kSet, of = wave - set * kSet;
    const int wi = (of / WJ) * TI * 16, wj = (of % WJ) * TJ * 16;
    const int steps = (int)((k1 - k0 + K - 1) / K);
    SA sa;
    SB sb;
    sa.init(A, i0, k0, lane, wave);
    sb.init(B, j0, k0, lane, wave);
#pragma unroll
    for (int x = 0; x < TI; ++x)
#pragma unroll
        for (int y = 0; y < TJ; ++y) acc[x][y] = 0;
    int64_t valid = depth - k0;
    auto stage = [&](int at) __attribute__((always_inline)) {
        sa.stage(lds + at, valid);
        sb.stage(lds + at + SA::kBytes, valid);
        valid -= K;
    };
#pragma unroll
    for (int r = 0; r < R - 1; ++r) stage(r * kTile);
    int now = 0, next = (R - 1) * kTile;
#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
        wait_loads<(R - 2) * kLoads>(lds + now);
        ring_barrier(lds + now, lds + next);
        ring_step<BI, BJ, K, TI, TJ, CA, CB>(lds + next, lds + now, sa, sb, valid, wi, wj, lane, set, acc);
        valid -= K;
        next = now;
        now += kTile;
        if (now == R * kTile) now = 0;
    }
}

}  // namespace tide
