// gated.hip -- the gated block in front of a layer's last product: both
// projections, the activation and the product in one kernel, and its gradients
// from 8-bit checkpoints, for gfx950.
//
//   forward   g = x Wg^T + bg, u = x Wu^T + bu, h = act(g) u
//   backward  dg = dh u act'(g), du = dh act(g), dx = dg Wg + du Wu,
//             dWg = dg^T x, dWu = du^T x, dbg and dbu the sums of dg and du
//
// The products run through the layer products' tile loop (tile_product.h,
// product.h) with two matrices as one operand.  Forward: 16 rows of Wg and the
// same 16 of Wu in turn, so that a lane's accumulators hold an element of g
// and the same of u, and neither is written in more than 8 bits.  dx: one
// contraction over [dg du] and Wg above Wu, so that the two halves are added in
// the accumulators.  dWg and dWu: one product [dg du]^T x, whose rows go to two
// places.  dg and du lie side by side in the workspace, each in rows rounded up
// to 64 elements, so that a step of the contraction stays within one matrix.
//
// The weights' bytes bound few tokens, the matrix pipes' power many: 1 token of
// 28672 x 8192 forward 136 us (6.9 TB/s), 24 of 13824 x 5120 45.5 (6.2), 4096 of
// 28672 x 8192 2944 (1.31 PFLOP/s); backward of the last 6027: dg and du 163, x
// widened 28, dx 2858 (1.35 PFLOP/s), the weights' gradients 2974 (1.29).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "act8.h"
#include "activation.h"
#include "bf16_io.h"
#include "linear_check.h"
#include "product.h"
#include "product_shape.h"
#include "tide.h"

using namespace tide;

namespace {

// ---- epilogues ---------------------------------------------------------------

// What happens to finished g and u.  I: rows of the two matrices together as the
// tile loop counts them, J: tokens.
struct GatedEpilogue {
    static constexpr bool kPairs = true;
    int64_t I, J, N;
    uint16_t* out;
    int64_t ldo;
    const uint16_t *bias_g, *bias_u;
    uint8_t *kept_g, *kept_u, *kept_h;
    int32_t act;
    __device__ __forceinline__ int64_t columns() const { return N; }
};

__device__ __forceinline__ void add_bias(const uint16_t* bias, int64_t n, int64_t have, float (&v)[8]) {
    float b[8];
    load8(bias + n, have, b);
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] += b[r];
}

// Eight of each at columns n .. n + 7 of token j; the four lanes of a
// checkpoint's block of 32 columns call this together.
__device__ __forceinline__ void finish(const GatedEpilogue& e, int64_t n, int64_t j, float (&g)[8],
                                       float (&u)[8]) {
    const int64_t have = j < e.J ? e.N - n : 0;
    if (e.bias_g) add_bias(e.bias_g, n, have, g);
    if (e.bias_u) add_bias(e.bias_u, n, have, u);
    if (e.kept_g) keep_unit(e.kept_g, e.N, e.J, n, j, have, g);
    if (e.kept_u) keep_unit(e.kept_u, e.N, e.J, n, j, have, u);
    apply_act(g, e.act);
#pragma unroll
    for (int r = 0; r < 8; ++r) g[r] *= u[r];
    if (e.kept_h) keep_unit(e.kept_h, e.N, e.J, n, j, have, g);
    if (have > 0) store8(e.out + j * e.ldo + n, have, g);
}

// Four of each, g before u; nothing is kept.
__device__ __forceinline__ void finish4(const GatedEpilogue& e, int64_t n, int64_t j, float (&v)[8]) {
    const int64_t have = j < e.J ? min((int64_t)4, e.N - n) : 0;
    if (have <= 0) return;
    float g[8] = {}, u[8] = {};
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        g[r] = v[r];
        u[r] = v[r + 4];
    }
    if (e.bias_g) add_bias(e.bias_g, n, have, g);
    if (e.bias_u) add_bias(e.bias_u, n, have, u);
    apply_act(g, e.act);
#pragma unroll
    for (int r = 0; r < 8; ++r) g[r] *= u[r];
    store8(e.out + j * e.ldo + n, have, g);
}

// dWg and dWu: rows j < turn of the product go to the first, the others to the
// second; each has N.
struct GradEpilogue {
    static constexpr bool kPairs = false, kNarrow = false;  // 2 * turn >= 128 rows
    int64_t I, J, N, turn;
    uint16_t *out, *out2;
    int64_t ldo;
};

__device__ __forceinline__ void finish(const GradEpilogue& e, int64_t i, int64_t j, bool there,
                                       float (&v)[8]) {
    const bool second = j >= e.turn;
    const int64_t row = second ? j - e.turn : j;
    if (there && row < e.N) store8((second ? e.out2 : e.out) + row * e.ldo + i, e.I - i, v);
}

// ---- dg and du -----------------------------------------------------------------

// dg and du rounded to bf16, side by side in rows of 2 * turn elements with
// zeros behind each one's N-th, and their column sums before the rounding
// over each chunk of rows (a row of `sums` for each chunk, dg's before du's).
// A lane keeps its 8 columns through a quarter of the chunk's rows; the
// quarters' sums meet in LDS.  (The rounding is the matrix instructions', which take
// bf16.  It leaves dx and the weights' gradients off by 2.4e-3 of themselves, root mean
// square, where their own rounding alone leaves 1.7e-3; dg and du in two parts, a rounded
// number and the rest of it, would double the work of the products, which are most of
// the time.)  Bound by memory: 4096 x 28672 with silu
// 165 us, 5.8 TB/s; 187 where the loads take place in the caches, 169 with the
// loads of 2 or 4 rows in flight in a lane.
constexpr int kDguLanes = 256;  // of 8 columns
constexpr int kDguQuarters = 4;
constexpr int64_t kDguOneChunk = 64;

struct DguArgs {
    const uint16_t* dh;
    int64_t ld;
    const uint8_t *g, *u;
    uint16_t* dgu;  // or NULL: sums only
    int64_t turn;
    float* sums;    // or NULL
    uint16_t *dbias_g, *dbias_u;  // the one chunk's sums go there, or NULL
    int64_t T, N, chunk;
    int32_t col_groups;
    bool want_sums;
};

template <int ACT, bool WHOLE>
__device__ __forceinline__ void dgu_lane(const DguArgs& p, int64_t c, int64_t t0, int64_t t1,
                                         float (&sum_g)[8], float (&sum_u)[8]) {
    constexpr float kHalf = ACT == TIDE_ACT_NONE || ACT == TIDE_ACT_RELU ? 1.0f : 0.5f;
    const int64_t pitch = act8_pitch(p.N), scales = p.T * pitch;
#pragma unroll 1
    for (int64_t t = t0; t < t1; ++t) {
        const int64_t at = t * pitch + c;
        const uint16_t* from = p.dh + t * p.ld + c;
        float d[8], g[8], u[8];
        const u32x2 qg = __builtin_nontemporal_load((const TIDE_GLOBAL_AS u32x2*)(p.g + at));
        const u32x2 qu = __builtin_nontemporal_load((const TIDE_GLOBAL_AS u32x2*)(p.u + at));
        const uint32_t sg = *(const TIDE_GLOBAL_AS uint8_t*)(p.g + scales + at / kActBlock);
        const uint32_t su = *(const TIDE_GLOBAL_AS uint8_t*)(p.u + scales + at / kActBlock);
        if constexpr (WHOLE)
            widen(load8_raw<true>(from), d);
        else
            load8(from, p.N - c, d);
        act8_unpack8(qg, act8_scale(sg), g);
        act8_unpack8(qu, act8_scale(su), u);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float slope;
            const float value = act_both<ACT>(g[k], &slope);
            // dg.  dh u may leave binary32 where dg does not (a slope of 0 would be NaN);
            // u times half the slope, which stays below 1, never does
            u[k] = d[k] * (u[k] * (kHalf * slope)) * (1.0f / kHalf);
            g[k] = d[k] * value;  // du
        }
        if constexpr (!WHOLE) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c + k >= p.N) g[k] = u[k] = 0.0f;
        }
        if (p.want_sums) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sum_g[k] += u[k];
                sum_u[k] += g[k];
            }
        }
        if (p.dgu) {
            store8(p.dgu + t * 2 * p.turn + c, 8, u);
            store8(p.dgu + t * 2 * p.turn + p.turn + c, 8, g);
        }
    }
}

template <int ACT>
__global__ __launch_bounds__(kDguLanes* kDguQuarters) void dgu_kernel(DguArgs p) {
    extern __shared__ __attribute__((aligned(16))) float part[];  // [quarters - 1][8][lanes]
    const int lanes = blockDim.x / kDguQuarters;
    const int quarter = threadIdx.x / lanes, lane = threadIdx.x - quarter * lanes;
    const int64_t cg = blockIdx.x % p.col_groups, ch = blockIdx.x / p.col_groups;
    const int64_t c = (cg * lanes + lane) * 8;
    const int64_t each = p.chunk / kDguQuarters;
    const int64_t t0 = ch * p.chunk + quarter * each, t1 = min(p.T, t0 + each);
    float sum_g[8] = {}, sum_u[8] = {};
    if (c + 8 <= p.N) {
        dgu_lane<ACT, true>(p, c, t0, t1, sum_g, sum_u);
    } else if (c < p.N) {
        dgu_lane<ACT, false>(p, c, t0, t1, sum_g, sum_u);
    } else if (c < p.turn && p.dgu) {
        const float zero[8] = {};
        for (int64_t t = t0; t < t1; ++t) {
            store8(p.dgu + t * 2 * p.turn + c, 8, zero);
            store8(p.dgu + t * 2 * p.turn + p.turn + c, 8, zero);
        }
    }
    if (!p.want_sums) return;
    auto add_up = [&](float (&sum)[8], float* sums, uint16_t* out) __attribute__((always_inline)) {
        __syncthreads();  // the sums before have been read
        if (quarter) {
#pragma unroll
            for (int r = 0; r < 8; ++r) part[((quarter - 1) * 8 + r) * lanes + lane] = sum[r];
        }
        __syncthreads();
        if (quarter) return;
#pragma unroll
        for (int q = 0; q < kDguQuarters - 1; ++q)
#pragma unroll
            for (int r = 0; r < 8; ++r) sum[r] += part[(q * 8 + r) * lanes + lane];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if (c + r >= p.N) continue;
            if (out)
                *(TIDE_GLOBAL_AS uint16_t*)(out + c + r) = to_bf16(sum[r]);
            else if (sums)
                sums[c + r] = sum[r];
        }
    };
    add_up(sum_g, p.sums ? p.sums + ch * 2 * p.N : nullptr, p.dbias_g);
    add_up(sum_u, p.sums ? p.sums + (ch * 2 + 1) * p.N : nullptr, p.dbias_u);
}

// A bias's gradient from the chunks' sums, `pitch` apart: a wave's lane takes a
// column, the workgroup's waves every kBiasWaves-th chunk.
constexpr int kBiasWaves = 8;

__global__ __launch_bounds__(64 * kBiasWaves) void gated_bias_kernel(const float* sums, int64_t chunks,
                                                                     int64_t N, uint16_t* dbias_g,
                                                                     uint16_t* dbias_u) {
    __shared__ float part[kBiasWaves][64];
    const int64_t groups = (N + 63) / 64;
    const bool second = blockIdx.x >= groups;
    uint16_t* out = second ? dbias_u : dbias_g;
    if (!out) return;
    if (second) sums += N;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)(blockIdx.x - (second ? groups : 0)) * 64 + lane;
    float s = 0.0f;
    if (c < N) {
#pragma unroll 4
        for (int64_t k = wave; k < chunks; k += kBiasWaves) s += sums[k * 2 * N + c];
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave || c >= N) return;
#pragma unroll
    for (int w = 1; w < kBiasWaves; ++w) s += part[w][lane];
    *(TIDE_GLOBAL_AS uint16_t*)(out + c) = to_bf16(s);
}

// ---- host ----------------------------------------------------------------------

tide_status check_dims(int64_t T, int64_t N, int64_t K, int32_t act, int32_t reserved) {
    if (T < 0 || N < 0 || K < 0 || act < TIDE_ACT_NONE || act > TIDE_ACT_SILU || reserved != 0)
        return TIDE_EINVAL;
    if (T > kMaxTokens || N > kMaxWidth / 2 || K > kMaxWidth) return TIDE_EUNSUPPORTED;
    if (T * N > kMaxElements / 2 || T * K > kMaxElements || N * K > kMaxElements / 2)
        return TIDE_EUNSUPPORTED;
    return TIDE_OK;
}

// ---- forward -------------------------------------------------------------------

struct ForwardPlan {
    bool gemv;
    Source x, gate, up;
    Shape shape;
    int64_t rows;  // of the two matrices together
    float* partial;
    int64_t bytes;
};

tide_status check_forward(const tide_gated_forward_args& a) {
    TIDE_TRY(check_dims(a.tokens, a.out_features, a.in_features, a.act, a.reserved));
    const int64_t T = a.tokens, N = a.out_features, K = a.in_features;
    if (T == 0 || N == 0) return TIDE_OK;
    TIDE_TRY(check_rows(a.x, a.ldx, T, K));
    TIDE_TRY(check_rows(a.gate, K, N, K));
    TIDE_TRY(check_rows(a.up, K, N, K));
    if (a.gate_bias) TIDE_TRY(check_rows(a.gate_bias, N, 1, N));
    if (a.up_bias) TIDE_TRY(check_rows(a.up_bias, N, 1, N));
    TIDE_TRY(check_rows(a.h, a.ldh, T, N));
    if (a.g_kept) TIDE_TRY(check_kept(a.g_kept, T, N));
    if (a.u_kept) TIDE_TRY(check_kept(a.u_kept, T, N));
    if (a.h_kept) TIDE_TRY(check_kept(a.h_kept, T, N));
    return TIDE_OK;
}

ForwardPlan plan_forward(const tide_gated_forward_args& a, void* ws) {
    ForwardPlan f;
    Carver c{static_cast<char*>(ws)};
    const int64_t T = a.tokens, N = a.out_features, K = a.in_features;
    const bool keep = a.g_kept || a.u_kept || a.h_kept;
    f.rows = 2 * round_up(N, 16);
    f.gemv = gated_by_rows(T, N, K, keep, direct(a.gate, K, N, K) && direct(a.up, K, N, K));
    f.bytes = 0;
    if (f.gemv) return f;
    f.x = {a.x, a.ldx, T, K};
    f.gate = {a.gate, K, N, K};
    f.up = {a.up, K, N, K};
    f.x.plan(c);
    f.gate.plan(c);
    f.up.plan(c);
    f.shape = choose_gated(f.rows, T, round_up(K, 8));
    f.partial = c.take<float>(partial_floats(f.shape, f.rows, T));
    f.bytes = c.used;
    return f;
}

}  // namespace

extern "C" tide_status tide_gated_forward_workspace(const tide_gated_forward_args* args,
                                                    size_t* bytes) {
    if (!args || !bytes) return TIDE_EINVAL;
    TIDE_TRY(check_forward(*args));
    *bytes = args->tokens && args->out_features ? (size_t)plan_forward(*args, nullptr).bytes : 0;
    return TIDE_OK;
}

extern "C" tide_status tide_gated_forward(const tide_gated_forward_args* args, void* workspace,
                                          size_t workspace_bytes, tide_stream_t stream) {
    if (!args) return TIDE_EINVAL;
    const tide_gated_forward_args& a = *args;
    TIDE_TRY(check_forward(a));
    const int64_t T = a.tokens, N = a.out_features, K = a.in_features;
    if (T == 0 || N == 0) return TIDE_OK;
    const Extent ext[] = {rows_extent(a.x, a.ldx, T, K),
                          rows_extent(a.gate, K, N, K),
                          rows_extent(a.up, K, N, K),
                          rows_extent(a.gate_bias, N, 1, N),
                          rows_extent(a.up_bias, N, 1, N),
                          rows_extent(a.h, a.ldh, T, N),
                          bytes_extent(a.g_kept, act8_bytes(T, N)),
                          bytes_extent(a.u_kept, act8_bytes(T, N)),
                          bytes_extent(a.h_kept, act8_bytes(T, N))};
    TIDE_TRY(check_apart(ext, 5, ext + 5, 4));
    const ForwardPlan f = plan_forward(a, workspace);
    TIDE_TRY(check_workspace(workspace, workspace_bytes, f.bytes, ext, 9));
    TIDE_TRY(check_stream_device(stream));
    GatedEpilogue e = {};
    e.I = f.rows;
    e.J = T;
    e.N = N;
    e.out = static_cast<uint16_t*>(a.h);
    e.ldo = a.ldh;
    e.bias_g = static_cast<const uint16_t*>(a.gate_bias);
    e.bias_u = static_cast<const uint16_t*>(a.up_bias);
    e.kept_g = static_cast<uint8_t*>(a.g_kept);
    e.kept_u = static_cast<uint8_t*>(a.u_kept);
    e.kept_h = static_cast<uint8_t*>(a.h_kept);
    e.act = a.act;
    if (f.gemv) {
        const Gemv<GatedEpilogue> gemv = {static_cast<const uint16_t*>(a.x), T > 1 ? a.ldx : K,
                                          static_cast<const uint16_t*>(a.gate),
                                          static_cast<const uint16_t*>(a.up), K, e};
        return launch(T == 1   ? gemv_kernel<1, GatedEpilogue>
                      : T == 2 ? gemv_kernel<2, GatedEpilogue>
                               : gemv_kernel<4, GatedEpilogue>,
                      ceil_div(N, kGemvRows / 2), kGemvThreads, stream, gemv);
    }
    TIDE_TRY(f.x.fill(stream));
    TIDE_TRY(f.gate.fill(stream));
    TIDE_TRY(f.up.fill(stream));
    const Operand gate = f.gate.operand(false), up = f.up.operand(false);
    Product<GatedEpilogue, PairOperand> p = {};
    p.A = {gate.p, up.p, gate.ld, gate.count, gate.depth, 0};
    p.B = f.x.operand(false);
    p.depth = round_up(K, 8);
    p.e = e;
    return run_product<kForward>(p, f.shape, f.partial, stream);
}

// ---- backward ------------------------------------------------------------------

namespace {

struct BackwardPlan {
    int64_t turn;
    int dgu_lanes;
    int64_t dgu_groups, chunk, chunks;
    Source gate, up;
    uint16_t* dgu = nullptr;
    float* sums = nullptr;
    uint16_t* x = nullptr;
    Gradients g;
    float* partial = nullptr;
    int64_t bytes;
};

bool wants_none(const tide_gated_backward_args& a) {
    return !a.dx && !a.dgate && !a.dup && !a.dgate_bias && !a.dup_bias;
}

tide_status check_backward(const tide_gated_backward_args& a) {
    TIDE_TRY(check_dims(a.tokens, a.out_features, a.in_features, a.act, a.reserved));
    const int64_t T = a.tokens, N = a.out_features, K = a.in_features;
    if (wants_none(a)) return TIDE_OK;
    if ((a.dgate == nullptr) != (a.dup == nullptr)) return TIDE_EINVAL;
    TIDE_TRY(check_rows(a.dh, a.lddh, T, N));
    TIDE_TRY(check_kept(a.g_kept, T, N));
    TIDE_TRY(check_kept(a.u_kept, T, N));
    if (a.dx) {
        TIDE_TRY(check_rows(a.gate, K, N, K));
        TIDE_TRY(check_rows(a.up, K, N, K));
        TIDE_TRY(check_rows(a.dx, a.lddx, T, K));
    }
    if (a.dgate) {
        TIDE_TRY(check_kept(a.x_kept, T, K));
        TIDE_TRY(check_rows(a.dgate, K, N, K));
        TIDE_TRY(check_rows(a.dup, K, N, K));
    }
    if (a.dgate_bias) TIDE_TRY(check_rows(a.dgate_bias, N, 1, N));
    if (a.dup_bias) TIDE_TRY(check_rows(a.dup_bias, N, 1, N));
    return TIDE_OK;
}

using DguKernel = void (*)(DguArgs);

DguKernel dgu_kernel_of(int32_t act) {
    switch (act) {
        case TIDE_ACT_RELU: return dgu_kernel<TIDE_ACT_RELU>;
        case TIDE_ACT_GELU: return dgu_kernel<TIDE_ACT_GELU>;
        case TIDE_ACT_GELU_TANH: return dgu_kernel<TIDE_ACT_GELU_TANH>;
        case TIDE_ACT_SILU: return dgu_kernel<TIDE_ACT_SILU>;
        default: return dgu_kernel<TIDE_ACT_NONE>;
    }
}

BackwardPlan plan_backward(const tide_gated_backward_args& a, void* ws) {
    BackwardPlan b;
    Carver c{static_cast<char*>(ws)};
    const int64_t T = a.tokens, N = a.out_features, K = a.in_features;
    const bool bias = a.dgate_bias || a.dup_bias;
    const bool dx = a.dx && T && N && K, dw = a.dgate && T && N && K;
    b.turn = round_up(N, 64);
    if (dx || dw) b.dgu = c.take<uint16_t>(T * 2 * b.turn);
    // Chunks of rows: about 512 workgroups of 16 waves, but where the column
    // sums are wanted at least 32 rows, so that the partial sums stay few
    const int64_t width = std::max<int64_t>(b.turn, 64);
    b.dgu_lanes = (int)std::min<int64_t>(kDguLanes, round_up(width / 8, 64));
    b.dgu_groups = ceil_div(width, 8 * b.dgu_lanes);
    b.chunk = std::max<int64_t>(bias ? 32 : kDguQuarters,
                                ceil_div(T, std::max<int64_t>(1, 512 / b.dgu_groups)));
    b.chunk = round_up(b.chunk, kDguQuarters);
    // few rows are one chunk, whose sums are the biases' gradients
    if (bias && T <= kDguOneChunk) b.chunk = round_up(std::max<int64_t>(T, 1), kDguQuarters);
    b.chunks = ceil_div(T, b.chunk);
    if (bias && b.chunks != 1) b.sums = c.take<float>(b.chunks * 2 * N);
    b.gate = {a.gate, K, dx ? N : 0, K};
    b.up = {a.up, K, dx ? N : 0, K};
    b.gate.plan(c);
    b.up.plan(c);
    b.g = choose_gated_gradients(T, b.turn, K, dx, dw);
    // the 256-wide tiles read x from here, widened (tile_product.h)
    if (dw && b.g.weight.bi == 256) b.x = c.take<uint16_t>(T * act8_pitch(K));
    int64_t floats = 0;
    if (dx) floats = std::max(floats, partial_floats(b.g.in, K, T));
    if (dw) floats = std::max(floats, partial_floats(b.g.weight, K, 2 * b.turn));
    b.partial = c.take<float>(floats);
    b.bytes = c.used;
    return b;
}

// Rows of zeros: gradients that are empty sums.
constexpr int kZeroThreads = 256;

__global__ __launch_bounds__(kZeroThreads) void zero_rows_kernel(uint16_t* p, int64_t ld, int64_t rows,
                                                                int64_t cols) {
    const int64_t per_row = (cols + 7) / 8;
    const int64_t u = (int64_t)blockIdx.x * kZeroThreads + threadIdx.x;
    const int64_t r = u / per_row, c = (u - r * per_row) * 8;
    const float zero[8] = {};
    if (r < rows) store8(p + r * ld + c, cols - c, zero);
}

tide_status zero_rows(void* p, int64_t ld, int64_t rows, int64_t cols, tide_stream_t stream) {
    if (!p || rows == 0 || cols == 0) return TIDE_OK;
    return launch(zero_rows_kernel, ceil_div(rows * ceil_div(cols, 8), kZeroThreads), kZeroThreads,
                  stream, static_cast<uint16_t*>(p), ld, rows, cols);
}

}  // namespace

extern "C" tide_status tide_gated_backward_workspace(const tide_gated_backward_args* args,
                                                     size_t* bytes) {
    if (!args || !bytes) return TIDE_EINVAL;
    TIDE_TRY(check_backward(*args));
    *bytes = wants_none(*args) || !args->tokens || !args->out_features
                 ? 0
                 : (size_t)plan_backward(*args, nullptr).bytes;
    return TIDE_OK;
}

extern "C" tide_status tide_gated_backward(const tide_gated_backward_args* args, void* workspace,
                                           size_t workspace_bytes, tide_stream_t stream) {
    if (!args) return TIDE_EINVAL;
    const tide_gated_backward_args& a = *args;
    TIDE_TRY(check_backward(a));
    if (wants_none(a)) return TIDE_OK;
    const int64_t T = a.tokens, N = a.out_features, K = a.in_features;
    const Extent ext[] = {rows_extent(a.dh, a.lddh, T, N),
                          a.dx ? rows_extent(a.gate, K, N, K) : Extent(),
                          a.dx ? rows_extent(a.up, K, N, K) : Extent(),
                          a.dgate ? bytes_extent(a.x_kept, act8_bytes(T, K)) : Extent(),
                          bytes_extent(a.g_kept, act8_bytes(T, N)),
                          bytes_extent(a.u_kept, act8_bytes(T, N)),
                          rows_extent(a.dx, a.lddx, T, K),
                          rows_extent(a.dgate, K, N, K),
                          rows_extent(a.dup, K, N, K),
                          rows_extent(a.dgate_bias, N, 1, N),
                          rows_extent(a.dup_bias, N, 1, N)};
    TIDE_TRY(check_apart(ext, 6, ext + 6, 5));
    if (T == 0 || N == 0) {
        TIDE_TRY(check_stream_device(stream));
        TIDE_TRY(zero_rows(a.dx, a.lddx, T, K, stream));
        TIDE_TRY(zero_rows(a.dgate, K, N, K, stream));
        TIDE_TRY(zero_rows(a.dup, K, N, K, stream));
        TIDE_TRY(zero_rows(a.dgate_bias, N, 1, N, stream));
        return zero_rows(a.dup_bias, N, 1, N, stream);
    }
    const BackwardPlan b = plan_backward(a, workspace);
    TIDE_TRY(check_workspace(workspace, workspace_bytes, b.bytes, ext, 11));
    TIDE_TRY(check_stream_device(stream));
    const bool bias = a.dgate_bias || a.dup_bias;
    if (b.dgu || bias) {
        DguArgs d = {};
        d.dh = static_cast<const uint16_t*>(a.dh);
        d.ld = a.lddh;
        d.g = static_cast<const uint8_t*>(a.g_kept);
        d.u = static_cast<const uint8_t*>(a.u_kept);
        d.dgu = b.dgu;
        d.turn = b.turn;
        d.sums = b.sums;
        d.want_sums = bias;
        if (b.chunks == 1) {
            d.dbias_g = static_cast<uint16_t*>(a.dgate_bias);
            d.dbias_u = static_cast<uint16_t*>(a.dup_bias);
        }
        d.T = T;
        d.N = N;
        d.chunk = b.chunk;
        d.col_groups = (int32_t)b.dgu_groups;
        const unsigned lds = bias ? (kDguQuarters - 1) * b.dgu_lanes * 8 * sizeof(float) : 0;
        TIDE_TRY(launch_lds(dgu_kernel_of(a.act), b.dgu_groups * b.chunks, b.dgu_lanes * kDguQuarters,
                            lds, stream, d));
    }
    if (bias && b.chunks != 1)
        TIDE_TRY(launch(gated_bias_kernel, 2 * ceil_div(N, 64), 64 * kBiasWaves, stream,
                        (const float*)b.sums, b.chunks, N, static_cast<uint16_t*>(a.dgate_bias),
                        static_cast<uint16_t*>(a.dup_bias)));
    if (!b.dgu) return TIDE_OK;

    Product<Epilogue, PairOperand> x = {};
    Product<GradEpilogue> w = {};
    if (a.dx) {
        TIDE_TRY(b.gate.fill(stream));
        TIDE_TRY(b.up.fill(stream));
        const Operand gate = b.gate.operand(true), up = b.up.operand(true);
        x.A = {gate.p, up.p, gate.ld, gate.count, gate.depth, b.turn};
        x.B = {b.dgu, 2 * b.turn, T, 2 * b.turn};
        x.depth = 2 * b.turn;
        x.e.I = K;
        x.e.J = T;
        x.e.out = static_cast<uint16_t*>(a.dx);
        x.e.ldo = a.lddx;
    }
    if (a.dgate) {
        w.A = {a.x_kept, act8_pitch(K), act8_pitch(K), T};
        if (b.x) {
            TIDE_TRY(act8_unpack_into(a.x_kept, T, K, b.x, act8_pitch(K), false, stream));
            w.A.p = b.x;
        }
        w.B = {b.dgu, 2 * b.turn, 2 * b.turn, T};
        w.depth = T;
        w.e.I = K;
        w.e.J = 2 * b.turn;
        w.e.N = N;
        w.e.turn = b.turn;
        w.e.out = static_cast<uint16_t*>(a.dgate);
        w.e.out2 = static_cast<uint16_t*>(a.dup);
        w.e.ldo = K;
    }
    return run_gradients(b.g, w, a.dgate != nullptr, x, a.dx != nullptr, b.partial, stream);
}
