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
#include "activation.h"
#include "bf16_io.h"
#include "linear_check.h"
#include "product.h"
#include "product_shape.h"
#include "tide.h"

using namespace tide;

namespace {

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
        const Gemv<Epilogue> gemv = {static_cast<const uint16_t*>(a.x), T > 1 ? a.ldx : K,
                                     static_cast<const uint16_t*>(a.weight), nullptr, K, e};
        return launch(T == 1   ? gemv_kernel<1, Epilogue>
                      : T == 2 ? gemv_kernel<2, Epilogue>
                               : gemv_kernel<4, Epilogue>,
                      ceil_div(N, kGemvRows), kGemvThreads, stream, gemv);
    }
    TIDE_TRY(f.x.fill(stream));
    TIDE_TRY(f.w.fill(stream));
    Product<Epilogue> p = {};
    p.A = f.w.operand(false);
    p.B = f.x.operand(false);
    p.depth = round_up(K, 8);
    p.e = e;
    return run_product<kForward>(p, f.shape, f.partial, stream);
}

// ---- backward ------------------------------------------------------------

namespace {

struct BackwardPlan {
    bool make_dz;   // dz is written (to the workspace), not dy itself
    int64_t width;  // of dz's rows there
    int dz_lanes;
    int64_t dz_groups, chunk, chunks;
    Source w;
    uint16_t* dz = nullptr;
    float* sums = nullptr;
    uint16_t* x = nullptr;
    Gradients g;
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
    b.g = choose_gradients(T, N, K, a.dx && T && N && K, a.dweight && T && N && K);
    // the 256-wide tiles read x from here, widened (tile_product.h)
    if (a.dweight && N && b.g.weight.bi == 256) b.x = c.take<uint16_t>(T * act8_pitch(K));
    int64_t floats = 0;
    if (a.dx) floats = std::max(floats, partial_floats(b.g.in, K, T));
    if (a.dweight) floats = std::max(floats, partial_floats(b.g.weight, K, N));
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
    Product<Epilogue> x = {}, w = {};
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
        if (b.g.weight.bi == 256) {
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
    return run_gradients(b.g, w, a.dweight && N, x, a.dx && T, b.partial, stream);
}
