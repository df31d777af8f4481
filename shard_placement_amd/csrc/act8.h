// act8.h -- the 8-bit activation checkpoint's format, shared by its kernels
// (act8.hip) and the products that write or read it (linear.hip).
//
// A checkpoint of a [rows, cols] matrix is rows * pitch bytes of e4m3 values
// (row-major, pitch = cols rounded up to 32, the padding columns 0) followed
// by rows * pitch / 32 scale bytes, one for each 32 consecutive columns of a
// row.  Scale byte e + 127 stands for 2^e; an element's value is its e4m3
// value times its block's scale.  With a the largest finite |x| of the block,
//   e = the smallest integer with a <= 448 * 2^e, but at least -110,
// so nothing saturates, and the scale being a power of two, dividing by it is
// exact and the only rounding is the one to e4m3 (half a step: 2^-4 relative,
// 2^-10 of the scale for e4m3's subnormals).  With e >= -110 every non-zero
// value is at least 2^-119, so values are normal binary32 and, having four
// significant bits, exactly bf16: reading a checkpoint back rounds nothing (in
// a block that reaches 2^127, values that round up to 2^128 read back as
// infinity).
// Elements that are not finite become the e4m3 NaN and leave the block's
// scale to the others.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace tide {

constexpr int kActBlock = 32;
constexpr int kActMinExp = -110;

__host__ __device__ constexpr int64_t act8_pitch(int64_t cols) {
    return (cols + kActBlock - 1) / kActBlock * kActBlock;
}
__host__ __device__ constexpr int64_t act8_scale_offset(int64_t rows, int64_t cols) {
    return rows * act8_pitch(cols);
}
__host__ __device__ constexpr int64_t act8_bytes(int64_t rows, int64_t cols) {
    return rows * (act8_pitch(cols) + act8_pitch(cols) / kActBlock);
}

// The block's exponent from its maximum.  448 = 1.75 * 2^8: a = m * 2^k has
// exponent k - 8 for m <= 1.75 and k - 7 above, and adding one less than
// 2^23 - 0x600000 to the bits carries into the exponent exactly then.
__device__ __forceinline__ int act8_exp(float amax) {
    const int e = (int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 127 - 8;
    return e > kActMinExp ? e : kActMinExp;
}

// A scale byte's scale.
__device__ __forceinline__ float act8_scale(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float act8_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Four elements to four e4m3 bytes (round to nearest even); inv = 2^-e.
__device__ __forceinline__ uint32_t act8_pack4(const float* x, float inv) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inv, x[1] * inv, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2] * inv, x[3] * inv, v, true);
}

// A lane's 8 of a block's 32 elements, the four lanes of a quad together:
// their bytes, and the block's exponent.  Magnitudes are compared as integers,
// which orders them, with whatever is not finite above the rest: only a block
// that has such elements looks at each.
typedef uint32_t act8_u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t act8_quad_max(uint32_t m) {
    m = max(m, (uint32_t)__shfl_xor((int)m, 1));
    return max(m, (uint32_t)__shfl_xor((int)m, 2));
}

__device__ __forceinline__ int act8_pack8(float (&x)[8], act8_u32x2* q) {
    constexpr uint32_t kInf = 0x7f800000u;
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(x[k]) & 0x7fffffffu);
    m = act8_quad_max(m);
    if (m >= kInf) {
        m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t b = __float_as_uint(x[k]) & 0x7fffffffu;
            if (b < kInf)
                m = max(m, b);
            else
                x[k] = __builtin_nanf("");  // the conversion could saturate an infinity
        }
        m = act8_quad_max(m);
    }
    const int e = act8_exp(__uint_as_float(m));
    const float inv = act8_pow2(-e);
    *q = act8_u32x2{act8_pack4(x, inv), act8_pack4(x + 4, inv)};
    return e;
}

// The four values of a word of e4m3 bytes, times the scale.
__device__ __forceinline__ void act8_unpack4(uint32_t w, float s, float (&v)[4]) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    v[0] = lo.x * s;
    v[1] = lo.y * s;
    v[2] = hi.x * s;
    v[3] = hi.y * s;
}

// Two bytes of a word (the upper two with HIGH) as bf16, times the scale: no
// rounding, bf16 has the value's four significant bits.
template <bool HIGH>
__device__ __forceinline__ uint32_t act8_bf16x2(uint32_t w, float s) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, s, HIGH);
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ void act8_unpack8(act8_u32x2 w, float s, float (&v)[8]) {
    float lo[4], hi[4];
    act8_unpack4(w.x, s, lo);
    act8_unpack4(w.y, s, hi);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[k] = lo[k];
        v[k + 4] = hi[k];
    }
}

}  // namespace tide
