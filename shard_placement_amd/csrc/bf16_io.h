// bf16_io.h -- loads, stores and conversions of bf16 rows, shared by the
// checkpoint kernels and the layer products.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tide {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
// The same without alignment beyond the element's: rows may start anywhere.
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef u32x4v u32x4_any __attribute__((aligned(2)));

#define TIDE_GLOBAL_AS __attribute__((address_space(1)))

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float bf16_at(const uint16_t* p) {
    return __uint_as_float((uint32_t) * (const TIDE_GLOBAL_AS uint16_t*)p << 16);
}

// Round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint16_t to_bf16(float f) {
    return __builtin_bit_cast(uint16_t, (__bf16)f);
}
__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

// Eight consecutive elements of a row, of which the first n are there.
__device__ __forceinline__ void load8(const uint16_t* p, int64_t n, float (&v)[8]) {
    if (n >= 8) {
        const u32x4v w = *(const TIDE_GLOBAL_AS u32x4_any*)p;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = bf16_lo(w[k]);
            v[2 * k + 1] = bf16_hi(w[k]);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? bf16_at(p + k) : 0.0f;
}

__device__ __forceinline__ void store8(uint16_t* p, int64_t n, const float (&v)[8]) {
    if (n >= 8) {
        const u32x4v w = {to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3]), to_bf16x2(v[4], v[5]),
                          to_bf16x2(v[6], v[7])};
        *(TIDE_GLOBAL_AS u32x4_any*)p = w;
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < n) *(TIDE_GLOBAL_AS uint16_t*)(p + k) = to_bf16(v[k]);
}

// Four consecutive elements of a row, of which the first n are there.
__device__ __forceinline__ void load4(const uint16_t* p, int64_t n, float (&v)[4]) {
    if (n >= 4) {
        const u32x2 w = *(const TIDE_GLOBAL_AS u32x2_any*)p;
        v[0] = bf16_lo(w.x);
        v[1] = bf16_hi(w.x);
        v[2] = bf16_lo(w.y);
        v[3] = bf16_hi(w.y);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = k < n ? bf16_at(p + k) : 0.0f;
}

__device__ __forceinline__ void store4(uint16_t* p, int64_t n, const float (&v)[4]) {
    if (n >= 4) {
        const u32x2 w = {to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3])};
        *(TIDE_GLOBAL_AS u32x2_any*)p = w;
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (k < n) *(TIDE_GLOBAL_AS uint16_t*)(p + k) = to_bf16(v[k]);
}

}  // namespace tide
