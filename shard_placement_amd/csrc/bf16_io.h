// bf16_io.h -- loads, stores and conversions of bf16 rows, shared by the
// checkpoint kernels and the layer products.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tide {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
// The same without alignment beyond the element's: rows may start anywhere.
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

// Eight consecutive elements as they lie in memory.  ONCE: they are read once
// and need no place in the caches.
template <bool ONCE = false>
__device__ __forceinline__ u32x4v load8_raw(const uint16_t* p) {
    if constexpr (ONCE)
        return __builtin_nontemporal_load((const TIDE_GLOBAL_AS u32x4_any*)p);
    else
        return *(const TIDE_GLOBAL_AS u32x4_any*)p;
}
__device__ __forceinline__ void widen(u32x4v w, float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = bf16_lo(w[k]);
        v[2 * k + 1] = bf16_hi(w[k]);
    }
}

// Eight consecutive elements of a row, of which the first n are there.
__device__ __forceinline__ void load8(const uint16_t* p, int64_t n, float (&v)[8]) {
    if (n >= 8) {
        widen(load8_raw(p), v);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? bf16_at(p + k) : 0.0f;
}

template <bool ONCE = false>
__device__ __forceinline__ void store8(uint16_t* p, int64_t n, const float (&v)[8]) {
    if (n >= 8) {
        const u32x4v w = {to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3]), to_bf16x2(v[4], v[5]),
                          to_bf16x2(v[6], v[7])};
        if constexpr (ONCE)
            __builtin_nontemporal_store(w, (TIDE_GLOBAL_AS u32x4_any*)p);
        else
            *(TIDE_GLOBAL_AS u32x4_any*)p = w;
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < n) *(TIDE_GLOBAL_AS uint16_t*)(p + k) = to_bf16(v[k]);
}

}  // namespace tide
