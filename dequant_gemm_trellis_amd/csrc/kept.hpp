// Rows kept in 8 bits (trellis_keep): their device-side coding, loads of rows at
// any boundary, and the launchers of kept.hip (internal to libtrellis.so; callers
// have validated arguments).
//
// 32 values of a row share E, the largest exponent field of their bf16 values. A
// value x is held as q = x 2^(133 - E), rounded half to even and cut off at +-127,
// and stands for q 2^(E - 133). The group's largest value has |x| in [2^(E - 127),
// 2^(E - 126)), i.e. |q| in [64, 127.5], so the error is at most half of 2^(E -
// 133); where E is 0 every value is a multiple of 2^-133 and held exactly. q has 7
// bits, so a held value is a bf16 value, and every step below is exact but the one
// rounding. A group with an infinity or NaN (E = 255) stands for NaN.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "launch.hpp"

namespace trellis {

constexpr int kKeptGroup = 32;

struct KeptRows {
    const int8_t* codes;       // [rows][width]
    const uint8_t* exponents;  // [rows][ceil(width / 32)]
};

hipError_t launch_keep(const uint16_t* x, int rows, int width, int8_t* codes, uint8_t* exponents,
                       hipStream_t st);
hipError_t launch_restore(const KeptRows& x, int rows, int width, uint16_t* out, hipStream_t st);

// gu [rows][2 inter]; codes and exponents of gu as [2 rows][inter], or null.
hipError_t launch_swiglu(const uint16_t* gu, int rows, int inter, uint16_t* h, int8_t* codes,
                         uint8_t* exponents, hipStream_t st);
// From gu, or, where it is null, from `kept`; h may be null.
hipError_t launch_swiglu_backward(const uint16_t* dh, const uint16_t* gu, const KeptRows& kept, int rows,
                                  int inter, uint16_t* dgu, uint16_t* h, hipStream_t st);

#ifdef __HIP__

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// Wide accesses at the boundary of an element: one instruction each, as global
// memory takes them anywhere.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

// 8 values of which `left` are in the row (the others are 0), and back.
__device__ __forceinline__ u32x4 load_values(const uint16_t* __restrict__ p, int left) {
    if (left >= 8) return *reinterpret_cast<const u32x4_any*>(p);
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t lo = 2 * d < left ? p[2 * d] : 0u, hi = 2 * d + 1 < left ? p[2 * d + 1] : 0u;
        v[d] = lo | (hi << 16);
    }
    return v;
}

__device__ __forceinline__ void store_values(uint16_t* __restrict__ p, int left, const u32x4& v) {
    if (left >= 8) {
        *reinterpret_cast<u32x4_any*>(p) = v;
        return;
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        if (2 * d < left) p[2 * d] = static_cast<uint16_t>(v[d]);
        if (2 * d + 1 < left) p[2 * d + 1] = static_cast<uint16_t>(v[d] >> 16);
    }
}

__device__ __forceinline__ u32x2 load_codes(const int8_t* __restrict__ p, int left) {
    if (left >= 8) return *reinterpret_cast<const u32x2_any*>(p);
    u32x2 v = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < left) v[i / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(p[i])) << (8 * (i % 4));
    return v;
}

__device__ __forceinline__ void store_codes(int8_t* __restrict__ p, int left, const u32x2& v) {
    if (left >= 8) {
        *reinterpret_cast<u32x2_any*>(p) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < left) p[i] = static_cast<int8_t>(v[i / 4] >> (8 * (i % 4)));
}

// 2^(E - 133) as a float32 (a subnormal for E <= 6), NaN for E = 255.
__device__ __forceinline__ float kept_step(uint32_t exponent) {
    const uint32_t normal = (exponent - 6u) << 23, small = 1u << (exponent + 16u);
    return __uint_as_float(exponent == 255u ? 0x7FC00000u : exponent > 6u ? normal : small);
}

// The 8 bf16 values that codes of one group stand for (the float32 product is a
// bf16 value: its upper half).
__device__ __forceinline__ u32x4 kept_values(const u32x2& codes, uint32_t exponent) {
    const float step = kept_step(exponent);
    u32x4 v;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t w = codes[d / 2] >> (16 * (d % 2));
        const float lo = static_cast<float>(static_cast<int8_t>(w)) * step;
        const float hi = static_cast<float>(static_cast<int8_t>(w >> 8)) * step;
        v[d] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
    }
    return v;
}

// The largest exponent field of 8 values.
__device__ __forceinline__ uint32_t largest_exponent(const u32x4& v) {
    uint32_t e = 0;
#pragma unroll
    for (int d = 0; d < 4; ++d) e = max(e, max((v[d] >> 7) & 255u, (v[d] >> 23) & 255u));
    return e;
}

// The largest of a value over the four lanes 4 i .. 4 i + 3, which hold a group.
__device__ __forceinline__ uint32_t largest_of_four(uint32_t v) {
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xF, 0xF, true)));
    return max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xF, 0xF, true)));
}

// Codes of 8 values of a group with exponent E: adding 1.5 * 2^23 leaves the rounded
// integer (half to even) in the low bits.
__device__ __forceinline__ u32x2 kept_codes(const u32x4& v, uint32_t exponent) {
    const int shift = 133 - static_cast<int>(exponent);
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = v[i / 2];
        const float x = ldexpf(__uint_as_float(i % 2 ? w & 0xFFFF0000u : w << 16), shift);
        q[i] = __float_as_uint(__builtin_amdgcn_fmed3f(x, -127.f, 127.f) + 12582912.f);
    }
    u32x2 r;
#pragma unroll
    for (int d = 0; d < 2; ++d) {
        const uint32_t lo = __builtin_amdgcn_perm(q[4 * d + 1], q[4 * d], 0x0C0C0400u);
        const uint32_t hi = __builtin_amdgcn_perm(q[4 * d + 3], q[4 * d + 2], 0x04000C0Cu);
        r[d] = exponent == 255u ? 0u : lo | hi;
    }
    return r;
}

#endif  // __HIP__

}  // namespace trellis
