// attn_common.hpp - pieces shared by the attention kernels on gfx950: operand types, widening of
// e4m3 codes, query loads, reductions over a wave, index arithmetic.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bfp8 {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xFF800000u); }

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));

// Eight e4m3 codes (two registers) times a power of two, as bf16 (exact).
__device__ __forceinline__ bf8v widen8(int w0, int w1, float scale) {
    const bf2v a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, false);
    const bf2v b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, true);
    const bf2v c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, false);
    const bf2v d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, true);
    return bf8v{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Eight elements of a bf16 query row (negated for a negative scale).
__device__ __forceinline__ bf8v load_q8(const uint16_t* p, bool vec, bool negate) {
    uint4 x;
    if (vec) {
        x = *(const uint4*)p;
    } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = (uint32_t)p[2 * j] | ((uint32_t)p[2 * j + 1] << 16);
        x = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (negate) {
        asm volatile("");                                       // a branch: otherwise the load is waited for here
        x = make_uint4(x.x ^ 0x80008000u, x.y ^ 0x80008000u, x.z ^ 0x80008000u, x.w ^ 0x80008000u);
    }
    return __builtin_bit_cast(bf8v, x);
}

// x / y for 0 <= x < 2^52, 0 < y, a quotient below 2^31: by the reciprocal in 64-bit floating point,
// refined twice, which is off by one at most.  The compiler's 64-bit division takes a kilobyte of
// code, and what a short call spends its time on is code that it runs for the first time.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
    const double d = (double)y;
    double inv = __builtin_amdgcn_rcp(d);
    inv = __builtin_fma(__builtin_fma(-d, inv, 1.0), inv, inv);
    inv = __builtin_fma(__builtin_fma(-d, inv, 1.0), inv, inv);
    int64_t q = (uint32_t)((double)x * inv);
    const int64_t left = x - q * y;
    if (left < 0) q -= 1;
    if (left >= y) q += 1;
    return q;
}

// How many of the lanes' conditions hold, from the first lane on, less one; at least 0.
__device__ __forceinline__ int last_of(bool holds) { return max(__popcll(__ballot(holds)) - 1, 0); }

// Maximum and sum of a lane and the one 32 lanes away.
__device__ __forceinline__ float half_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

}  // namespace bfp8
