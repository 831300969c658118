// qc_int8_rows.cuh -- the row code of the 8-bit layer: int8 codes under one
// power-of-two scale.
//
// For a row with a = max|x| > 0, s = 2^e is the smallest power of two >= 2^-126
// with a / s < 127.5.  Writing a = m * 2^E with 1 <= m < 2, a / 2^(E-6) = 64 m is
// in [64, 128), so e = E - 6, plus one where 64 m >= 127.5, which is where the
// 23-bit fraction field is 0x7F0000 or more: adding 0x10000 to a's bit pattern
// carries into the exponent field there and nowhere below.  s is at most 2^121,
// so that 127 s is finite in fp32 and bf16: a row beyond 127.5 * 2^121 saturates.
#pragma once

#include "qc_device.cuh"

namespace qc {

// Biased exponent field of the scale for the bit pattern of a finite a > 0.
__device__ __forceinline__ uint32_t row_scale_exponent(uint32_t abits) {
    const int e = static_cast<int>((abits + 0x10000u) >> 23) - 6;
    return static_cast<uint32_t>(e < 1 ? 1 : e > 248 ? 248 : e);
}

constexpr float kRowCap = 0x1.FCp127f;  // 127 * 2^121

struct RowScale {
    float scale;    // as stored: 0 for a row of zeros, NaN for one with a NaN or an infinity
    float inverse;  // 1 / scale (exact), or 0 where every code is 0
    bool saturates; // some |x| is above kRowCap and has to be clamped to it first
};

// From the largest |x| bit pattern of the row (patterns of |x| order like the
// values, infinities and NaN above every finite one).
__device__ __forceinline__ RowScale row_scale_of(uint32_t abits) {
    if (abits == 0u) return {0.0f, 0.0f, false};
    if (abits >= 0x7F800000u) return {__uint_as_float(0x7FC00000u), 0.0f, false};
    const uint32_t e = row_scale_exponent(abits);
    return {__uint_as_float(e << 23), __uint_as_float((254u - e) << 23), abits > __float_as_uint(kRowCap)};
}

__device__ __forceinline__ float clamp_to_cap(float x) { return fminf(fmaxf(x, -kRowCap), kRowCap); }

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// rint(x * inverse), ties to even, in the low byte (two's complement): the exact
// product plus 1.5 * 2^23 leaves the integer in the low mantissa bits.  A row
// whose codes are all 0 has inverse 0; an infinity or NaN there is masked.
__device__ __forceinline__ uint32_t code_bits(float x, float inverse) {
    return __float_as_uint(__fmaf_rn(x, inverse, 12582912.0f));
}

// The low bytes of four code_bits() in one word, the first lowest.
__device__ __forceinline__ uint32_t pack_codes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Round to nearest even to bf16 bits; a NaN stays one.
__device__ __forceinline__ uint16_t to_bf16(float x) {
    unsigned short r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float load_as_float(const float *p) { return *p; }
__device__ __forceinline__ float load_as_float(const uint16_t *p) { return bf16_bits_to_float(*p); }
__device__ __forceinline__ void store_from_float(float *p, float x) { *p = x; }
__device__ __forceinline__ void store_from_float(uint16_t *p, float x) { *p = to_bf16(x); }

}  // namespace qc
