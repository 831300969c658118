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

// The larger of m and |x|, a NaN if either is one.
__device__ __forceinline__ float max_magnitude(float m, float x) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(x)));
    return m;
}

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

// Two of them in a word, `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float load_as_float(const float *p) { return *p; }
__device__ __forceinline__ float load_as_float(const uint16_t *p) { return bf16_bits_to_float(*p); }
__device__ __forceinline__ void store_from_float(float *p, float x) { *p = x; }
__device__ __forceinline__ void store_from_float(uint16_t *p, float x) { *p = to_bf16(x); }


constexpr int kRowThreads = 256;

// U consecutive elements of a row, as they lie in memory: fp32 values, or pairs of
// bf16 in words (a word's halves become fp32 by one shift or mask each).
template <int U>
struct alignas(U * 4 > 16 ? 16 : U * 4) RawF32 {
    float v[U];
    __device__ __forceinline__ float get(int j) const { return v[j]; }
    __device__ __forceinline__ void set(int j, float x) { v[j] = x; }
    __device__ __forceinline__ void set_all(const float (&x)[U]) {
#pragma unroll
        for (int j = 0; j < U; ++j) v[j] = x[j];
    }
};
template <int U>
struct alignas(U * 2 > 16 ? 16 : U * 2) RawBf16 {
    uint32_t w[U / 2];
    __device__ __forceinline__ float get(int j) const {
        return __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
    }
    // in order of j
    __device__ __forceinline__ void set(int j, uint16_t x) {
        w[j / 2] = j & 1 ? w[j / 2] | static_cast<uint32_t>(x) << 16 : static_cast<uint32_t>(x);
    }
    __device__ __forceinline__ void set_all(const float (&x)[U]) {
#pragma unroll
        for (int j = 0; j < U; j += 2) w[j / 2] = pack_bf16(x[j], x[j + 1]);
    }
};
template <>
struct RawBf16<1> {
    uint16_t v;
    __device__ __forceinline__ float get(int) const { return bf16_bits_to_float(v); }
    __device__ __forceinline__ void set_all(const float (&x)[1]) { v = to_bf16(x[0]); }
};

// The largest magnitude pattern of a unit, as an fp32 pattern.
template <int U>
__device__ __forceinline__ uint32_t unit_max(const RawF32<U> &r, uint32_t m) {
#pragma unroll
    for (int j = 0; j < U; ++j) m = max(m, abs_bits(r.v[j]));
    return m;
}
// bf16 patterns order like fp32 ones: pairs of them are compared at once.
template <int U>
__device__ __forceinline__ uint32_t unit_max(const RawBf16<U> &r, uint32_t m) {
    uint32_t p = r.w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int j = 1; j < U / 2; ++j) p = __vmaxu2(p, r.w[j] & 0x7FFF7FFFu);
    return max(m, max(p & 0xFFFF0000u, p << 16));
}

template <typename T, int U>
struct RawOf;
template <int U>
struct RawOf<float, U> {
    using type = RawF32<U>;
};
template <int U>
struct RawOf<uint16_t, U> {
    using type = RawBf16<U>;
};

template <typename T, int U>
__device__ __forceinline__ typename RawOf<T, U>::type load_unit(const T *p) {
    return *reinterpret_cast<const typename RawOf<T, U>::type *>(p);
}

// The codes of eight elements, four to a word.
__device__ __forceinline__ void store_codes(int8_t *p, const uint32_t (&c)[8]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_codes(c[0], c[1], c[2], c[3]), pack_codes(c[4], c[5], c[6], c[7]));
}

// U fp32 values rounded to the output's type.
template <typename T, int U>
__device__ __forceinline__ void store_values(T *p, const float (&v)[U]) {
    typename RawOf<T, U>::type r;
    r.set_all(v);
    *reinterpret_cast<typename RawOf<T, U>::type *>(p) = r;
}

// A sum's two scales become one factor, v * (xs * ws), so that the sum is rounded once more.
// Where the factor is subnormal or leaves fp32's range, which says nothing about the result,
// the scales' fractions are multiplied and their exponents applied last.  Scales outside 2^-63 ..
// 2^63, whose products may do so, are "far"; 0 is not (its products are 0 whatever the other
// scale), nor is what is not finite.
__device__ __forceinline__ bool far_scale(float s) {
    const uint32_t e = (__float_as_uint(s) >> 23) & 0xFFu;
    return (e < 64u || e > 190u) && e != 255u && s != 0.0f;
}

// s = fraction * 2^exponent, 1 <= |fraction| < 2; 0 and what is not finite as they are.
__device__ __forceinline__ float fraction(float s, int &exponent) {
    const bool small = fabsf(s) < 0x1p-126f;
    const uint32_t b = __float_as_uint(small ? __fmul_rn(s, 0x1p24f) : s), e = (b >> 23) & 0xFFu;
    exponent = 0;
    if (e == 0u || e == 255u) return s;
    exponent = static_cast<int>(e) - (small ? 151 : 127);
    return __uint_as_float((b & 0x807FFFFFu) | 0x3F800000u);
}

// v is 0 or 1 <= |v| < 2^40.  Halves of the exponent have one sign, so only the last product
// can leave the normal range.
__device__ __forceinline__ float scaled_far(float v, float xs, float ws) {
    int ex, ew;
    const float p = __fmul_rn(v, __fmul_rn(fraction(xs, ex), fraction(ws, ew)));
    const int e = max(-252, min(254, ex + ew)), half = e / 2;
    return __fmul_rn(__fmul_rn(p, __int_as_float((127 + half) << 23)), __int_as_float((127 + e - half) << 23));
}
// The same as a call, to keep it out of unrolled loops.
static __device__ __noinline__ float scaled_far_call(float v, float xs, float ws) { return scaled_far(v, xs, ws); }

// A team of `lanes` threads (a power of two, 8 to THREADS) and the rows it owns.
struct Team {
    uint32_t lanes, lane, first, stride;
    __device__ explicit Team(uint32_t lanes_) : lanes(lanes_) {
        const uint32_t teams = blockDim.x / lanes;
        lane = threadIdx.x & (lanes - 1);
        first = blockIdx.x * teams + threadIdx.x / lanes;
        stride = gridDim.x * teams;
    }
};

// The largest of v[0..N) over the team, in every lane.  A team of several warps
// meets in shared memory, in one of two buffers used in turn, so one block barrier
// a row is enough; every thread of the block takes part.
template <int N>
__device__ __forceinline__ void team_max(uint32_t (&v)[N], uint32_t lanes, uint32_t (*red)[32][N], int &turn) {
    for (uint32_t o = min(lanes, 32u) >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = max(v[i], __shfl_xor_sync(kFull, v[i], o));
    if (lanes > 32) {
        const uint32_t warp = threadIdx.x >> 5, w0 = threadIdx.x / lanes * (lanes >> 5);
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[turn][warp][i] = v[i];
        __syncthreads();
        for (uint32_t w = 0; w < (lanes >> 5); ++w)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = max(v[i], red[turn][w0 + w][i]);
        turn ^= 1;
    }
}

// Codes of U elements under a scale that neither zeroes nor saturates them.
template <int U, typename Get>
__device__ __forceinline__ void encode_unit(int8_t *out, float inverse, Get get) {
    uint32_t c[U];
#pragma unroll
    for (int j = 0; j < U; ++j) c[j] = code_bits(get(j), inverse);
    store_codes(out, c);
}

// U codes as they lie in memory.  A code becomes a float without a conversion
// instruction (those run at a quarter of the rate): its byte, offset by 128, under
// the exponent of 2^23, minus 2^23 + 128.
template <int U>
struct alignas(U) RawCodes {
    uint32_t w[U / 4];
    __device__ __forceinline__ float get(int j) const {
        return __fsub_rn(__uint_as_float(__byte_perm(w[j / 4] ^ 0x80808080u, 0x4B000000u, 0x7440 + (j & 3))), 8388736.0f);
    }
};
template <>
struct RawCodes<1> {
    int8_t b;
    __device__ __forceinline__ float get(int) const { return static_cast<float>(b); }
};

// Four codes -> two f16 pairs: each byte, offset by 128, under the exponent of
// 2^10 (1024 + 128 + code), minus 1152.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    w ^= 0x80808080u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(w, 0x64646464u, 0x4140)), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(w, 0x64646464u, 0x4342)), "r"(0x64806480u));
}

// sigma(g) = 1 / (1 + exp(-g)) and 1 - sigma(g).
//
// fp32 inputs: both to fp32's relative precision.  With e = exp(-|g|) <= 1 and r = 1 / (1 + e)
// they are r and e r, in this order for g >= 0 and in the other for g < 0: nothing overflows, and
// the smaller one is not a difference.  expf() is within 2 units in the last place and 1 + e
// rounds once; 1 + e is in [1, 2], where the hardware's reciprocal is within one unit.
//
// bf16 inputs: the hardware's exponential (base 2) and reciprocal.  The argument's rounding (half a
// unit of |g| log2(e)) and the constant's make up to 2^-17 of sigma at |g| = 80, a 256th of the rounding
// of a bf16 result and less of a code's step; a sigma below 2^-126 (g < -87.3) is 0.  With the form
// above the forward pass of 16384 x 2048 bf16 takes 53 us against 46; in fp32, whose loads are
// twice as long, it costs 71 against 66, and 90.5 against 90 backwards.
struct Sigma {
    float s, other;
};
template <typename T>
__device__ __forceinline__ Sigma sigma_of(float g) {
    float e, r;
    if constexpr (sizeof(T) == 2) {
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(g, -1.4426950408889634f)));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.0f, e)));
        return {r, __fsub_rn(1.0f, r)};
    } else {
        e = expf(-fabsf(g));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.0f, e)));
        const float er = __fmul_rn(e, r);
        return {g < 0.0f ? er : r, g < 0.0f ? r : er};
    }
}

// T: the type of the inputs.
template <typename T>
__device__ __forceinline__ float swiglu(float g, float u) {
    return __fmul_rn(__fmul_rn(g, sigma_of<T>(g).s), u);
}

// Lanes of a team that covers `units` with up to V units per lane: 8 to `most`.
inline uint32_t lanes_for(uint32_t units, int v, uint32_t most) {
    uint32_t lanes = 8;
    while (lanes < most && lanes * v < units) lanes *= 2;
    return lanes;
}

template <typename P>
cudaError_t launch_rows(void (*kernel)(const P, uint32_t), const P &p, uint32_t lanes, int threads,
                        cudaStream_t stream) {
    const uint64_t teams = threads / lanes;
    const int grid = persistent_grid(reinterpret_cast<const void *>(kernel), threads, (p.rows + teams - 1) / teams);
    kernel<<<grid, threads, 0, stream>>>(p, lanes);
    return cudaGetLastError();
}

}  // namespace qc
