// qc_int8_ragged.cu -- the row codes and the gated activation for rows that start
// anywhere (odd lengths, odd strides, shifted buffers): the kernels of qc_int8_rows.cu
// with units of eight elements laid on the output's 8- or 16-byte boundaries, so that
// stores stay vectors.  The input, which then starts anywhere, is read as the aligned
// vectors around a unit and shifted in registers; one element at a time (a load and a
// byte store per element) 16384 x 8191 bf16 took 221 us to encode, this 117.  Vectors
// that reach outside the matrix are not read: those units load single elements.
#include <algorithm>

#include "qc_chain.cuh"
#include "qc_int8_rows.cuh"
#include "qc_internal.h"

namespace qc {
namespace {

// Elements e .. e + 7 of a row of `dim` elements, zero where that is outside the row.
// [begin, end) is the whole matrix.  ALIGNED: element e starts on 16 bytes.
template <bool ALIGNED, typename T>
__device__ __forceinline__ typename RawOf<T, 8>::type load8_any(const T *row, int e, int dim, const T *begin, const T *end) {
    using R = typename RawOf<T, 8>::type;
    constexpr int kVectors = (sizeof(T) == 2 ? 1 : 2) + (ALIGNED ? 0 : 1), kWords = 4 * kVectors, kOut = sizeof(T) * 2;
    const uintptr_t p = reinterpret_cast<uintptr_t>(row) + static_cast<intptr_t>(e) * static_cast<int>(sizeof(T));
    const uintptr_t a = p & ~static_cast<uintptr_t>(15);
    const bool inside = ALIGNED || (a >= reinterpret_cast<uintptr_t>(begin) && a + 16 * kVectors <= reinterpret_cast<uintptr_t>(end));
    if (inside && e >= 0 && e + 8 <= dim) {
        union {
            uint4 v[kVectors];
            uint32_t w[kWords];
            R r;
        } u;
#pragma unroll
        for (int i = 0; i < kVectors; ++i) u.v[i] = __ldg(reinterpret_cast<const uint4 *>(a) + i);
        if constexpr (!ALIGNED) {
            const bool two = (p & 8) != 0, one = (p & 4) != 0;
#pragma unroll
            for (int i = 0; i + 2 < kWords; ++i) u.w[i] = two ? u.w[i + 2] : u.w[i];
#pragma unroll
            for (int i = 0; i < kOut + (sizeof(T) == 2 ? 1 : 0); ++i) u.w[i] = one ? u.w[i + 1] : u.w[i];
            if constexpr (sizeof(T) == 2)
#pragma unroll
                for (int i = 0; i < kOut; ++i) u.w[i] = __funnelshift_r(u.w[i], u.w[i + 1], 8 * static_cast<uint32_t>(p & 2));
        }
        return u.r;
    }
    R r;  // the ends of a row
#pragma unroll
    for (int j = 0; j < 8; ++j) r.set(j, e + j >= 0 && e + j < dim ? row[e + j] : static_cast<T>(0));
    return r;
}

// Codes of the elements e .. e + 7, inside the row, at out + e (8-byte aligned).
__device__ __forceinline__ void store8_any(int8_t *out, int e, int dim, const uint32_t (&c)[8]) {
    if (e >= 0 && e + 8 <= dim) {
        store_codes(out + e, c);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (e + j >= 0 && e + j < dim) out[e + j] = static_cast<int8_t>(c[j] & 0xFFu);
    }
}

template <typename Get>
__device__ __forceinline__ void encode_any(int8_t *out, int e, int dim, const RowScale &s, Get get) {
    uint32_t c[8];
    if (s.inverse == 0.0f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = 0u;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = code_bits(s.saturates ? clamp_to_cap(get(j)) : get(j), s.inverse);
    }
    store8_any(out, e, dim, c);
}

// Units of eight on the codes' 8-byte boundaries: unit u is elements 8 u - phase on.
__device__ __forceinline__ int phase8(const void *p) { return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 7u); }

// ALIGNED: a unit of codes on 8 bytes is a unit of the input on 16 or 32, as in a dense
// matrix from an aligned base, whatever the length of its rows.
template <typename T, bool ALIGNED, int V, bool HELD, int BLOCKS>
__global__ void __launch_bounds__(kRowThreads, BLOCKS) ragged_encode(const RowCodesParams P, uint32_t lanes) {
    __shared__ uint32_t red[2][32][1];
    using R = typename RawOf<T, 8>::type;
    const Team team(lanes);
    const int dim = static_cast<int>(P.dim);
    const uint32_t chunk = lanes * V;
    const T *begin = static_cast<const T *>(P.x), *end = begin + (P.rows - 1) * P.x_stride + P.dim;
    int turn = 0;
    for (uint64_t r0 = team.first - threadIdx.x / lanes; r0 < P.rows; r0 += team.stride) {
        const uint64_t r = r0 + threadIdx.x / lanes;
        const bool live = r < P.rows;
        const T *x = begin + (live ? r : 0) * P.x_stride;
        int8_t *out = P.codes + (live ? r : 0) * P.dim;
        const int phase = phase8(out);
        const uint32_t units = static_cast<uint32_t>(dim + phase + 7) / 8;
        R held[V];
        uint32_t m[1] = {0};
        auto load = [&](uint32_t base) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t u = base + v * lanes + team.lane;
                if (u < units) held[v] = load8_any<ALIGNED>(x, static_cast<int>(8 * u) - phase, dim, begin, end);
            }
        };
        for (uint32_t base = 0; base < (HELD ? 1u : units); base += chunk) {
            load(base);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (base + v * lanes + team.lane < units) m[0] = unit_max(held[v], m[0]);
        }
        team_max(m, lanes, red, turn);
        if (!live) continue;
        const RowScale s = row_scale_of(m[0]);
        if (team.lane == 0) P.row_scale[r] = s.scale;
        for (uint32_t base = 0; base < (HELD ? 1u : units); base += chunk) {
            if (!HELD) load(base);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t u = base + v * lanes + team.lane;
                if (u < units) encode_any(out, static_cast<int>(8 * u) - phase, dim, s, [&](int j) { return held[v].get(j); });
            }
        }
    }
}

// U codes from element e on, anywhere, as words; [begin, end) is the whole matrix.
template <int U>
__device__ __forceinline__ RawCodes<U> load_codes_any(const int8_t *row, int e, int dim, const int8_t *begin, const int8_t *end) {
    RawCodes<U> c;
    const uintptr_t p = reinterpret_cast<uintptr_t>(row + e), a = p & ~static_cast<uintptr_t>(3);
    if (a >= reinterpret_cast<uintptr_t>(begin) && a + U + 4 <= reinterpret_cast<uintptr_t>(end)) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(a), shift = 8 * static_cast<uint32_t>(p & 3);
        uint32_t v[U / 4 + 1];
#pragma unroll
        for (int i = 0; i <= U / 4; ++i) v[i] = __ldg(w + i);
#pragma unroll
        for (int i = 0; i < U / 4; ++i) c.w[i] = __funnelshift_r(v[i], v[i + 1], shift);
    } else {
#pragma unroll
        for (int i = 0; i < U / 4; ++i) {
            c.w[i] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = e + 4 * i + j;
                if (at >= 0 && at < dim) c.w[i] |= static_cast<uint32_t>(static_cast<uint8_t>(row[at])) << (8 * j);
            }
        }
    }
    return c;
}

template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) ragged_decode(const RowCodesParams P, uint32_t lanes) {
    let_next_start();
    constexpr int U = 16 / sizeof(T);
    const Team team(lanes);
    const int dim = static_cast<int>(P.dim);
    for (uint64_t row = team.first; row < P.rows; row += team.stride) {
        const bool second = row >= P.first_rows;
        const uint64_t r = second ? row - P.first_rows : row, rows = second ? P.rows - P.first_rows : P.first_rows;
        const float *scale = second ? P.scale_in2 : P.scale_in;
        const float s = scale ? __ldg(scale + r) : 1.0f;
        const int8_t *begin = second ? P.codes_in2 : P.codes_in, *end = begin + rows * P.dim, *codes = begin + r * P.dim;
        T *out = static_cast<T *>(second ? P.out2 : P.out) + r * P.out_stride;
        const int phase = static_cast<int>((reinterpret_cast<uintptr_t>(out) & 15u) / sizeof(T));
        const uint32_t units = static_cast<uint32_t>(dim + phase + U - 1) / U;
        for (uint32_t base = team.lane; base < units; base += lanes * V) {
            RawCodes<U> c[V];
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (base + v * lanes < units)
                    c[v] = load_codes_any<U>(codes, static_cast<int>(U * (base + v * lanes)) - phase, dim, begin, end);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (base + v * lanes < units) {
                    const int e = static_cast<int>(U * (base + v * lanes)) - phase;
                    float f[U];
#pragma unroll
                    for (int j = 0; j < U; ++j) f[j] = __fmul_rn(c[v].get(j), s);
                    if (e >= 0 && e + U <= dim) {
                        store_values<T, U>(out + e, f);
                    } else {
#pragma unroll
                        for (int j = 0; j < U; ++j)
                            if (e + j >= 0 && e + j < dim) store_from_float(out + e + j, f[j]);
                    }
                }
        }
    }
}

// The three outputs of a row start on boundaries of their own: after the pass for the
// maxima, each is written in a pass of its own, with its inputs read again from L1 or
// L2.  ALIGNED: the saved codes' units are units of the input, as above.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kRowThreads, 4) ragged_swiglu_encode(const SwigluParams P, uint32_t lanes) {
    __shared__ uint32_t red[2][32][3];
    const Team team(lanes);
    const int dim = static_cast<int>(P.dim);
    const T *begin = static_cast<const T *>(P.in), *end = begin + (P.rows - 1) * P.in_stride + 2 * static_cast<uint64_t>(P.dim);
    int turn = 0;
    for (uint64_t r0 = team.first - threadIdx.x / lanes; r0 < P.rows; r0 += team.stride) {
        const uint64_t r = r0 + threadIdx.x / lanes;
        const bool live = r < P.rows;
        const T *gate = begin + (live ? r : 0) * P.in_stride, *up = gate + dim;
        int8_t *saved = P.saved_codes + (live ? r : 0) * 2 * P.dim, *out = P.h_codes + (live ? r : 0) * P.dim;
        const int step = 8 * static_cast<int>(lanes), lane8 = 8 * static_cast<int>(team.lane);
        uint32_t m[3] = {0, 0, 0};
#pragma unroll 1
        for (int e = lane8 - phase8(saved); e < dim; e += step) {
            const auto g = load8_any<ALIGNED>(gate, e, dim, begin, end);
            const auto w = load8_any<false>(up, e, dim, begin, end);
            m[0] = unit_max(g, m[0]);
            m[1] = unit_max(w, m[1]);
#pragma unroll
            for (int j = 0; j < 8; ++j) m[2] = max(m[2], abs_bits(swiglu<T>(g.get(j), w.get(j))));
        }
        team_max(m, lanes, red, turn);
        if (!live) continue;
        const RowScale sg = row_scale_of(m[0]), su = row_scale_of(m[1]), sh = row_scale_of(m[2]);
        if (team.lane == 0) {
            P.saved_scale[2 * r] = sg.scale;
            P.saved_scale[2 * r + 1] = su.scale;
            P.h_scale[r] = sh.scale;
        }
#pragma unroll 1
        for (int e = lane8 - phase8(saved); e < dim; e += step) {
            const auto g = load8_any<ALIGNED>(gate, e, dim, begin, end);
            encode_any(saved, e, dim, sg, [&](int j) { return g.get(j); });
        }
#pragma unroll 1
        for (int e = lane8 - phase8(saved + dim); e < dim; e += step) {
            const auto w = load8_any<ALIGNED>(up, e, dim, begin, end);
            encode_any(saved + dim, e, dim, su, [&](int j) { return w.get(j); });
        }
#pragma unroll 1
        for (int e = lane8 - phase8(out); e < dim; e += step) {
            const auto g = load8_any<false>(gate, e, dim, begin, end), w = load8_any<false>(up, e, dim, begin, end);
            encode_any(out, e, dim, sh, [&](int j) { return swiglu<T>(g.get(j), w.get(j)); });
        }
    }
}

// Rows of 16-bit elements, or of codes, copied to rows on 16-byte boundaries, as TMA
// reads them.
__global__ void __launch_bounds__(kRowThreads) ragged_copy16(const uint16_t *x, uint64_t stride, uint64_t rows, uint32_t dim,
                                                             uint16_t *out, uint64_t out_stride, uint32_t lanes) {
    let_next_start();
    after_previous();
    const Team team(lanes);
    const uint16_t *end = x + (rows - 1) * stride + dim;
    for (uint64_t r = team.first; r < rows; r += team.stride)
#pragma unroll 4
        for (uint32_t e = 8 * team.lane; e < dim; e += 8 * lanes)
            *reinterpret_cast<RawBf16<8> *>(out + r * out_stride + e) =
                load8_any<false>(x + r * stride, static_cast<int>(e), static_cast<int>(dim), x, end);
}

// Two matrices of codes of one row length in one launch.
__global__ void __launch_bounds__(kRowThreads) ragged_copy8(const int8_t *a, uint64_t rows_a, int8_t *to_a, const int8_t *b,
                                                            uint64_t rows_b, int8_t *to_b, uint32_t dim, uint64_t out_stride,
                                                            uint32_t lanes) {
    const Team team(lanes);
    for (uint64_t row = team.first; row < rows_a + rows_b; row += team.stride) {
        const bool second = row >= rows_a;
        const uint64_t r = second ? row - rows_a : row;
        const int8_t *codes = second ? b : a, *end = codes + (second ? rows_b : rows_a) * dim;
        int8_t *out = (second ? to_b : to_a) + r * out_stride;
#pragma unroll 4
        for (uint32_t e = 16 * team.lane; e < dim; e += 16 * lanes) {
            const RawCodes<16> c = load_codes_any<16>(codes + r * dim, static_cast<int>(e), static_cast<int>(dim), codes, end);
            *reinterpret_cast<uint4 *>(out + e) = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
        }
    }
}

// Whether codes on 8 bytes are elements of `esize` bytes on 8 of them, in every row.
bool in_step(const void *x, uint64_t x_stride, size_t esize, const void *codes, uint64_t dim) {
    return x_stride == dim && reinterpret_cast<uintptr_t>(x) % (8 * esize) == reinterpret_cast<uintptr_t>(codes) % 8 * esize;
}

// Lanes of a team that goes over its row several times, about `most` units to a lane.
// A team of one warp meets without a block barrier, and a row's two ends, which load
// single elements, hold up fewer warps: 16384 x 4099 fp32 takes 76 us to encode with 32
// lanes to a row and 101 with enough lanes to hold it.  With few rows, more lanes each.
uint32_t few_lanes(uint32_t units, int most, uint64_t rows) {
    uint32_t lanes = lanes_for(units, most, kRowThreads);
    while (lanes < kRowThreads && lanes < units && rows * lanes < 152 * 512) lanes *= 2;
    return lanes;
}

template <typename T, bool ALIGNED>
cudaError_t encode(const RowCodesParams &p, cudaStream_t stream) {
    const uint32_t units = (p.dim + 14) / 8;  // at the worst phase
    constexpr int kBlocks = sizeof(T) == 2 ? 4 : 3;
    if (units <= 32) return launch_rows(ragged_encode<T, ALIGNED, 1, true, 6>, p, lanes_for(units, 1, 32), kRowThreads, stream);
    if (units <= 128 || (p.rows < 8 * 304 && units <= 4 * kRowThreads))
        return launch_rows(ragged_encode<T, ALIGNED, 4, true, kBlocks>, p, lanes_for(units, 4, kRowThreads), kRowThreads, stream);
    return launch_rows(ragged_encode<T, ALIGNED, 4, false, kBlocks>, p, std::max(32u, few_lanes(units, 36, p.rows)), kRowThreads, stream);
}

template <typename T>
cudaError_t decode(const RowCodesParams &p, cudaStream_t stream) {
    constexpr uint32_t U = 16 / sizeof(T);
    return launch_rows(ragged_decode<T, 4>, p, lanes_for((p.dim + 2 * U - 2) / U, 4, kRowThreads), kRowThreads, stream);
}

}  // namespace

cudaError_t launch_ragged_copy16(const uint16_t *x, uint64_t stride, uint64_t rows, uint32_t dim, uint16_t *out,
                                 uint64_t out_stride, cudaStream_t stream) {
    const uint32_t lanes = lanes_for((dim + 7) / 8, 4, kRowThreads);
    const uint64_t teams = kRowThreads / lanes;
    const int grid = persistent_grid(reinterpret_cast<const void *>(&ragged_copy16), kRowThreads, (rows + teams - 1) / teams);
    return launch_chained(ragged_copy16, grid, kRowThreads, 0, stream, x, stride, rows, dim, out, out_stride, lanes);
}

cudaError_t launch_ragged_copy8(const int8_t *a, uint64_t rows_a, int8_t *to_a, const int8_t *b, uint64_t rows_b, int8_t *to_b,
                                uint32_t dim, uint64_t out_stride, cudaStream_t stream) {
    const uint32_t lanes = lanes_for((dim + 15) / 16, 4, kRowThreads);
    const uint64_t teams = kRowThreads / lanes;
    const int grid = persistent_grid(reinterpret_cast<const void *>(&ragged_copy8), kRowThreads, (rows_a + rows_b + teams - 1) / teams);
    ragged_copy8<<<grid, kRowThreads, 0, stream>>>(a, rows_a, to_a, b, rows_b, to_b, dim, out_stride, lanes);
    return cudaGetLastError();
}

cudaError_t launch_ragged_encode(const RowCodesParams &p, int bf16, cudaStream_t stream) {
    if (in_step(p.x, p.x_stride, bf16 ? 2 : 4, p.codes, p.dim))
        return bf16 ? encode<uint16_t, true>(p, stream) : encode<float, true>(p, stream);
    return bf16 ? encode<uint16_t, false>(p, stream) : encode<float, false>(p, stream);
}

cudaError_t launch_ragged_decode(const RowCodesParams &p, int bf16, cudaStream_t stream) {
    return bf16 ? decode<uint16_t>(p, stream) : decode<float>(p, stream);
}

cudaError_t launch_ragged_swiglu_encode(const SwigluParams &p, int bf16, cudaStream_t stream) {
    const uint32_t lanes = few_lanes((p.dim + 14) / 8, 9, p.rows);
    const bool aligned = in_step(p.in, p.in_stride, bf16 ? 2 : 4, p.saved_codes, 2 * static_cast<uint64_t>(p.dim));
    const auto kernel = bf16 ? aligned ? ragged_swiglu_encode<uint16_t, true> : ragged_swiglu_encode<uint16_t, false>
                             : aligned ? ragged_swiglu_encode<float, true> : ragged_swiglu_encode<float, false>;
    return launch_rows(kernel, p, lanes, kRowThreads, stream);
}

}  // namespace qc
