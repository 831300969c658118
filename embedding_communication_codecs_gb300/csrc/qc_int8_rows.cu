// qc_int8_rows.cu -- row codes of activations and back, and the gated activation
// that keeps its inputs and its result in row codes.
//
// All four kernels move a few bytes per element and compute little: memory
// bandwidth bounds them.  A team of 8 to 512 lanes (a power of two) owns a row and
// covers it in units of U consecutive elements, V units per lane at a time.  The
// encoders read a row once, hold it in registers while the team agrees on the
// largest magnitude, and write the codes from there; a row that is longer than
// the largest team holds is read a second time, from L2.  U is 8 (or 16) where
// rows start on the vector's boundary, so that a lane moves 8 to 32 bytes with one
// instruction, and 1 elsewhere.
#include "qc_int8_rows.cuh"
#include "qc_internal.h"

namespace qc {
namespace {

constexpr int kRowThreads = 256;

// U consecutive elements of a row, as they lie in memory.
template <int U>
struct alignas(U * 4 > 16 ? 16 : U * 4) RawF32 {
    float v[U];
    __device__ __forceinline__ float get(int j) const { return v[j]; }
};
template <int U>
struct alignas(U * 2 > 16 ? 16 : U * 2) RawBf16 {
    uint16_t v[U];
    __device__ __forceinline__ float get(int j) const { return bf16_bits_to_float(v[j]); }
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
    if constexpr (U == 1) {
        return max(m, (static_cast<uint32_t>(r.v[0]) & 0x7FFFu) << 16);
    } else {
        uint32_t p = 0;
#pragma unroll
        for (int j = 0; j < U; j += 2) {
            const uint32_t w = static_cast<uint32_t>(r.v[j]) | static_cast<uint32_t>(r.v[j + 1]) << 16;
            p = __vmaxu2(p, w & 0x7FFF7FFFu);
        }
        return max(m, max(p & 0xFFFF0000u, p << 16));
    }
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

// The codes of U elements, four to a word.
template <int U>
__device__ __forceinline__ void store_codes(int8_t *p, const uint32_t (&c)[U]) {
    if constexpr (U == 1) {
        *p = static_cast<int8_t>(c[0] & 0xFFu);
    } else {
        static_assert(U == 8, "a unit is 8 bytes of codes");
        *reinterpret_cast<uint2 *>(p) =
            make_uint2(pack_codes(c[0], c[1], c[2], c[3]), pack_codes(c[4], c[5], c[6], c[7]));
    }
}

// U fp32 values rounded to the output's type.
template <typename T, int U>
__device__ __forceinline__ void store_values(T *p, const float (&v)[U]) {
    typename RawOf<T, U>::type r;
#pragma unroll
    for (int j = 0; j < U; ++j) store_from_float(&r.v[j], v[j]);
    *reinterpret_cast<typename RawOf<T, U>::type *>(p) = r;
}

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
__device__ __forceinline__ void team_max(uint32_t (&v)[N], uint32_t lanes, uint32_t (*red)[16][N], int &turn) {
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
    store_codes<U>(out, c);
}

// The rare rows: all codes 0 (it may hold infinities and NaN, which are not
// multiplied), or values to clamp.  Read again, a unit at a time, to keep their
// code and registers out of the fast path.
template <int U, typename Get>
__device__ __noinline__ void encode_rare_row(int8_t *out, uint32_t units, uint32_t lane, uint32_t lanes, float inverse,
                                             Get get) {
#pragma unroll 1
    for (uint32_t u = lane; u < units; u += lanes) {
        uint32_t c[U];
#pragma unroll
        for (int j = 0; j < U; ++j) c[j] = inverse == 0.0f ? 0u : code_bits(clamp_to_cap(get(u * U + j)), inverse);
        store_codes<U>(out + u * U, c);
    }
}

// HELD: a team's lanes hold their row (units <= lanes * V); otherwise the second
// pass reads it again.
template <typename T, int U, int V, bool HELD, int BLOCKS>
__global__ void __launch_bounds__(kRowThreads, BLOCKS) rows_encode(const RowCodesParams P, uint32_t lanes) {
    __shared__ uint32_t red[2][16][1];
    using R = typename RawOf<T, U>::type;
    const Team team(lanes);
    const uint32_t units = P.dim / U, chunk = lanes * V;
    int turn = 0;
    // every team of the block goes round as often as the block's first one
    for (uint64_t r0 = team.first - threadIdx.x / lanes; r0 < P.rows; r0 += team.stride) {
        const uint64_t r = r0 + threadIdx.x / lanes;
        const bool live = r < P.rows;
        const T *x = static_cast<const T *>(P.x) + (live ? r : 0) * P.x_stride;
        R held[V];
        uint32_t m[1] = {0};
        auto load = [&](uint32_t base) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t u = base + v * lanes + team.lane;
                if (u < units) held[v] = load_unit<T, U>(x + u * U);
            }
        };
        auto largest = [&](uint32_t base) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (base + v * lanes + team.lane < units) m[0] = unit_max(held[v], m[0]);
        };
        if constexpr (HELD) {
            load(0);
            largest(0);
        } else {
            for (uint32_t base = 0; base < units; base += chunk) {
                load(base);
                largest(base);
            }
        }
        team_max(m, lanes, red, turn);
        const RowScale s = row_scale_of(m[0]);
        if (!live) continue;
        int8_t *out = P.codes + r * P.dim;
        auto encode = [&](uint32_t base) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t u = base + v * lanes + team.lane;
                if (u < units) encode_unit<U>(out + u * U, s.inverse, [&](int j) { return held[v].get(j); });
            }
        };
        if (team.lane == 0) P.row_scale[r] = s.scale;
        if (s.inverse == 0.0f || s.saturates) {
            encode_rare_row<U>(out, units, team.lane, lanes, s.inverse, [=](uint32_t j) { return load_as_float(x + j); });
        } else if constexpr (HELD) {
            encode(0);
        } else {
            for (uint32_t base = 0; base < units; base += chunk) {
                load(base);
                encode(base);
            }
        }
    }
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

template <typename T, int U, int V>
__global__ void __launch_bounds__(kRowThreads) rows_decode(const RowCodesParams P, uint32_t lanes) {
    const Team team(lanes);
    const uint32_t units = P.dim / U;
    for (uint64_t row = team.first; row < P.rows; row += team.stride) {
        const bool second = row >= P.first_rows;
        const uint64_t r = second ? row - P.first_rows : row;
        const float *scale = second ? P.scale_in2 : P.scale_in;
        const float s = scale ? __ldg(scale + r) : 1.0f;
        const int8_t *codes = (second ? P.codes_in2 : P.codes_in) + r * P.dim;
        T *out = static_cast<T *>(second ? P.out2 : P.out) + r * P.out_stride;
        for (uint32_t base = team.lane; base < units; base += lanes * V) {
            RawCodes<U> c[V];
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (base + v * lanes < units)
                    c[v] = *reinterpret_cast<const RawCodes<U> *>(codes + static_cast<uint64_t>(base + v * lanes) * U);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (base + v * lanes < units) {
                    float f[U];
#pragma unroll
                    for (int j = 0; j < U; ++j) f[j] = __fmul_rn(c[v].get(j), s);
                    store_values<T, U>(out + static_cast<uint64_t>(base + v * lanes) * U, f);
                }
        }
    }
}

// 1 / (1 + exp(-g)) by the hardware's exponential (base 2) and reciprocal: their
// errors and the argument's rounding (|g| half units) stay below 2^-19 relative for
// |g| < 16, an eighth of a per cent of half a code's step.  Saturates to 1 and 0.
__device__ __forceinline__ float sigmoid(float g) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(g, -1.4426950408889634f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.0f, e)));
    return r;
}

__device__ __forceinline__ float swiglu(float g, float u) { return __fmul_rn(__fmul_rn(g, sigmoid(g)), u); }

// HELD: h is held in registers between the two passes.  Gate and up are read again,
// from L1 or L2: holding them too would leave one block to an SM.
template <typename T, int U, int V, bool HELD, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) swiglu_encode(const SwigluParams P, uint32_t lanes) {
    __shared__ uint32_t red[2][16][3];
    using R = typename RawOf<T, U>::type;
    const Team team(lanes);
    const uint32_t units = P.dim / U, chunk = lanes * V;
    int turn = 0;
    for (uint64_t r0 = team.first - threadIdx.x / lanes; r0 < P.rows; r0 += team.stride) {
        const uint64_t r = r0 + threadIdx.x / lanes;
        const bool live = r < P.rows;
        const T *gate = static_cast<const T *>(P.in) + (live ? r : 0) * P.in_stride, *up = gate + P.dim;
        float h[V][U];
        uint32_t m[3] = {0, 0, 0};
        auto products = [&](uint32_t base) {
            R g[V], w[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t u = base + v * lanes + team.lane;
                if (u < units) {
                    g[v] = load_unit<T, U>(gate + u * U);
                    w[v] = load_unit<T, U>(up + u * U);
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (base + v * lanes + team.lane < units) {
                    m[0] = unit_max(g[v], m[0]);
                    m[1] = unit_max(w[v], m[1]);
#pragma unroll
                    for (int j = 0; j < U; ++j) {
                        h[v][j] = swiglu(g[v].get(j), w[v].get(j));
                        m[2] = max(m[2], abs_bits(h[v][j]));
                    }
                }
            }
        };
        if constexpr (HELD) {
            products(0);
        } else {
            for (uint32_t base = 0; base < units; base += chunk) products(base);
        }
        team_max(m, lanes, red, turn);
        const RowScale sg = row_scale_of(m[0]), su = row_scale_of(m[1]), sh = row_scale_of(m[2]);
        if (!live) continue;
        int8_t *saved = P.saved_codes + r * 2 * P.dim, *out = P.h_codes + r * P.dim;
        if (team.lane == 0) {
            P.saved_scale[2 * r] = sg.scale;
            P.saved_scale[2 * r + 1] = su.scale;
            P.h_scale[r] = sh.scale;
        }
        auto encode = [&](uint32_t base) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t u = base + v * lanes + team.lane;
                if (u < units) {
                    const R g = load_unit<T, U>(gate + u * U), w = load_unit<T, U>(up + u * U);
                    encode_unit<U>(saved + u * U, sg.inverse, [&](int j) { return g.get(j); });
                    encode_unit<U>(saved + P.dim + u * U, su.inverse, [&](int j) { return w.get(j); });
                    encode_unit<U>(out + u * U, sh.inverse, [&](int j) { return h[v][j]; });
                }
            }
        };
        if (sg.inverse == 0.0f || su.inverse == 0.0f || sh.inverse == 0.0f || sg.saturates || su.saturates || sh.saturates) {
            encode_rare_row<U>(saved, units, team.lane, lanes, sg.inverse, [=](uint32_t j) { return load_as_float(gate + j); });
            encode_rare_row<U>(saved + P.dim, units, team.lane, lanes, su.inverse, [=](uint32_t j) { return load_as_float(up + j); });
            encode_rare_row<U>(out, units, team.lane, lanes, sh.inverse,
                               [=](uint32_t j) { return swiglu(load_as_float(gate + j), load_as_float(up + j)); });
        } else if constexpr (HELD) {
            encode(0);
        } else {
            for (uint32_t base = 0; base < units; base += chunk) {
                products(base);
                encode(base);
            }
        }
    }
}

template <typename T, int U, int V>
__global__ void __launch_bounds__(kRowThreads) swiglu_backward(const SwigluParams P, uint32_t lanes) {
    using R = typename RawOf<T, U>::type;
    const Team team(lanes);
    const uint32_t units = P.dim / U;
    for (uint64_t r = team.first; r < P.rows; r += team.stride) {
        const T *dh = static_cast<const T *>(P.in) + r * P.in_stride;
        const int8_t *saved = P.saved_codes_in + r * 2 * P.dim;
        const float sg = __ldg(P.saved_scale_in + 2 * r), su = __ldg(P.saved_scale_in + 2 * r + 1);
        T *out = static_cast<T *>(P.dgate_up) + r * P.dgate_up_stride;
        for (uint32_t base = team.lane; base < units; base += lanes * V) {
            R d[V];
            RawCodes<U> cg[V], cu[V];
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (base + v * lanes < units) {
                    const uint64_t at = static_cast<uint64_t>(base + v * lanes) * U;
                    d[v] = load_unit<T, U>(dh + at);
                    cg[v] = *reinterpret_cast<const RawCodes<U> *>(saved + at);
                    cu[v] = *reinterpret_cast<const RawCodes<U> *>(saved + P.dim + at);
                }
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (base + v * lanes < units) {
                    const uint64_t at = static_cast<uint64_t>(base + v * lanes) * U;
                    float dg[U], du[U];
#pragma unroll
                    for (int j = 0; j < U; ++j) {
                        const float g = __fmul_rn(cg[v].get(j), sg);
                        const float u = __fmul_rn(cu[v].get(j), su);
                        const float x = d[v].get(j), sig = sigmoid(g);
                        const float slope = __fmul_rn(sig, __fmaf_rn(g, __fsub_rn(1.0f, sig), 1.0f));
                        dg[j] = __fmul_rn(__fmul_rn(x, u), slope);
                        du[j] = __fmul_rn(x, __fmul_rn(g, sig));
                    }
                    store_values<T, U>(out + at, dg);
                    store_values<T, U>(out + P.dim + at, du);
                }
        }
    }
}

// Lanes of a team that covers `units` with up to V units per lane: 8 to `most`.
uint32_t lanes_for(uint32_t units, int v, uint32_t most) {
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

// Rows of the buffer start on a boundary of `bytes` and units of u elements fill them.
bool fits(const void *p, uint64_t stride, size_t esize, uint32_t dim, uint32_t u, size_t bytes) {
    return dim % u == 0 && reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * esize % bytes == 0;
}

template <typename T>
cudaError_t encode_rows(const RowCodesParams &p, cudaStream_t stream) {
    constexpr bool kWide = sizeof(T) == 4;  // fp32 units take twice the registers
    const uint32_t d = p.dim;
    if (!fits(p.x, p.x_stride, sizeof(T), d, 8, 16) || !fits(p.codes, d, 1, d, 8, 8)) {
        if (d <= 8 * kRowThreads) return launch_rows(rows_encode<T, 1, 8, true, 6>, p, lanes_for(d, 8, kRowThreads), kRowThreads, stream);
        if (d <= 32 * kRowThreads) return launch_rows(rows_encode<T, 1, 32, true, 3>, p, kRowThreads, kRowThreads, stream);
        return launch_rows(rows_encode<T, 1, 8, false, 6>, p, kRowThreads, kRowThreads, stream);
    }
    const uint32_t units = d / 8;
    if (units <= 32) return launch_rows(rows_encode<T, 8, 1, true, 8>, p, lanes_for(units, 1, 32), kRowThreads, stream);
    if (units <= 4 * kRowThreads)
        return launch_rows(rows_encode<T, 8, 4, true, kWide ? 4 : 6>, p, lanes_for(units, 4, kRowThreads), kRowThreads, stream);
    if (units <= 8 * kRowThreads) return launch_rows(rows_encode<T, 8, 8, true, kWide ? 2 : 3>, p, kRowThreads, kRowThreads, stream);
    return launch_rows(rows_encode<T, 8, 4, false, 4>, p, kRowThreads, kRowThreads, stream);
}

// A lane's store is one 16-byte piece, so that a warp's store covers whole sectors
// (two pieces per lane measured 4.7 TB/s against 5.9 for 16384 x 8192).
template <typename T>
cudaError_t decode_rows(const RowCodesParams &p, cudaStream_t stream) {
    constexpr int U = 16 / sizeof(T);
    const uint32_t d = p.dim;
    if (fits(p.out, p.out_stride, sizeof(T), d, U, 16) && fits(p.codes_in, d, 1, d, U, U) &&
        (p.rows == p.first_rows || (fits(p.out2, p.out_stride, sizeof(T), d, U, 16) && fits(p.codes_in2, d, 1, d, U, U))))
        return launch_rows(rows_decode<T, U, 8>, p, lanes_for(d / U, 8, kRowThreads), kRowThreads, stream);
    return launch_rows(rows_decode<T, 1, 8>, p, lanes_for(d, 8, kRowThreads), kRowThreads, stream);
}

template <typename T>
cudaError_t encode_swiglu(const SwigluParams &p, cudaStream_t stream) {
    const uint32_t d = p.dim;
    // the ups start dim elements into a row: dim % 8 == 0 aligns them as the gates
    if (!fits(p.in, p.in_stride, sizeof(T), d, 8, 16) || !fits(p.h_codes, d, 1, d, 8, 8) ||
        !fits(p.saved_codes, 2 * d, 1, d, 8, 8))
        return d <= 8 * 512 ? launch_rows(swiglu_encode<T, 1, 8, true, 512, 2>, p, lanes_for(d, 8, 512), 512, stream)
                            : launch_rows(swiglu_encode<T, 1, 4, false, 512, 2>, p, 512, 512, stream);
    const uint32_t units = d / 8;
    // blocks to an SM as the registers allow without spills
    constexpr bool kWide = sizeof(T) == 4;
    if (units <= 512)
        return launch_rows(swiglu_encode<T, 8, 2, true, 256, kWide ? 3 : 4>, p, lanes_for(units, 2, 256), 256, stream);
    if (units <= 2048)
        return launch_rows(swiglu_encode<T, 8, 4, true, 512, 1>, p, lanes_for(units, 4, 512), 512, stream);
    return launch_rows(swiglu_encode<T, 8, 1, false, 256, 3>, p, 256, 256, stream);
}

template <typename T>
cudaError_t backward_swiglu(const SwigluParams &p, cudaStream_t stream) {
    const uint32_t d = p.dim;
    if (fits(p.in, p.in_stride, sizeof(T), d, 8, 16) && fits(p.dgate_up, p.dgate_up_stride, sizeof(T), d, 8, 16) &&
        fits(p.saved_codes_in, 2 * d, 1, d, 8, 8))
        return launch_rows(swiglu_backward<T, 8, 2>, p, lanes_for(d / 8, 2, kRowThreads), kRowThreads, stream);
    return launch_rows(swiglu_backward<T, 1, 4>, p, lanes_for(d, 4, kRowThreads), kRowThreads, stream);
}

}  // namespace

cudaError_t launch_rows_int8_encode(const RowCodesParams &p, int bf16, cudaStream_t stream) {
    return bf16 ? encode_rows<uint16_t>(p, stream) : encode_rows<float>(p, stream);
}

cudaError_t launch_rows_int8_decode(const RowCodesParams &p, int bf16, cudaStream_t stream) {
    return bf16 ? decode_rows<uint16_t>(p, stream) : decode_rows<float>(p, stream);
}

cudaError_t launch_swiglu_encode(const SwigluParams &p, int bf16, cudaStream_t stream) {
    return bf16 ? encode_swiglu<uint16_t>(p, stream) : encode_swiglu<float>(p, stream);
}

cudaError_t launch_swiglu_backward(const SwigluParams &p, int bf16, cudaStream_t stream) {
    return bf16 ? backward_swiglu<uint16_t>(p, stream) : backward_swiglu<float>(p, stream);
}

}  // namespace qc
