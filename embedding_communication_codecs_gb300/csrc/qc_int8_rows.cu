// qc_int8_rows.cu -- row codes of activations and back, and the gated activation
// that keeps its inputs and its result in row codes.
//
// All four kernels move a few bytes per element and compute little: memory
// bandwidth bounds them.  A team of 8 to 512 lanes (a power of two) owns a row and
// covers it in units of U consecutive elements, V units per lane at a time.  The
// encoders read a row once, hold it in registers while the team agrees on the
// largest magnitude, and write the codes from there; a row that is longer than
// the largest team holds is read a second time, from L2.  U is 8 (4 where fp32 is
// written), a lane's 8 to 32 bytes, for rows that start on the vector's boundary; rows that
// start anywhere are qc_int8_ragged.cu's, but for the gated activation's backward pass,
// which takes them here one element at a time.
#include <algorithm>

#include "qc_chain.cuh"
#include "qc_int8_rows.cuh"
#include "qc_internal.h"
#include "qc_pipeline.cuh"

namespace qc {

__device__ unsigned int g_gate_error;
QC_DEFINE_TAKE_FLAG(take_gate_errors, g_gate_error)

namespace {

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
        store_codes(out + u * U, c);
    }
}

// HELD: a team's lanes hold their row (units <= lanes * V); otherwise the second
// pass reads it again.
template <typename T, int U, int V, bool HELD, int BLOCKS>
__global__ void __launch_bounds__(kRowThreads, BLOCKS) rows_encode(const RowCodesParams P, uint32_t lanes) {
    __shared__ uint32_t red[2][32][1];
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

template <typename T, int U, int V>
__global__ void __launch_bounds__(kRowThreads) rows_decode(const RowCodesParams P, uint32_t lanes) {
    let_next_start();
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

// HELD: h is held in registers between the two passes.  Gate and up are read again,
// from L1 or L2: holding them too would leave one block to an SM.
template <typename T, int U, int V, bool HELD, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) swiglu_encode(const SwigluParams P, uint32_t lanes) {
    __shared__ uint32_t red[2][32][3];
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
        float top = 0.0f;  // largest |h|; a NaN stays
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
                        h[v][j] = swiglu<T>(g[v].get(j), w[v].get(j));
                        top = max_magnitude(top, h[v][j]);
                    }
                }
            }
        };
        if constexpr (HELD) {
            products(0);
        } else {
            for (uint32_t base = 0; base < units; base += chunk) products(base);
        }
        m[2] = abs_bits(top);
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
                               [=](uint32_t j) { return swiglu<T>(load_as_float(gate + j), load_as_float(up + j)); });
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

// The same for many rows: groups of rows stream through shared memory (bulk copies, a
// ring of stages), so that loads stay in flight while the block's teams wait for each
// other's maxima and convert.  Both passes read the stage; h stays in registers.
constexpr int kRingThreads = 512, kRingUnits = 4;

struct GateRing {
    uint32_t lanes;       // of a team, which holds a row: units <= lanes * kRingUnits
    uint32_t rows;        // of a stage: one per team
    uint32_t row_bytes, stages;
};

template <typename T>
__global__ void __launch_bounds__(kRingThreads, 1) swiglu_encode_ring(const SwigluParams P, const GateRing G) {
    using R = typename RawOf<T, 8>::type;
    extern __shared__ __align__(16) uint8_t stage_bytes[];
    __shared__ uint32_t red[2][32][3];
    __shared__ uint64_t full[8];
    const uint32_t lanes = G.lanes, lane = threadIdx.x & (lanes - 1), team = threadIdx.x / lanes;
    const uint32_t units = P.dim / 8, stage = G.rows * G.row_bytes;
    const uint64_t groups = (P.rows + G.rows - 1) / G.rows;
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < G.stages; ++i) mbar_init(&full[i], 1);
        fence_barrier_init();
    }
    __syncthreads();
    // iteration i's group into its stage
    auto fetch = [&](uint32_t i) {
        const uint64_t g = blockIdx.x + static_cast<uint64_t>(i) * gridDim.x;
        if (g >= groups) return;
        const uint64_t r0 = g * G.rows;
        const uint32_t n = static_cast<uint32_t>(min(static_cast<uint64_t>(G.rows), P.rows - r0));
        uint64_t *bar = &full[i % G.stages];
        mbar_arrive_expect_tx(bar, n * G.row_bytes);
        for (uint32_t k = 0; k < n; ++k)
            bulk_load(stage_bytes + (i % G.stages) * stage + k * G.row_bytes,
                      static_cast<const T *>(P.in) + (r0 + k) * P.in_stride, G.row_bytes, bar);
    };
    if (threadIdx.x == 0)
        for (uint32_t i = 0; i + 1 < G.stages; ++i) fetch(i);
    int turn = 0;
    bool ok = true;
    uint32_t i = 0;
    for (uint64_t g = blockIdx.x; g < groups; g += gridDim.x, ++i) {
        ok = mbar_wait(&full[i % G.stages], (i / G.stages) & 1);
        // every thread is past its reads of the previous stage, which is filled again
        if (!__syncthreads_and(ok)) {
            ok = false;
            break;
        }
        if (threadIdx.x == 0) {
            fence_proxy_async_shared();
            fetch(i + G.stages - 1);
        }
        const uint64_t r = g * G.rows + team;
        const bool live = r < P.rows;
        const uint8_t *gate = stage_bytes + (i % G.stages) * stage + team * G.row_bytes;
        const uint8_t *up = gate + P.dim * sizeof(T);
        float h[kRingUnits][8], top = 0.0f;
        uint32_t m[3] = {0, 0, 0};
#pragma unroll
        for (int v = 0; v < kRingUnits; ++v) {
            const uint32_t u = v * lanes + lane;
            if (live && u < units) {
                const R a = *reinterpret_cast<const R *>(gate + u * sizeof(R)), b = *reinterpret_cast<const R *>(up + u * sizeof(R));
                m[0] = unit_max(a, m[0]);
                m[1] = unit_max(b, m[1]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    h[v][j] = swiglu<T>(a.get(j), b.get(j));
                    top = max_magnitude(top, h[v][j]);
                }
            }
        }
        m[2] = abs_bits(top);
        team_max(m, lanes, red, turn);
        if (!live) continue;
        const RowScale sg = row_scale_of(m[0]), su = row_scale_of(m[1]), sh = row_scale_of(m[2]);
        int8_t *saved = P.saved_codes + r * 2 * P.dim, *out = P.h_codes + r * P.dim;
        if (lane == 0) {
            P.saved_scale[2 * r] = sg.scale;
            P.saved_scale[2 * r + 1] = su.scale;
            P.h_scale[r] = sh.scale;
        }
        if (sg.inverse == 0.0f || su.inverse == 0.0f || sh.inverse == 0.0f || sg.saturates || su.saturates || sh.saturates) {
            const T *x = static_cast<const T *>(P.in) + r * P.in_stride, *y = x + P.dim;
            encode_rare_row<8>(saved, units, lane, lanes, sg.inverse, [=](uint32_t j) { return load_as_float(x + j); });
            encode_rare_row<8>(saved + P.dim, units, lane, lanes, su.inverse, [=](uint32_t j) { return load_as_float(y + j); });
            encode_rare_row<8>(out, units, lane, lanes, sh.inverse,
                               [=](uint32_t j) { return swiglu<T>(load_as_float(x + j), load_as_float(y + j)); });
            continue;
        }
#pragma unroll
        for (int v = 0; v < kRingUnits; ++v) {
            const uint32_t u = v * lanes + lane;
            if (u < units) {
                const R a = *reinterpret_cast<const R *>(gate + u * sizeof(R)), b = *reinterpret_cast<const R *>(up + u * sizeof(R));
                encode_unit<8>(saved + u * 8, sg.inverse, [&](int j) { return a.get(j); });
                encode_unit<8>(saved + P.dim + u * 8, su.inverse, [&](int j) { return b.get(j); });
                encode_unit<8>(out + u * 8, sh.inverse, [&](int j) { return h[v][j]; });
            }
        }
    }
    if (!ok) {
        // the block stays while a copy is in flight
        if (threadIdx.x == 0) {
            for (uint32_t k = i; k + 1 < i + G.stages; ++k)
                if (blockIdx.x + static_cast<uint64_t>(k) * gridDim.x < groups) mbar_wait(&full[k % G.stages], (k / G.stages) & 1);
            report_failure(&g_gate_error, P.status, kErrPipelineTimeout);
        }
        __syncthreads();
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
                        const float x = d[v].get(j);
                        const Sigma sig = sigma_of<T>(g);
                        const float slope = __fmul_rn(sig.s, __fmaf_rn(g, sig.other, 1.0f));
                        dg[j] = __fmul_rn(__fmul_rn(x, u), slope);
                        du[j] = __fmul_rn(x, __fmul_rn(g, sig.s));
                    }
                    store_values<T, U>(out + at, dg);
                    store_values<T, U>(out + P.dim + at, du);
                }
        }
    }
}

// Rows of the buffer start on a boundary of `bytes` and units of u elements fill them.
bool fits(const void *p, uint64_t stride, size_t esize, uint32_t dim, uint32_t u, size_t bytes) {
    return dim % u == 0 && reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * esize % bytes == 0;
}

template <typename T>
cudaError_t encode_rows(const RowCodesParams &p, cudaStream_t stream) {
    constexpr bool kWide = sizeof(T) == 4;  // fp32 units take twice the registers
    const uint32_t d = p.dim;
    if (!fits(p.x, p.x_stride, sizeof(T), d, 8, 16) || !fits(p.codes, d, 1, d, 8, 8))
        return launch_ragged_encode(p, sizeof(T) == 2, stream);
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
    return launch_ragged_decode(p, sizeof(T) == 2, stream);
}

template <typename T>
cudaError_t encode_swiglu(const SwigluParams &p, cudaStream_t stream) {
    const uint32_t d = p.dim;
    // the ups start dim elements into a row: dim % 8 == 0 aligns them as the gates
    if (!fits(p.in, p.in_stride, sizeof(T), d, 8, 16) || !fits(p.h_codes, d, 1, d, 8, 8) ||
        !fits(p.saved_codes, 2 * d, 1, d, 8, 8))
        return launch_ragged_swiglu_encode(p, sizeof(T) == 2, stream);
    const uint32_t units = d / 8;
    // Streaming pays where every SM has several groups of rows and a ring holds at least
    // two of them (8192 x 16384: 163 us against 226 for blocks that load their own rows).
    GateRing ring{};
    ring.lanes = lanes_for(units, kRingUnits, kRingThreads);
    ring.rows = kRingThreads / ring.lanes;
    ring.row_bytes = 2 * d * sizeof(T);
    const uint32_t stage = ring.rows * ring.row_bytes;
    ring.stages = std::min(6u, 200u * 1024u / stage);
    const uint64_t groups = (p.rows + ring.rows - 1) / ring.rows;
    if (units <= kRingUnits * ring.lanes && ring.stages >= 2 && groups >= 3 * 152) {
        const auto kernel = swiglu_encode_ring<T>;
        const size_t smem = static_cast<size_t>(ring.stages) * stage;
        const cudaError_t e = prepare_dynamic_smem(reinterpret_cast<const void *>(kernel), 200 * 1024);
        if (e != cudaSuccess) return e;
        const int grid = persistent_grid(reinterpret_cast<const void *>(kernel), kRingThreads, groups, smem);
        kernel<<<grid, kRingThreads, smem, stream>>>(p, ring);
        return cudaGetLastError();
    }
    // 64 registers a thread (fp32: 80) leave room for 32 warps (24) on an SM
    constexpr bool kWide = sizeof(T) == 4;
    if (units <= 512)
        return launch_rows(swiglu_encode<T, 8, 2, true, 256, kWide ? 3 : 4>, p, lanes_for(units, 2, 256), 256, stream);
    if (units <= 1024) return launch_rows(swiglu_encode<T, 8, 2, true, 512, kWide ? 1 : 2>, p, 512, 512, stream);
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
