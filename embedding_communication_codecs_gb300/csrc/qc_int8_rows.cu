// qc_int8_rows.cu -- row codes of activations and back, and the gated activation
// that keeps its inputs and its result in row codes.
//
// One block owns a row: a pass for the row's largest magnitude, and a pass that
// writes the codes (the second read hits L2).
#include "qc_int8_rows.cuh"
#include "qc_internal.h"

namespace qc {
namespace {

constexpr int kRowThreads = 256;

// Largest of v over the block, in every thread.
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t *red) {
    v = __reduce_max_sync(kFull, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < kRowThreads / 32; ++w) v = max(v, red[w]);
    return v;
}

__device__ __forceinline__ int8_t code_of(float x, const RowScale &s) {
    if (s.inverse == 0.0f) return 0;
    if (s.saturates) x = clamp_to_cap(x);
    return static_cast<int8_t>(code_bits(x, s.inverse) & 0xFFu);
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) rows_encode(const RowCodesParams P) {
    __shared__ uint32_t red[kRowThreads / 32];
    for (uint64_t r = blockIdx.x; r < P.rows; r += gridDim.x) {
        const T *x = static_cast<const T *>(P.x) + r * P.x_stride;
        uint32_t m = 0;
        for (uint32_t j = threadIdx.x; j < P.dim; j += kRowThreads) m = max(m, abs_bits(load_as_float(x + j)));
        const RowScale s = row_scale_of(block_max(m, red));
        for (uint32_t j = threadIdx.x; j < P.dim; j += kRowThreads)
            P.codes[r * P.dim + j] = code_of(load_as_float(x + j), s);
        if (threadIdx.x == 0) P.row_scale[r] = s.scale;
    }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) rows_decode(const RowCodesParams P) {
    for (uint64_t r = blockIdx.x; r < P.rows; r += gridDim.x) {
        const float s = P.scale_in ? P.scale_in[r] : 1.0f;
        T *out = static_cast<T *>(P.out) + r * P.out_stride;
        for (uint32_t j = threadIdx.x; j < P.dim; j += kRowThreads)
            store_from_float(out + j, __fmul_rn(static_cast<float>(P.codes_in[r * P.dim + j]), s));
    }
}

__device__ __forceinline__ float sigmoid(float g) { return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-g))); }

__device__ __forceinline__ float swiglu(float g, float u) {
    return __fmul_rn(__fdiv_rn(g, __fadd_rn(1.0f, expf(-g))), u);
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) swiglu_encode(const SwigluParams P) {
    __shared__ uint32_t red[kRowThreads / 32];
    for (uint64_t r = blockIdx.x; r < P.rows; r += gridDim.x) {
        const T *gate = static_cast<const T *>(P.in) + r * P.in_stride, *up = gate + P.dim;
        uint32_t mg = 0, mu = 0, mh = 0;
        for (uint32_t j = threadIdx.x; j < P.dim; j += kRowThreads) {
            const float g = load_as_float(gate + j), u = load_as_float(up + j);
            mg = max(mg, abs_bits(g));
            mu = max(mu, abs_bits(u));
            mh = max(mh, abs_bits(swiglu(g, u)));
        }
        const RowScale sg = row_scale_of(block_max(mg, red)), su = row_scale_of(block_max(mu, red)),
                       sh = row_scale_of(block_max(mh, red));
        int8_t *saved = P.saved_codes + r * 2 * P.dim;
        for (uint32_t j = threadIdx.x; j < P.dim; j += kRowThreads) {
            const float g = load_as_float(gate + j), u = load_as_float(up + j);
            saved[j] = code_of(g, sg);
            saved[P.dim + j] = code_of(u, su);
            P.h_codes[r * P.dim + j] = code_of(swiglu(g, u), sh);
        }
        if (threadIdx.x == 0) {
            P.saved_scale[2 * r] = sg.scale;
            P.saved_scale[2 * r + 1] = su.scale;
            P.h_scale[r] = sh.scale;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) swiglu_backward(const SwigluParams P) {
    for (uint64_t r = blockIdx.x; r < P.rows; r += gridDim.x) {
        const T *dh = static_cast<const T *>(P.in) + r * P.in_stride;
        const int8_t *saved = P.saved_codes_in + r * 2 * P.dim;
        const float sg = P.saved_scale_in[2 * r], su = P.saved_scale_in[2 * r + 1];
        T *out = static_cast<T *>(P.dgate_up) + r * P.dgate_up_stride;
        for (uint32_t j = threadIdx.x; j < P.dim; j += kRowThreads) {
            const float g = __fmul_rn(static_cast<float>(saved[j]), sg);
            const float u = __fmul_rn(static_cast<float>(saved[P.dim + j]), su);
            const float d = load_as_float(dh + j), sig = sigmoid(g);
            const float slope = __fmul_rn(sig, __fmaf_rn(g, __fsub_rn(1.0f, sig), 1.0f));
            store_from_float(out + j, __fmul_rn(__fmul_rn(d, u), slope));
            store_from_float(out + P.dim + j, __fmul_rn(d, __fmul_rn(g, sig)));
        }
    }
}

template <typename P>
cudaError_t launch_rows(void (*kernel)(const P), const P &p, cudaStream_t stream) {
    const int grid = persistent_grid(reinterpret_cast<const void *>(kernel), kRowThreads, p.rows);
    kernel<<<grid, kRowThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rows_int8_encode(const RowCodesParams &p, int bf16, cudaStream_t stream) {
    return launch_rows(bf16 ? rows_encode<uint16_t> : rows_encode<float>, p, stream);
}

cudaError_t launch_rows_int8_decode(const RowCodesParams &p, int bf16, cudaStream_t stream) {
    return launch_rows(bf16 ? rows_decode<uint16_t> : rows_decode<float>, p, stream);
}

cudaError_t launch_swiglu_encode(const SwigluParams &p, int bf16, cudaStream_t stream) {
    return launch_rows(bf16 ? swiglu_encode<uint16_t> : swiglu_encode<float>, p, stream);
}

cudaError_t launch_swiglu_backward(const SwigluParams &p, int bf16, cudaStream_t stream) {
    return launch_rows(bf16 ? swiglu_backward<uint16_t> : swiglu_backward<float>, p, stream);
}

}  // namespace qc
