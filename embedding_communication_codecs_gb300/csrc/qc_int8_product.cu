// qc_int8_product.cu -- the products of the 8-bit linear layer.
//
// out[m, n] = sum over l of A(m, l) * B(l, n), both operands read as fp32 through
// a functor and summed in order of l by one thread per output, in 64 x 64 tiles.
#include "qc_int8_rows.cuh"
#include "qc_internal.h"

namespace qc {
namespace {

constexpr int kTile = 64, kDepth = 16, kThreads = 256;

struct Shape {
    uint64_t M, N, L;
};

// A and B: float operator()(outer index, l).  Out: void operator()(m, n, sum).
template <typename A, typename B, typename Out>
__global__ void __launch_bounds__(kThreads) product(const Shape S, const A a, const B b, const Out out) {
    __shared__ float sa[kDepth][kTile + 1], sb[kDepth][kTile + 1];
    const uint64_t ntn = (S.N + kTile - 1) / kTile;
    const uint64_t m0 = blockIdx.x / ntn * kTile, n0 = blockIdx.x % ntn * kTile;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float acc[4][4] = {};
    for (uint64_t l0 = 0; l0 < S.L; l0 += kDepth) {
        for (int i = threadIdx.x; i < kTile * kDepth; i += kThreads) {
            const int r = i / kDepth, l = i % kDepth;
            const bool in = l0 + l < S.L;
            sa[l][r] = in && m0 + r < S.M ? a(m0 + r, l0 + l) : 0.0f;
            sb[l][r] = in && n0 + r < S.N ? b(n0 + r, l0 + l) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int l = 0; l < kDepth; ++l)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __fmaf_rn(sa[l][ty + 16 * i], sb[l][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < S.M && n < S.N) out(m, n, acc[i][j]);
        }
}

struct CodeRows {  // (row, l) of dense codes
    const int8_t *codes;
    uint64_t dim;
    __device__ float operator()(uint64_t r, uint64_t l) const { return codes[r * dim + l]; }
};

struct DecodedColumns {  // (column, l) of decoded codes, rounded to bf16; l is the row
    const int8_t *codes;
    const float *scale;
    uint64_t dim;
    __device__ float operator()(uint64_t c, uint64_t l) const {
        return bf16_bits_to_float(to_bf16(__fmul_rn(codes[l * dim + c], scale[l])));
    }
};

struct Bf16Rows {
    const uint16_t *x;
    uint64_t stride;
    __device__ float operator()(uint64_t r, uint64_t l) const { return bf16_bits_to_float(x[r * stride + l]); }
};

struct Bf16Columns {
    const uint16_t *x;
    uint64_t stride;
    __device__ float operator()(uint64_t c, uint64_t l) const { return bf16_bits_to_float(x[l * stride + c]); }
};

struct StoreOut {
    void *out;
    uint64_t stride;
    int bf16, accumulate;
    const float *m_scale, *n_scale, *bias;
    __device__ void operator()(uint64_t m, uint64_t n, float v) const {
        if (m_scale) v = __fmul_rn(v, __fmul_rn(m_scale[m], n_scale[n]));
        if (bias) v = __fadd_rn(v, bias[n]);
        if (bf16) {
            static_cast<uint16_t *>(out)[m * stride + n] = to_bf16(v);
        } else {
            float *o = static_cast<float *>(out) + m * stride + n;
            *o = accumulate ? __fadd_rn(*o, v) : v;
        }
    }
};

__global__ void column_sums(const uint16_t *x, uint64_t stride, uint64_t rows, uint64_t cols, float *out,
                            int accumulate) {
    const uint64_t c = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (c >= cols) return;
    DWord s{0.0f, 0.0f};
    for (uint64_t r = 0; r < rows; ++r) s = dw_add(s, bf16_bits_to_float(x[r * stride + c]));
    const float v = __fadd_rn(s.hi, s.lo);
    out[c] = accumulate ? __fadd_rn(out[c], v) : v;
}

template <typename A, typename B>
cudaError_t launch(const Shape &s, const A &a, const B &b, const StoreOut &o, cudaStream_t stream) {
    const uint64_t tiles = ((s.M + kTile - 1) / kTile) * ((s.N + kTile - 1) / kTile);
    if (tiles > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
    product<<<static_cast<unsigned>(tiles), kThreads, 0, stream>>>(s, a, b, o);
    return cudaGetLastError();
}

}  // namespace

size_t int8_matmul_workspace(uint64_t, uint64_t, uint64_t) { return 0; }
size_t int8_input_grad_workspace(uint64_t, uint64_t, uint64_t) { return 0; }
size_t int8_weight_grad_workspace(uint64_t, uint64_t, uint64_t) { return 0; }

cudaError_t launch_int8_matmul(const ProductParams &p, cudaStream_t stream) {
    return launch({p.T, p.N, p.K}, CodeRows{p.x_codes, p.K}, CodeRows{p.w_codes, p.K},
                  StoreOut{p.out, p.out_stride, p.out_bf16, 0, p.x_scale, p.w_scale, p.bias}, stream);
}

cudaError_t launch_int8_input_grad(const ProductParams &p, cudaStream_t stream) {
    return launch({p.T, p.K, p.N}, Bf16Rows{p.dy, p.dy_stride}, DecodedColumns{p.w_codes, p.w_scale, p.K},
                  StoreOut{p.out, p.out_stride, p.out_bf16, 0, nullptr, nullptr, nullptr}, stream);
}

cudaError_t launch_int8_weight_grad(const ProductParams &p, cudaStream_t stream) {
    cudaError_t e = launch({p.N, p.K, p.T}, Bf16Columns{p.dy, p.dy_stride},
                           DecodedColumns{p.x_codes, p.x_scale, p.K},
                           StoreOut{p.out, p.out_stride, p.out_bf16, p.accumulate, nullptr, nullptr, nullptr},
                           stream);
    if (e != cudaSuccess || !p.dbias) return e;
    column_sums<<<static_cast<unsigned>((p.N + 127) / 128), 128, 0, stream>>>(p.dy, p.dy_stride, p.T, p.N,
                                                                              p.dbias, p.accumulate);
    return cudaGetLastError();
}

}  // namespace qc
