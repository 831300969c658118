// qc_int8_few.cu -- the product of the 8-bit layer for few tokens (one new token per
// request).
//
// The weights' N K bytes are read once and bound it.  A block owns 16 outputs for
// 8 NT tokens; its eight warps take 64-element chunks of the contraction in turn.
// A lane loads 16 consecutive codes of a weight row (eight rows of 64 bytes per
// instruction) and the same 16 of a token, and widens both to f16 in registers
// (exactly: |code| <= 128) as fragments of m16n8k16 matrix instructions.  The order
// of the contraction inside a fragment is free, as long as both operands use the
// same one, so the codes need no shuffle: bytes 4j .. 4j+3 of a lane are its share
// of the j-th instruction.  The warps' sums meet in shared memory and are added in
// order.  (mma.sync runs at 300 T multiply-adds/s here for f16 and 75 for int8,
// measured: at 16 tokens the weights' stream already needs 107.)
#include "qc_int8_rows.cuh"
#include "qc_internal.h"

namespace qc {
namespace {

constexpr int kFewWarps = 8;
constexpr int kChunk = 64;
// The matrix instruction's running sum drops what is below its last place; a warp's sum
// is cut into parts of 32 chunks = 2048 terms, added in fp32.
constexpr int kPartChunks = 32;

struct FewParams {
    const int8_t *x, *w;
    const float *x_scale, *w_scale, *bias;
    uint64_t T, N, K;
    void *y;
    uint64_t y_stride;
    int y_bf16;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The aligned word at `p`, of which only the bytes inside [begin, end) are read.
__device__ __forceinline__ uint32_t word_inside(const uint8_t *p, const uint8_t *begin, const uint8_t *end) {
    if (p >= begin && p + 4 <= end) return __ldg(reinterpret_cast<const uint32_t *>(p));
    uint32_t v = 0;
    for (int i = 0; i < 4; ++i)
        if (p + i >= begin && p + i < end) v |= static_cast<uint32_t>(__ldg(p + i)) << (8 * i);
    return v;
}

// The vectors around 16 codes that start anywhere, and the codes out of them.
struct Around {
    uint4 lo, hi;
    uint32_t off;  // of the first code in lo, in bytes
};
template <bool ALIGNED>
struct PieceOf {
    using type = uint4;
};
template <>
struct PieceOf<false> {
    using type = Around;
};

// 16 codes from element k of a row on, as loaded; beyond the rows or K, zeros.  Past K
// inside a piece lie other codes, which multiply the tokens' zeros (below).  ALIGNED:
// every row starts on 16 bytes and K is a multiple of 16.
template <bool ALIGNED>
__device__ __forceinline__ typename PieceOf<ALIGNED>::type load16(const int8_t *base, uint64_t row, uint64_t k, uint64_t rows,
                                                                  uint64_t K) {
    const int8_t *p = base + row * K + k;
    const bool in = row < rows && k < K;
    if constexpr (ALIGNED) {
        return in ? __ldg(reinterpret_cast<const uint4 *>(p)) : make_uint4(0u, 0u, 0u, 0u);
    } else {
        Around a{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u), 0u};
        if (!in) return a;
        const uint8_t *begin = reinterpret_cast<const uint8_t *>(base), *end = begin + rows * K;
        const uint8_t *v = reinterpret_cast<const uint8_t *>(reinterpret_cast<uintptr_t>(p) & ~static_cast<uintptr_t>(15));
        a.off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
        if (v >= begin && v + 32 <= end) {
            a.lo = __ldg(reinterpret_cast<const uint4 *>(v));
            a.hi = __ldg(reinterpret_cast<const uint4 *>(v) + 1);
        } else {
            a.lo = make_uint4(word_inside(v, begin, end), word_inside(v + 4, begin, end), word_inside(v + 8, begin, end),
                              word_inside(v + 12, begin, end));
            a.hi = make_uint4(word_inside(v + 16, begin, end), word_inside(v + 20, begin, end), word_inside(v + 24, begin, end),
                              word_inside(v + 28, begin, end));
        }
        return a;
    }
}

__device__ __forceinline__ uint4 codes_of(const uint4 &v) { return v; }
__device__ __forceinline__ uint4 codes_of(const Around &a) {
    uint32_t w[8] = {a.lo.x, a.lo.y, a.lo.z, a.lo.w, a.hi.x, a.hi.y, a.hi.z, a.hi.w};
    const bool two = (a.off & 8) != 0, one = (a.off & 4) != 0;
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = two ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = one ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (a.off & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The codes of a token's piece, zeros from K on.
template <bool ALIGNED>
__device__ __forceinline__ uint4 token_codes(const typename PieceOf<ALIGNED>::type &piece, uint64_t k, uint64_t K) {
    uint4 c = codes_of(piece);
    if constexpr (!ALIGNED) {
        if (k < K && K - k < 16) {
            const int left = static_cast<int>(K - k);
            auto keep = [&](uint32_t v, int i) {
                return left <= 4 * i ? 0u : left >= 4 * i + 4 ? v : v & (0xFFFFFFFFu >> (32 - 8 * (left - 4 * i)));
            };
            c = make_uint4(keep(c.x, 0), keep(c.y, 1), keep(c.z, 2), keep(c.w, 3));
        }
    }
    return c;
}

__device__ __forceinline__ uint32_t word_of(const uint4 &v, int j) {
    return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

// AHEAD chunks of a warp are loaded before the first of them is multiplied.
template <int NT, int AHEAD, int BLOCKS, bool ALIGNED>
__global__ void __launch_bounds__(32 * kFewWarps, BLOCKS) few_tokens(const FewParams P) {
    extern __shared__ float sums[];  // [warp][token][output], outputs padded by one
    constexpr int kOut = 16, kTok = 8 * NT, kPitch = kOut + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const uint64_t n0 = static_cast<uint64_t>(blockIdx.x) * kOut, t0 = static_cast<uint64_t>(blockIdx.y) * kTok;
    static_assert(kPartChunks % AHEAD == 0, "parts are whole rounds of loads");
    constexpr uint32_t step = kFewWarps * kChunk;
    const uint32_t K = static_cast<uint32_t>(P.K);
    float *mine = sums + warp * kTok * kPitch;
    for (uint32_t part = 0; part < K; part += kPartChunks * step) {
        float acc[NT][4] = {};
        const uint32_t end = min(K, part + kPartChunks * step);
        for (uint32_t k0 = part + warp * kChunk; k0 < end; k0 += AHEAD * step) {
            typename PieceOf<ALIGNED>::type w[AHEAD][2], x[AHEAD][NT];
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                const uint64_t k = k0 + a * step + 16 * q;
                w[a][0] = load16<ALIGNED>(P.w, n0 + g, k, P.N, P.K);
                w[a][1] = load16<ALIGNED>(P.w, n0 + g + 8, k, P.N, P.K);
#pragma unroll
                for (int j = 0; j < NT; ++j) x[a][j] = load16<ALIGNED>(P.x, t0 + 8 * j + g, k, P.T, P.K);
            }
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                const uint4 w0 = codes_of(w[a][0]), w1 = codes_of(w[a][1]);
                uint4 xc[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) xc[j] = token_codes<ALIGNED>(x[a][j], k0 + a * step + 16 * q, P.K);
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    uint32_t l0, h0, l1, h1;
                    widen4(word_of(w0, f), l0, h0);
                    widen4(word_of(w1, f), l1, h1);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        uint32_t xl, xh;
                        widen4(word_of(xc[j], f), xl, xh);
                        mma_f16(acc[j], l0, l1, h0, h1, xl, xh);
                    }
                }
            }
        }
        // acc[j]: outputs g and g + 8, tokens 8 j + 2 q and + 1
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float &sum = mine[(8 * j + 2 * q + (c & 1)) * kPitch + g + 8 * (c >> 1)];
                sum = part == 0 ? acc[j][c] : __fadd_rn(sum, acc[j][c]);
            }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kTok * kOut; i += 32 * kFewWarps) {
        const uint64_t t = t0 + i / kOut, n = n0 + i % kOut;
        if (t >= P.T || n >= P.N) continue;
        const float xs = __ldg(P.x_scale + t), ws = __ldg(P.w_scale + n), bias = P.bias ? __ldg(P.bias + n) : 0.0f;
        float v = 0.0f;
#pragma unroll
        for (int s = 0; s < kFewWarps; ++s) v = __fadd_rn(v, sums[(s * kTok + i / kOut) * kPitch + i % kOut]);
        v = far_scale(xs) || far_scale(ws) ? scaled_far(v, xs, ws) : __fmul_rn(v, __fmul_rn(xs, ws));
        if (P.bias) v = __fadd_rn(v, bias);
        if (P.y_bf16)
            static_cast<uint16_t *>(P.y)[t * P.y_stride + n] = to_bf16(v);
        else
            static_cast<float *>(P.y)[t * P.y_stride + n] = v;
    }
}

template <int NT, int AHEAD, int BLOCKS, bool ALIGNED>
cudaError_t launch(const FewParams &p, cudaStream_t stream) {
    constexpr size_t smem = sizeof(float) * kFewWarps * 8 * NT * 17;
    const dim3 grid(static_cast<unsigned>((p.N + 15) / 16), static_cast<unsigned>((p.T + 8 * NT - 1) / (8 * NT)));
    few_tokens<NT, AHEAD, BLOCKS, ALIGNED><<<grid, 32 * kFewWarps, smem, stream>>>(p);
    return cudaGetLastError();
}

// Up to 8 tokens: where every block is resident at once with two to an SM, each
// loads its whole share ahead (4096 x 4096: 5.5 us, against 6.2 for four blocks with
// half of it ahead); with more blocks, more of them to an SM hide each other's ends
// (16384 x 4096: 14.3 us against 16.1).
cudaError_t launch_aligned(const FewParams &p, cudaStream_t stream) {
    if (p.T <= 8) return p.N <= 16 * 304 ? launch<1, 8, 2, true>(p, stream) : launch<1, 4, 4, true>(p, stream);
    return launch<2, 4, 3, true>(p, stream);
}

// Pieces that start anywhere hold twice the registers until they are shifted.
cudaError_t launch_anywhere(const FewParams &p, cudaStream_t stream) {
    return p.T <= 8 ? launch<1, 4, 2, false>(p, stream) : launch<2, 2, 2, false>(p, stream);
}

}  // namespace

cudaError_t launch_int8_few(const ProductParams &p, cudaStream_t stream) {
    const FewParams f{p.x_codes, p.w_codes, p.x_scale, p.w_scale, p.bias, p.T,
                      p.N,       p.K,       p.out,     p.out_stride, p.out_bf16};
    const bool aligned = p.K % 16 == 0 && ((reinterpret_cast<uintptr_t>(p.x_codes) | reinterpret_cast<uintptr_t>(p.w_codes)) & 15) == 0;
    return aligned ? launch_aligned(f, stream) : launch_anywhere(f, stream);
}

}  // namespace qc
