// qc_int8_wide.cu -- the product of the 8-bit layer for a batch of tokens, the weights
// read from memory once and as codes.
//
// For tens to hundreds of tokens the weights' N K bytes are what has to be read, and
// widening them in memory first would move five times that.  The product is turned
// round, y^T = W X^T: the weights are the tensor core's A operand, which may come
// from tensor memory, so a widened weight never passes through shared memory again:
//
//     TMA -> codes in shared memory -> registers -> f16 in tensor memory -> tcgen05.mma
//
// (f16 holds every int8 exactly.)  The tokens are B, widened to f16 once by a small
// launch (T K elements) and loaded by TMA.  A pair of blocks owns 256 weight rows x BT
// tokens and a range of the contraction; per step of 128 codes each block loads 16 KB
// of codes and half of the tokens' 256 BT bytes.  Warp 0 loads, warp 1 of the leading
// block issues the matrix instructions, warps 4 to 11 widen (two groups of four warps
// take alternate steps; a warp reaches 32 lanes of tensor memory), warps 12 to 15
// store.  Tensor memory: two sums of BT columns, and four stages of 64 columns of
// widened codes.  The lanes of a storing warp hold neighbouring outputs of one
// token, so its stores are whole lines wherever y's rows start.
#include <cuda.h>

#include "qc_int8_rows.cuh"
#include "qc_internal.h"
#include "qc_tc.cuh"
#include "qc_tc_host.h"

namespace qc {

__device__ unsigned int g_wide_error;
QC_DEFINE_TAKE_FLAG(take_wide_errors, g_wide_error)

namespace {

constexpr int kStepK = 128;
constexpr int kRows = 128, kPairRows = 256;
constexpr int kThreads = 512;
constexpr int kAStages = 4, kACols = kStepK / 2;
constexpr int kTmemCols = 512, kATmem = 256;  // sums from column 0, widened codes from column 256

template <int BT>
struct Wide {
    static constexpr int kBytesW = kRows * kStepK;
    static constexpr int kBytesX = BT / 2 * kStepK * 2;  // two boxes of BT / 2 rows of 128 bytes
    static constexpr int kStage = kBytesW + kBytesX;
    static constexpr int kStages = BT == 128 ? 6 : BT == 64 ? 8 : 9;
    static constexpr int kSmem = kStages * kStage + 1024;
};

struct WideParams {
    uint64_t T, N, K;
    uint32_t splits, split_steps;
    float *partial;
    void *y;
    uint64_t y_stride;
    int y_bf16;
    const float *x_scale, *w_scale, *bias;
    uint32_t *status;
};

struct WideUnit {
    uint32_t n, t, split, first, steps;
};

// Units in order: the token tiles of a weight tile next to each other.
template <int BT>
__device__ __forceinline__ WideUnit wide_unit(uint32_t u, const WideParams &P) {
    const uint32_t tiles_t = static_cast<uint32_t>((P.T + BT - 1) / BT);
    const uint32_t tiles_n = static_cast<uint32_t>((P.N + kPairRows - 1) / kPairRows);
    const uint32_t all = static_cast<uint32_t>((P.K + kStepK - 1) / kStepK);
    const uint32_t split = u / (tiles_t * tiles_n), first = split * P.split_steps;
    return {u / tiles_t % tiles_n, u % tiles_t, split, first, min(P.split_steps, all - first)};
}

// Four codes -> two f16 pairs (each byte, offset by 128, under the exponent of 2^10,
// minus 1024 + 128).
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    w ^= 0x80808080u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(w, 0x64646464u, 0x4140)), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(w, 0x64646464u, 0x4342)), "r"(0x64806480u));
}

template <int BT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    wide_tokens(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const WideParams P) {
    using C = Wide<BT>;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full_w[S], full_x[S], empty[S], a_full[kAStages], a_empty[kAStages], sums_full[2], sums_empty[2], drained;
    __shared__ uint32_t tmem_slot;
    uint8_t *const tiles = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), npairs = gridDim.x / 2, pair = blockIdx.x / 2;
    const uint32_t units = static_cast<uint32_t>((P.T + BT - 1) / BT) * static_cast<uint32_t>((P.N + kPairRows - 1) / kPairRows) * P.splits;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full_w[s], 1);   // this block's codes
            mbar_init(&full_x[s], 1);   // both blocks' tokens, in the leading block
            mbar_init(&empty[s], 5);    // the four warps that widened it, and the instructions that read the tokens
        }
        for (int a = 0; a < kAStages; ++a) {
            mbar_init(&a_full[a], 8);   // four widening warps in each block, in the leading block
            mbar_init(&a_empty[a], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sums_full[b], 1);
            mbar_init(&sums_empty[b], 8);
        }
        mbar_init(&drained, 1);
        fence_barrier_init();
        prefetch_map(&map_w);
        prefetch_map(&map_x);
    }
    if (warp == 1) tmem_alloc_pair<kTmemCols>(&tmem_slot);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            for (uint32_t u = pair; u < units && ok; u += npairs) {
                const WideUnit w = wide_unit<BT>(u, P);
                const int n0 = static_cast<int>(w.n * kPairRows + rank * kRows), t0 = static_cast<int>(w.t * BT + rank * (BT / 2));
                for (uint32_t k = 0; k < w.steps; ++k, ++it) {
                    const uint32_t s = it % S;
                    if (!mbar_wait_cluster(&empty[s], ((it / S) & 1) ^ 1)) {
                        ok = false;
                        break;
                    }
                    uint8_t *codes = tiles + s * C::kStage, *x = codes + C::kBytesW;
                    const int k0 = static_cast<int>((w.first + k) * kStepK);
                    mbar_arrive_expect_tx(&full_w[s], C::kBytesW);
                    tma_load(codes, &map_w, k0, n0, &full_w[s]);
                    const uint32_t bar = in_block(&full_x[s], 0);
                    if (rank == 0) mbar_arrive_expect_tx(&full_x[s], 2 * C::kBytesX);
                    tma_load_pair(x, &map_x, k0, t0, bar);
                    tma_load_pair(x + C::kBytesX / 2, &map_x, k0 + 64, t0, bar);
                }
            }
            // no block leaves while a copy into either one is in flight
            for (uint32_t i = it > S ? it - S : 0; i < it; ++i) {
                ok &= mbar_wait_cluster(&full_w[i % S], (i / S) & 1);
                if (rank == 0) ok &= mbar_wait_cluster(&full_x[i % S], (i / S) & 1);
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && lane == 0) {
            constexpr uint32_t kInstr = f16_instruction(kPairRows, BT);
            uint32_t it = 0, done = 0;
            for (uint32_t u = pair; u < units && ok; u += npairs, ++done) {
                const uint32_t steps = wide_unit<BT>(u, P).steps, buf = done & 1;
                if (!mbar_wait_cluster(&sums_empty[buf], ((done >> 1) & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                for (uint32_t k = 0; k < steps; ++k, ++it) {
                    const uint32_t s = it % S, a = it % kAStages;
                    if (!mbar_wait_cluster(&full_x[s], (it / S) & 1) || !mbar_wait_cluster(&a_full[a], (it / kAStages) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint8_t *x = tiles + s * C::kStage + C::kBytesW;
                    const uint64_t b0 = smem_operand(x, 0), b1 = smem_operand(x + C::kBytesX / 2, 0);
#pragma unroll
                    for (int j = 0; j < kStepK / 16; ++j)
                        mma_pair_tmem(tmem + buf * BT, tmem + kATmem + a * kACols + 8 * j, (j < 4 ? b0 : b1) + (j & 3) * 2, kInstr,
                                      k > 0 || j > 0);
                    mma_commit_pair(&empty[s]);
                    mma_commit_pair(&a_empty[a]);
                }
                mma_commit_pair(&sums_full[buf]);
            }
            mma_commit_pair(&drained);
        }
        // neither block leaves before the leading block's last instruction and the
        // arrivals that it sent to both blocks
        if (lane == 0) ok &= mbar_wait_cluster(&drained, 0);
    } else if (warp >= 4 && warp < 12) {
        const uint32_t group = (warp - 4) >> 2;
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t to = tmem + kATmem + (static_cast<uint32_t>(quarter * 32) << 16);
        uint32_t it = 0;
        for (uint32_t u = pair; u < units && ok; u += npairs) {
            const uint32_t steps = wide_unit<BT>(u, P).steps;
            for (uint32_t k = 0; k < steps; ++k, ++it) {
                if ((it & 1) != group) continue;
                const uint32_t s = it % S, a = it % kAStages;
                ok = mbar_wait_cluster(&full_w[s], (it / S) & 1) && mbar_wait_cluster(&a_empty[a], ((it / kAStages) & 1) ^ 1);
                if (__any_sync(kFull, !ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint8_t *codes = tiles + s * C::kStage + row * 128;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t f[32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 c = *reinterpret_cast<const uint4 *>(codes + (((4 * h + i) ^ (row & 7)) << 4));
                        widen4(c.x, f[8 * i], f[8 * i + 1]);
                        widen4(c.y, f[8 * i + 2], f[8 * i + 3]);
                        widen4(c.z, f[8 * i + 4], f[8 * i + 5]);
                        widen4(c.w, f[8 * i + 6], f[8 * i + 7]);
                    }
                    tmem_store32(to + a * kACols + 32 * h, f);
                }
                tmem_wait_store();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&empty[s]);
                    mbar_arrive_cluster(in_block(&a_full[a], 0));
                }
            }
        }
    } else if (warp >= 12) {
        const int quarter = warp & 3;
        uint32_t done = 0;
        for (uint32_t u = pair; u < units; u += npairs, ++done) {
            const uint32_t buf = done & 1;
            ok = mbar_wait_cluster(&sums_full[buf], (done >> 1) & 1);
            if (__any_sync(kFull, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const WideUnit w = wide_unit<BT>(u, P);
            const uint64_t n = static_cast<uint64_t>(w.n) * kPairRows + rank * kRows + quarter * 32 + lane;
            const uint64_t t0 = static_cast<uint64_t>(w.t) * BT;
            const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * BT;
            const bool live = n < P.N;
            const float ws = live ? __ldg(P.w_scale + n) : 0.0f, bias = live && P.bias ? __ldg(P.bias + n) : 0.0f;
            const uint64_t rows = (P.T + 31) / 32 * 32, pitch = (P.N + 31) / 32 * 32;
#pragma unroll 1
            for (int c = 0; c < BT && t0 + c < P.T; c += 8) {
                uint32_t v[8];
                tmem_load8(from + c, v);
                tmem_wait_load();
                if (live) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint64_t t = t0 + c + j;
                        if (t >= P.T) break;
                        float r = __uint_as_float(v[j]);
                        if (P.splits > 1) {
                            P.partial[(w.split * rows + t) * pitch + n] = r;
                            continue;
                        }
                        r = __fmul_rn(r, __fmul_rn(__ldg(P.x_scale + t), ws));
                        if (P.bias) r = __fadd_rn(r, bias);
                        if (P.y_bf16)
                            static_cast<uint16_t *>(P.y)[t * P.y_stride + n] = to_bf16(r);
                        else
                            static_cast<float *>(P.y)[t * P.y_stride + n] = r;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(in_block(&sums_empty[buf], 0));
        }
    }
    if (!ok) report_failure(&g_wide_error, P.status, kErrPipelineTimeout);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) tmem_free_pair<kTmemCols>(tmem);
}

// Codes of a row -> f16, eight at a time where rows start on 8 bytes.
template <int U>
__global__ void __launch_bounds__(256) widen_tokens(const int8_t *codes, uint64_t T, uint64_t K, uint16_t *out, uint64_t pitch) {
    const uint64_t per_row = K / U, total = T * per_row;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<uint64_t>(gridDim.x) * 256) {
        const uint64_t t = i / per_row, k = i % per_row * U;
        if constexpr (U == 8) {
            const uint2 c = __ldg(reinterpret_cast<const uint2 *>(codes + t * K + k));
            uint4 f;
            widen4(c.x, f.x, f.y);
            widen4(c.y, f.z, f.w);
            *reinterpret_cast<uint4 *>(out + t * pitch + k) = f;
        } else {
            uint32_t lo, hi;
            widen4(static_cast<uint8_t>(codes[t * K + k]), lo, hi);
            out[t * pitch + k] = static_cast<uint16_t>(lo & 0xFFFFu);
        }
    }
}

struct WidePlan {
    int bt;
    uint32_t splits, split_steps;
};

// Token tiles of 32, 64 or 128, and the contraction cut so that about 76 pairs have
// work: a step takes a pair about 700 cycles at its share of the memory's rate, or
// the tensor core's 4 BT; a unit starts and stores in about 3000; a join is a launch
// and its sums written and read.
WidePlan wide_plan(uint64_t T, uint64_t N, uint64_t K) {
    constexpr uint64_t kPairs = 76;
    const int bt = T <= 32 ? 32 : T <= 64 ? 64 : 128;
    const uint64_t steps = (K + kStepK - 1) / kStepK;
    const uint64_t tiles = ((T + bt - 1) / bt) * ((N + kPairRows - 1) / kPairRows);
    WidePlan best{bt, 1, static_cast<uint32_t>(steps)};
    double best_cost = 1e300;
    for (uint64_t s = 1; s <= 16 && (s == 1 || steps / s >= 2); ++s) {
        const uint64_t per = (steps + s - 1) / s, splits = (steps + per - 1) / per;
        const uint64_t waves = (tiles * splits + kPairs - 1) / kPairs;
        double cost = static_cast<double>(waves) * (static_cast<double>(per) * 700 + 3000);
        if (splits > 1) cost += 5000 + static_cast<double>(splits) * T * N * 8 / 5000;
        if (cost < best_cost) {
            best_cost = cost;
            best = {bt, static_cast<uint32_t>(splits), static_cast<uint32_t>(per)};
        }
    }
    return best;
}

uint64_t pitch_of(uint64_t K) { return (K + 63) / 64 * 64; }
uint64_t tokens_bytes(uint64_t T, uint64_t K) { return (T * pitch_of(K) * 2 + 255) / 256 * 256; }

bool map_rows(CUtensorMap *map, CUtensorMapDataType type, const void *p, uint64_t rows, uint64_t dim, uint64_t stride_bytes,
              uint32_t box_dim, uint32_t box_rows) {
    const cuuint64_t dims[2] = {dim, rows}, strides[1] = {stride_bytes};
    const cuuint32_t box[2] = {box_dim, box_rows}, unit[2] = {1, 1};
    EncodeTiled fn = encode_tiled();
    return fn && fn(map, type, 2, const_cast<void *>(p), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BT>
cudaError_t launch_wide(const ProductParams &p, const uint16_t *x, const WideParams &w, cudaStream_t stream) {
    using C = Wide<BT>;
    const auto kernel = wide_tokens<BT>;
    CUtensorMap mw, mx;
    if (!map_rows(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.w_codes, p.N, p.K, p.K, kStepK, kRows) ||
        !map_rows(&mx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x, p.T, p.K, pitch_of(p.K) * 2, 64, BT / 2))
        return cudaErrorInvalidValue;
    const cudaError_t e = prepare_dynamic_smem(reinterpret_cast<const void *>(kernel), C::kSmem);
    if (e != cudaSuccess) return e;
    const uint64_t units = ((p.T + BT - 1) / BT) * ((p.N + kPairRows - 1) / kPairRows) * w.splits;
    const uint64_t most = sm_count() / 2;
    kernel<<<static_cast<unsigned>(2 * (units < most ? units : most)), kThreads, C::kSmem, stream>>>(mw, mx, w);
    return cudaGetLastError();
}

}  // namespace

bool wide_tokens_fit(const void *w_codes, uint64_t K) {
    return K % 16 == 0 && (reinterpret_cast<uintptr_t>(w_codes) & 15) == 0;
}

size_t wide_tokens_workspace(uint64_t T, uint64_t N, uint64_t K) {
    const WidePlan plan = wide_plan(T, N, K);
    return tokens_bytes(T, K) + (plan.splits > 1 ? plan.splits * ceil32(T) * ceil32(N) * 4 : 0);
}

cudaError_t launch_int8_wide(const ProductParams &p, cudaStream_t stream) {
    const WidePlan plan = wide_plan(p.T, p.N, p.K);
    uint16_t *x = static_cast<uint16_t *>(p.workspace);
    const bool eights = p.K % 8 == 0 && (reinterpret_cast<uintptr_t>(p.x_codes) & 7) == 0;
    const auto widen = eights ? widen_tokens<8> : widen_tokens<1>;
    const uint64_t work = p.T * (eights ? p.K / 8 : p.K);
    widen<<<persistent_grid(reinterpret_cast<const void *>(widen), 256, (work + 255) / 256), 256, 0, stream>>>(p.x_codes, p.T, p.K, x,
                                                                                                         pitch_of(p.K));
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    WideParams w{};
    w.T = p.T;
    w.N = p.N;
    w.K = p.K;
    w.splits = plan.splits;
    w.split_steps = plan.split_steps;
    w.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(p.workspace) + tokens_bytes(p.T, p.K));
    w.y = p.out;
    w.y_stride = p.out_stride;
    w.y_bf16 = p.out_bf16;
    w.x_scale = p.x_scale;
    w.w_scale = p.w_scale;
    w.bias = p.bias;
    w.status = p.status;
    e = plan.bt == 32 ? launch_wide<32>(p, x, w, stream) : plan.bt == 64 ? launch_wide<64>(p, x, w, stream)
                                                                         : launch_wide<128>(p, x, w, stream);
    if (e != cudaSuccess || w.splits == 1) return e;
    return launch_join({w.partial, w.splits, p.T, p.N, p.out, p.out_stride, p.out_bf16, 0, p.x_scale, p.w_scale, p.bias}, stream);
}

}  // namespace qc
