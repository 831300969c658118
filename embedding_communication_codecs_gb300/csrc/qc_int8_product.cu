// qc_int8_product.cu -- the products of the 8-bit linear layer on the tensor cores.
//
// sm_103a has no 8-bit integer matrix instruction, so the codes are widened to bf16
// (exactly: |code| <= 128 times a power of two) and every product is
//
//     out[m, n] = sum over l of A(m, l) B(n, l),   bf16 x bf16 -> fp32,
//
// with each operand either K-major (rows of the outer index) or MN-major (rows of
// the contraction index), as it lies in memory:
//
//     matmul       A = x codes [T, K]   K-major    B = w codes [N, K]   K-major
//     input grad   A = dy      [T, N]   K-major    B = w values [N, K]  MN-major
//     weight grad  A = dy      [T, N]   MN-major   B = x values [T, K]  MN-major
//
// A pair of blocks (a cluster of two) owns a 256 x BN tile: each holds 128 rows of A
// and BN / 2 rows of B per step of 64 along l, and 128 x BN sums in its tensor
// memory, twice, so that one is read while the next is summed.  Warp 0 loads (TMA),
// warp 1 of the leading block issues the matrix instructions, warps 2 to 9 add the
// parts of a sum and store.  Every wait is bounded (qc_pipeline.cuh).
#include <cuda.h>

#include <algorithm>

#include "qc_chain.cuh"
#include "qc_int8_rows.cuh"
#include "qc_internal.h"
#include "qc_tc.cuh"
#include "qc_tc_host.h"

namespace qc {

__device__ unsigned int g_product_error;
QC_DEFINE_TAKE_FLAG(take_product_errors, g_product_error)

namespace {

constexpr int kStep = 64;       // contraction elements per stage: one 128-byte row
constexpr int kBlockM = 128;    // rows of A per block
constexpr int kPairM = 2 * kBlockM;
constexpr int kStoreWarps = 8;
constexpr int kGemmThreads = 32 * (2 + kStoreWarps);
constexpr int kTmemCols = 512;  // all of tensor memory, so it starts at column 0
constexpr int kGroupM = 8;      // tiles along M that share their B tiles in L2
// The tensor core's running sum loses up to a unit in the last place per
// instruction, always towards zero, so its error grows with the length of the sum
// (1.1e-6 of the result after 8192 terms, measured).  A sum is cut into parts of
// 32 steps = 2048 terms, which the storing warps add in fp32, rounding to nearest.
constexpr uint32_t kPartSteps = 32;

template <int BN>
struct Tile {
    static constexpr int kRowsB = BN / 2;
    static constexpr int kBytesA = kBlockM * kStep * 2, kBytesB = kRowsB * kStep * 2;
    static constexpr int kStage = kBytesA + kBytesB;
    static constexpr int kStages = BN == 256 ? 6 : 8;
    static constexpr int kWarpCols = BN / 2;               // columns of a storing warp
    static constexpr int kSmem = kStages * kStage + kStoreWarps * 4096 + 1024;  // tiles start on 1024 bytes
};

struct GemmParams {
    uint64_t M, N, L;
    uint32_t splits, split_steps;  // the contraction in `splits` ranges of split_steps steps
    float *partial;                // where splits > 1: splits x ceil32(M) rows of partial_pitch sums
    uint64_t partial_pitch;
    void *out;
    uint64_t out_stride;
    int out_bf16, accumulate;
    const float *m_scale, *n_scale, *bias;
    uint32_t *status;
};

// A pair's unit of work: one tile, one range of the contraction.
struct Unit {
    uint32_t m, n, split, first_step, steps;
};

// Units in order: all tiles of the first range, then of the next.  Tiles in groups
// of kGroupM tile rows, column by column inside a group.
__device__ __forceinline__ Unit unit_at(uint32_t u, uint32_t tiles_m, uint32_t tiles_n, const GemmParams &P) {
    const uint32_t ntiles = tiles_m * tiles_n, split = u / ntiles, t = u % ntiles;
    const uint32_t per_group = kGroupM * tiles_n;
    const uint32_t g = t / per_group, r = t % per_group;
    const uint32_t rows = min(tiles_m - g * kGroupM, static_cast<uint32_t>(kGroupM));
    const uint32_t all = static_cast<uint32_t>((P.L + kStep - 1) / kStep), first = split * P.split_steps;
    return {g * kGroupM + r % rows, r / rows, split, first, min(P.split_steps, all - first)};
}

// Adds a storing warp's C columns of tensor memory to its registers.
template <int C>
__device__ __forceinline__ void add_sums(uint32_t at, float (&acc)[C]) {
#pragma unroll
    for (int c = 0; c < C; c += 8) {
        uint32_t v[8];
        tmem_load8(at + c, v);
        tmem_wait_load();
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[c + j] = __fadd_rn(acc[c + j], __uint_as_float(v[j]));
    }
}

// How a kernel writes its results.
enum Output : int {
    kSums,       // fp32 sums of a split contraction, by TMA
    kF32,        // fp32 results, by TMA
    kF32Add,     // added to what is there, by TMA
    kBf16,       // bf16 results, by TMA
    kAnywhere    // rows that TMA cannot write (not on 16-byte boundaries), element by element
};

// Byte offset of 16-byte piece `i` of row `r` in a warp's 32 rows of 128 bytes, as the
// 128-byte swizzle lays them out; pieces i of 8 neighbouring rows share no bank.
__device__ __forceinline__ uint32_t swizzled(int r, int i) { return r * 128 + ((i ^ (r & 7)) << 4); }

// A scale or bias, loaded where it stands: hoisted above the stores, these loads'
// registers would push sums into local memory.
__device__ __forceinline__ float load_here(const float *p) {
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

// Four sums of columns n .. n + 3 scaled and biased (the columns past the last are
// not stored; their scales are read from the last one).
__device__ __forceinline__ float4 finish4(const GemmParams &P, float ms, uint32_t n, const float *v) {
    float r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t c = min(n + j, static_cast<uint32_t>(P.N) - 1);
        r[j] = v[j];
        if (P.m_scale) r[j] = __fmul_rn(r[j], __fmul_rn(ms, load_here(P.n_scale + c)));
        if (P.bias) r[j] = __fadd_rn(r[j], load_here(P.bias + c));
    }
    return make_float4(r[0], r[1], r[2], r[3]);
}

// Whether any scale of a warp's 32 rows and C columns is far (only the forward product, whose
// operands are both K-major, has scales here).
template <int C>
__device__ __forceinline__ bool far_scales(const GemmParams &P, uint32_t m0, uint32_t n, int lane) {
    bool far = far_scale(load_here(P.m_scale + min(m0 + lane, static_cast<uint32_t>(P.M) - 1)));
#pragma unroll
    for (int c = 0; c < C; c += 32) far |= far_scale(load_here(P.n_scale + min(n + c + lane, static_cast<uint32_t>(P.N) - 1)));
    return __any_sync(kFull, far);
}

// A storing warp's C columns from n on of the 32 rows from m0 on (lane l holds row
// m0 + l): scaled, biased, written to the warp's 4 KB of shared memory as 32 rows of
// 128 bytes and stored from there by TMA.
template <int C, Output OUT>
__device__ __forceinline__ void store_tma(const GemmParams &P, const CUtensorMap &map, uint32_t split, uint32_t m0,
                                          uint32_t n, int lane, uint8_t *buf, const float (&acc)[C]) {
    constexpr int kCols = OUT == kBf16 ? 64 : 32;
    const float ms = OUT != kSums && P.m_scale ? __ldg(P.m_scale + (m0 + lane < P.M ? m0 + lane : P.M - 1)) : 1.0f;
    const int y = static_cast<int>(OUT == kSums ? split * ((static_cast<uint32_t>(P.M) + 31) / 32 * 32) + m0 : m0);
#pragma unroll
    for (int c = 0; c < C; c += kCols) {
        if (n + c >= P.N) break;
        if (lane == 0) tma_store_wait_read();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint4 w;
            if constexpr (OUT == kBf16) {
                const float4 lo = finish4(P, ms, n + c + 8 * i, acc + c + 8 * i), hi = finish4(P, ms, n + c + 8 * i + 4, acc + c + 8 * i + 4);
                w = make_uint4(pack_bf16(lo.x, lo.y), pack_bf16(lo.z, lo.w), pack_bf16(hi.x, hi.y), pack_bf16(hi.z, hi.w));
            } else {
                float4 v = make_float4(acc[c + 4 * i], acc[c + 4 * i + 1], acc[c + 4 * i + 2], acc[c + 4 * i + 3]);
                if constexpr (OUT != kSums) v = finish4(P, ms, n + c + 4 * i, acc + c + 4 * i);
                w = make_uint4(__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w));
            }
            *reinterpret_cast<uint4 *>(buf + swizzled(lane, i)) = w;
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
            tma_store<OUT == kF32Add>(&map, static_cast<int>(n + c), y, buf);
            tma_store_commit();
        }
    }
}

// The same, element by element: 32 x 32 sums through the warp's shared memory, so
// that its lanes store neighbouring columns of one row.  Far scales are only multiplied
// here: in store_tma() a test for each sum cost 8192 x 16384 x 4096 800 us instead of 580.
template <int C>
__device__ __forceinline__ void store_anywhere(const GemmParams &P, uint32_t m0, uint32_t n, int lane, uint8_t *buf,
                                               const float (&acc)[C], bool far) {
    if (lane == 0) tma_store_wait_read();  // of an earlier tile, whose scales were not far
    const int rows = P.M - m0 < 32 ? static_cast<int>(P.M - m0) : 32;
#pragma unroll
    for (int c = 0; c < C; c += 32) {
        if (n + c >= P.N) break;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4 *>(buf + swizzled(lane, i)) =
                make_float4(acc[c + 4 * i], acc[c + 4 * i + 1], acc[c + 4 * i + 2], acc[c + 4 * i + 3]);
        __syncwarp();
        const uint32_t col = n + c + lane;
        if (col < P.N) {
            const float ns = P.m_scale ? __ldg(P.n_scale + col) : 1.0f, bias = P.bias ? __ldg(P.bias + col) : 0.0f;
            const auto sum_at = [&](int r) {
                return *reinterpret_cast<const float *>(buf + swizzled(r, lane >> 2) + 4 * (lane & 3));
            };
            const auto store = [&](int r, float v) {
                if (P.bias) v = __fadd_rn(v, bias);
                const uint64_t at = static_cast<uint64_t>(m0 + r) * P.out_stride + col;
                if (P.out_bf16) {
                    static_cast<uint16_t *>(P.out)[at] = to_bf16(v);
                } else {
                    float *o = static_cast<float *>(P.out) + at;
                    *o = P.accumulate ? __fadd_rn(*o, v) : v;
                }
            };
            if (far) {
#pragma unroll 1
                for (int r = 0; r < rows; ++r) store(r, scaled_far_call(sum_at(r), __ldg(P.m_scale + m0 + r), ns));
            } else {
#pragma unroll 4
                for (int r = 0; r < rows; ++r) {
                    const float v = sum_at(r);
                    store(r, P.m_scale ? __fmul_rn(v, __fmul_rn(__ldg(P.m_scale + m0 + r), ns)) : v);
                }
            }
        }
    }
}

template <int BN, bool A_MN, bool B_MN, Output OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    gemm(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
         const __grid_constant__ CUtensorMap map_out, const GemmParams P) {
    using T = Tile<BN>;
    constexpr int S = T::kStages;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[S], empty[S], sums_full[2], sums_empty[2], drained;
    __shared__ uint32_t tmem_slot;
    uint8_t *const tiles = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t tiles_m = static_cast<uint32_t>((P.M + kPairM - 1) / kPairM);
    const uint32_t tiles_n = static_cast<uint32_t>((P.N + BN - 1) / BN);
    const uint32_t units = tiles_m * tiles_n * P.splits, npairs = gridDim.x / 2, pair = blockIdx.x / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);     // the leading block's load thread; bytes of both blocks
            mbar_init(&empty[s], 1);    // the matrix instructions that read the stage
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sums_full[b], 1);
            mbar_init(&sums_empty[b], 2 * kStoreWarps);  // the storing warps of both blocks
        }
        mbar_init(&drained, 1);
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc_pair<kTmemCols>(&tmem_slot);
    if (threadIdx.x == 0) {
        prefetch_map(&map_a);
        prefetch_map(&map_b);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    after_previous();
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            for (uint32_t u = pair; u < units && ok; u += npairs) {
                const Unit w = unit_at(u, tiles_m, tiles_n, P);
                const int m0 = static_cast<int>(w.m * kPairM + rank * kBlockM);
                const int n0 = static_cast<int>(w.n * BN + rank * T::kRowsB);
                for (uint32_t k = 0; k < w.steps; ++k, ++it) {
                    const uint32_t s = it % S, phase = (it / S) & 1;
                    if (!mbar_wait_cluster(&empty[s], phase ^ 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = in_block(&full[s], 0);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * T::kStage);
                    uint8_t *a = tiles + s * T::kStage, *b = a + T::kBytesA;
                    const int l0 = static_cast<int>((w.first_step + k) * kStep);
                    if (A_MN) {
                        tma_load_pair(a, &map_a, m0, l0, bar);
                        tma_load_pair(a + T::kBytesA / 2, &map_a, m0 + 64, l0, bar);
                    } else {
                        tma_load_pair(a, &map_a, l0, m0, bar);
                    }
                    if (B_MN) {
#pragma unroll
                        for (int j = 0; j < T::kRowsB / 64; ++j)
                            tma_load_pair(b + j * 64 * kStep * 2, &map_b, n0 + 64 * j, l0, bar);
                    } else {
                        tma_load_pair(b, &map_b, l0, n0, bar);
                    }
                }
            }
            // no block leaves while a copy into either one is in flight
            if (rank == 0)
                for (uint32_t i = it > S ? it - S : 0; i < it; ++i) ok &= mbar_wait_cluster(&full[i % S], (i / S) & 1);
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // the whole warp goes round, one lane issues
            constexpr uint32_t kInstr = bf16_instruction(kPairM, BN, A_MN, B_MN);
            // 16 contraction elements on: 32 bytes inside a row, or 16 rows of 128 bytes
            constexpr uint32_t kNextA = (A_MN ? 2048 : 32) >> 4, kNextB = (B_MN ? 2048 : 32) >> 4;
            const bool issues = one_lane();
            uint32_t it = 0, part = 0;  // parts so far: the two sums in tensor memory are used in turn
            for (uint32_t u = pair; u < units && ok; u += npairs) {
                const uint32_t steps = unit_at(u, tiles_m, tiles_n, P).steps;
                for (uint32_t k0 = 0; k0 < steps && ok; k0 += kPartSteps, ++part) {
                    const uint32_t buf = part & 1, k1 = min(k0 + kPartSteps, steps);
                    ok = __all_sync(kFull, mbar_wait_cluster(&sums_empty[buf], ((part >> 1) & 1) ^ 1));
                    if (!ok) break;
                    tc_fence_after();
                    for (uint32_t k = k0; k < k1; ++k, ++it) {
                        const uint32_t s = it % S;
                        ok = __all_sync(kFull, mbar_wait_cluster(&full[s], (it / S) & 1));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t a = smem_operand(tiles + s * T::kStage, 64 * kStep * 2);
                        const uint64_t b = smem_operand(tiles + s * T::kStage + T::kBytesA, 64 * kStep * 2);
                        if (issues) {
#pragma unroll
                            for (int j = 0; j < kStep / 16; ++j)
                                mma_pair(buf * BN, a + j * kNextA, b + j * kNextB, kInstr, k > k0 || j > 0);
                            mma_commit_pair(&empty[s]);
                        }
                        __syncwarp();
                    }
                    if (issues) mma_commit_pair(&sums_full[buf]);
                    __syncwarp();
                }
            }
            if (issues) mma_commit_pair(&drained);
            __syncwarp();
        }
        // neither block leaves before the leading block's last instruction and the
        // arrivals that it sent to both blocks
        if (lane == 0) ok &= mbar_wait_cluster(&drained, 0);
    } else {
        const int quarter = warp & 3;                         // the 32 lanes of tensor memory that this warp may read
        const uint32_t c0 = (warp - 2) / 4 * T::kWarpCols;    // its half of the columns
        const uint32_t from = (static_cast<uint32_t>(quarter * 32) << 16) + c0;
        uint8_t *const buf = tiles + S * T::kStage + (warp - 2) * 4096;
        uint32_t part = 0;
        for (uint32_t u = pair; u < units && ok; u += npairs) {
            float acc[T::kWarpCols] = {};
            const uint32_t parts = (unit_at(u, tiles_m, tiles_n, P).steps + kPartSteps - 1) / kPartSteps;
            for (uint32_t left = parts; left > 0; --left, ++part) {
                ok = mbar_wait_cluster(&sums_full[part & 1], (part >> 1) & 1);
                if (__any_sync(kFull, !ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                add_sums(from + (part & 1) * BN, acc);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(in_block(&sums_empty[part & 1], 0));
            }
            if (!ok) break;
            const Unit w = unit_at(u, tiles_m, tiles_n, P);
            const uint32_t m0 = w.m * kPairM + rank * kBlockM + quarter * 32, n = w.n * BN + c0;
            if (m0 >= P.M || n >= P.N) continue;
            const bool far = !B_MN && OUT != kSums && far_scales<T::kWarpCols>(P, m0, n, lane);
            if (OUT == kAnywhere || far)
                store_anywhere<T::kWarpCols>(P, m0, n, lane, buf, acc, far);
            else
                store_tma<T::kWarpCols, OUT>(P, map_out, w.split, m0, n, lane, buf, acc);
        }
        if (lane == 0) tma_store_wait_read();  // the block's shared memory outlives the stores' reads
    }
    if (!ok) report_failure(&g_product_error, P.status, kErrPipelineTimeout);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) tmem_free_pair<kTmemCols>(0);
}

// Four columns of a row per thread.
__global__ void __launch_bounds__(256) join(const JoinParams P) {
    const uint64_t per_row = (P.N + 3) / 4, total = P.M * per_row, rows = (P.M + 31) / 32 * 32, pitch = (P.N + 31) / 32 * 32;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<uint64_t>(gridDim.x) * 256) {
        const uint64_t m = i / per_row, n = i % per_row * 4;
        float v[4] = {};
        for (uint32_t s = 0; s < P.splits; ++s) {
            const float4 w = *reinterpret_cast<const float4 *>(P.partial + (s * rows + m) * pitch + n);
            v[0] = __fadd_rn(v[0], w.x);
            v[1] = __fadd_rn(v[1], w.y);
            v[2] = __fadd_rn(v[2], w.z);
            v[3] = __fadd_rn(v[3], w.w);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (n + j >= P.N) break;
            float r = v[j];
            if (P.m_scale) {
                const float ms = __ldg(P.m_scale + m), ns = __ldg(P.n_scale + n + j);
                r = far_scale(ms) || far_scale(ns) ? scaled_far(r, ms, ns) : __fmul_rn(r, __fmul_rn(ms, ns));
            }
            if (P.bias) r = __fadd_rn(r, __ldg(P.bias + n + j));
            if (P.out_bf16) {
                static_cast<uint16_t *>(P.out)[m * P.out_stride + n + j] = to_bf16(r);
            } else {
                float *o = static_cast<float *>(P.out) + m * P.out_stride + n + j;
                *o = P.accumulate ? __fadd_rn(*o, r) : r;
            }
        }
    }
}

// ------------------------------------------------------------------ the host

// `rows` rows of `dim` elements `stride` apart, as boxes of box_rows rows of 128
// bytes under the 128-byte swizzle; reads outside give zeros, writes are dropped.
bool make_map(CUtensorMap *map, const void *p, bool bf16, uint64_t rows, uint64_t dim, uint64_t stride, uint32_t box_rows) {
    const uint32_t esize = bf16 ? 2 : 4;
    const cuuint64_t dims[2] = {dim, rows}, strides[1] = {stride * esize};
    const cuuint32_t box[2] = {128 / esize, box_rows}, unit[2] = {1, 1};
    EncodeTiled fn = encode_tiled();
    return fn && fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                    const_cast<void *>(p), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A 16-bit operand in memory.
struct Operand {
    const void *p;
    uint64_t rows, dim, stride;
};

bool tma_fits(const void *p, uint64_t stride, size_t esize) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride * esize % 16 == 0;
}

// How a product of M x N results over L terms is cut.
struct Plan {
    int bn;
    uint32_t splits, split_steps;
};

constexpr uint32_t kMaxSplits = 16;

// The cheapest of a few cuts by an estimate in SM cycles: a pair goes through
// ceil(units / pairs) units, each of its steps at 512 cycles (the tensor core's rate
// for 256 x 256 x 64) or, for the narrower tile, hardly less (its loads bound it),
// plus a start and a store of about 3000; a split one
// also writes and reads its sums (about 5000 bytes a cycle) in a second launch.
// `pairs` is fixed, so that the workspace's size does not depend on the device.
Plan plan_for(uint64_t M, uint64_t N, uint64_t L) {
    constexpr uint64_t kPairs = 76;
    const uint64_t steps = std::max<uint64_t>(1, (L + kStep - 1) / kStep);
    Plan best{256, 1, static_cast<uint32_t>(steps)};
    double best_cost = 1e300;
    for (int bn : {256, 128}) {
        const uint64_t tiles = ((M + kPairM - 1) / kPairM) * ((N + bn - 1) / bn);
        for (uint32_t s = 1; s <= kMaxSplits && (s == 1 || (steps / s >= 4 && tiles < kPairs)); ++s) {
            const uint64_t per = (steps + s - 1) / s, splits = (steps + per - 1) / per;
            const uint64_t waves = (tiles * splits + kPairs - 1) / kPairs;
            double cost = static_cast<double>(waves) * (static_cast<double>(per) * (bn == 256 ? 512 : 480) + 3000);
            if (splits > 1) cost += 6000 + static_cast<double>(splits) * M * N * 8 / 5000;
            if (cost < best_cost) {
                best_cost = cost;
                best = {bn, static_cast<uint32_t>(splits), static_cast<uint32_t>(per)};
            }
        }
    }
    return best;
}

// Sums of a split contraction: rows and row pitch in whole 32s.
uint64_t partial_bytes(uint64_t M, uint64_t N, uint64_t L) {
    const Plan p = plan_for(M, N, L);
    return p.splits > 1 ? p.splits * ceil32(M) * ceil32(N) * 4 : 0;
}

template <int BN, bool A_MN, bool B_MN, Output OUT>
cudaError_t launch_gemm(const Operand &a, const Operand &b, const GemmParams &g, cudaStream_t stream) {
    using T = Tile<BN>;
    const auto kernel = gemm<BN, A_MN, B_MN, OUT>;
    CUtensorMap ma, mb, mo{};
    bool mapped = make_map(&ma, a.p, true, a.rows, a.dim, a.stride, A_MN ? kStep : kBlockM) &&
                  make_map(&mb, b.p, true, b.rows, b.dim, b.stride, B_MN ? kStep : T::kRowsB);
    if (OUT == kSums) mapped = mapped && make_map(&mo, g.partial, false, g.splits * ceil32(g.M), g.N, g.partial_pitch, 32);
    if (OUT == kF32 || OUT == kF32Add || OUT == kBf16) mapped = mapped && make_map(&mo, g.out, OUT == kBf16, g.M, g.N, g.out_stride, 32);
    if (!mapped) return cudaErrorInvalidValue;
    cudaError_t e = prepare_dynamic_smem(reinterpret_cast<const void *>(kernel), T::kSmem);
    if (e != cudaSuccess) return e;
    const uint64_t units = ((g.M + kPairM - 1) / kPairM) * ((g.N + BN - 1) / BN) * g.splits;
    if (units > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
    const uint64_t most = sm_count() / 2;  // one block per SM, in pairs
    return launch_chained(kernel, static_cast<unsigned>(2 * (units < most ? units : most)), kGemmThreads, T::kSmem, stream, ma, mb,
                          mo, g);
}

template <bool A_MN, bool B_MN, Output OUT>
cudaError_t launch_tile(int bn, const Operand &a, const Operand &b, const GemmParams &g, cudaStream_t stream) {
    return bn == 256 ? launch_gemm<256, A_MN, B_MN, OUT>(a, b, g, stream) : launch_gemm<128, A_MN, B_MN, OUT>(a, b, g, stream);
}

// ADDS: this product may accumulate.
template <bool A_MN, bool B_MN, bool ADDS>
cudaError_t launch_product(const Operand &a, const Operand &b, GemmParams g, void *partial, cudaStream_t stream) {
    const Plan plan = plan_for(g.M, g.N, g.L);
    g.splits = plan.splits;
    g.split_steps = plan.split_steps;
    g.partial = static_cast<float *>(partial);
    g.partial_pitch = ceil32(g.N);
    if (g.splits > 1) {
        const cudaError_t e = launch_tile<A_MN, B_MN, kSums>(plan.bn, a, b, g, stream);
        if (e != cudaSuccess) return e;
        return launch_join({g.partial, g.splits, g.M, g.N, g.out, g.out_stride, g.out_bf16, g.accumulate, g.m_scale,
                            g.n_scale, g.bias}, stream);
    }
    if (!tma_fits(g.out, g.out_stride, g.out_bf16 ? 2 : 4)) return launch_tile<A_MN, B_MN, kAnywhere>(plan.bn, a, b, g, stream);
    if (g.out_bf16) return launch_tile<A_MN, B_MN, kBf16>(plan.bn, a, b, g, stream);
    if constexpr (ADDS)
        if (g.accumulate) return launch_tile<A_MN, B_MN, kF32Add>(plan.bn, a, b, g, stream);
    return launch_tile<A_MN, B_MN, kF32>(plan.bn, a, b, g, stream);
}

// Column sums of bf16 rows: a cluster of eight blocks owns 32 Q columns, lane l columns
// Q l .. Q l + Q - 1, and the cluster's 256 warps every 256th row, eight rows in
// flight; the warps' fp32 sums are added in order in each block, the blocks' in order
// by the first.  Loads in flight bound it: 8192 x 4096 takes 20 us, 28 with 64 warps.
template <int Q>
__global__ void __cluster_dims__(8, 1, 1) __launch_bounds__(1024)
    column_sums(const uint16_t *x, uint64_t stride, uint64_t rows, uint64_t cols, float *out, int accumulate) {
    __shared__ float sums[32][32 * Q], total[32 * Q];
    using R = typename RawOf<uint16_t, Q>::type;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = cluster_rank();
    const uint64_t first = static_cast<uint64_t>(blockIdx.x / 8) * 32 * Q, c = first + lane * Q;
    float s[Q] = {};
    if (c < cols) {
#pragma unroll 8
        for (uint64_t r = rank * 32 + warp; r < rows; r += 256) {
            const R v = load_unit<uint16_t, Q>(x + r * stride + c);
#pragma unroll
            for (int j = 0; j < Q; ++j) s[j] = __fadd_rn(s[j], v.get(j));
        }
    }
#pragma unroll
    for (int j = 0; j < Q; ++j) sums[warp][j * 32 + lane] = s[j];
    __syncthreads();
    if (threadIdx.x < 32 * Q) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < 32; ++w) v = __fadd_rn(v, sums[w][threadIdx.x]);
        total[threadIdx.x] = v;
    }
    cluster_sync();
    const uint64_t mine = first + (threadIdx.x & 31) * Q + threadIdx.x / 32;
    if (rank == 0 && threadIdx.x < 32 * Q && mine < cols) {
        float v = 0.0f;
#pragma unroll
        for (uint32_t b = 0; b < 8; ++b) {
            float part;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(part) : "r"(in_block(&total[threadIdx.x], b)) : "memory");
            v = __fadd_rn(v, part);
        }
        out[mine] = accumulate ? __fadd_rn(out[mine], v) : v;
    }
    cluster_sync();  // the first block reads the others' shared memory
}

cudaError_t launch_column_sums(const ProductParams &p, cudaStream_t stream) {
    const bool eights = p.N % 8 == 0 && tma_fits(p.dy, p.dy_stride, 2);
    const int cols = eights ? 256 : 32;
    const auto kernel = eights ? column_sums<8> : column_sums<1>;
    kernel<<<static_cast<unsigned>(8 * ((p.N + cols - 1) / cols)), 1024, 0, stream>>>(p.dy, p.dy_stride, p.T, p.N, p.dbias,
                                                                                    p.accumulate);
    return cudaGetLastError();
}

// Row length, in elements, of a widened matrix in the workspace: whole 128-byte rows.
uint64_t padded(uint64_t dim) { return (dim + 63) / 64 * 64; }
uint64_t widened_bytes(uint64_t rows, uint64_t dim) { return (rows * padded(dim) * 2 + 255) / 256 * 256; }

// Codes (times their scale, if there is one) as bf16 rows in the workspace; two
// matrices of one row length in one launch.
struct Widen {
    const int8_t *codes;
    const float *scale;
    uint64_t rows;
    void *to;
    Operand op(uint64_t dim) const { return {to, rows, dim, padded(dim)}; }
};

cudaError_t widen(uint64_t dim, const Widen &a, const Widen &b, cudaStream_t stream) {
    RowCodesParams p{};
    p.codes_in = a.codes;
    p.scale_in = a.scale;
    p.out = a.to;
    p.first_rows = a.rows;
    p.codes_in2 = b.codes;
    p.scale_in2 = b.scale;
    p.out2 = b.to;
    p.rows = a.rows + b.rows;
    p.dim = static_cast<uint32_t>(dim);
    p.out_stride = padded(dim);
    return launch_rows_int8_decode(p, 1, stream);
}

// dy as TMA can read it: in place, or copied to the workspace.
cudaError_t readable_dy(const ProductParams &p, void *room, Operand &op, cudaStream_t stream) {
    op = {p.dy, p.T, p.N, p.dy_stride};
    if (tma_fits(p.dy, p.dy_stride, 2)) return cudaSuccess;
    op = {room, p.T, p.N, padded(p.N)};
    return launch_ragged_copy16(p.dy, p.dy_stride, p.T, static_cast<uint32_t>(p.N), static_cast<uint16_t *>(room), padded(p.N),
                                stream);
}

GemmParams outputs(const ProductParams &p, uint64_t M, uint64_t N, uint64_t L) {
    GemmParams g{};
    g.M = M;
    g.N = N;
    g.L = L;
    g.out = p.out;
    g.out_stride = p.out_stride;
    g.out_bf16 = p.out_bf16;
    g.accumulate = p.accumulate;
    g.status = p.status;
    return g;
}

}  // namespace

cudaError_t launch_join(const JoinParams &p, cudaStream_t stream) {
    const uint64_t work = p.M * ((p.N + 3) / 4);
    const int grid = persistent_grid(reinterpret_cast<const void *>(&join), 256, (work + 255) / 256);
    join<<<grid, 256, 0, stream>>>(p);  // chained, it measured 1 us slower
    return cudaGetLastError();
}

// Which kernel multiplies T tokens: the weights are read as codes by qc_int8_few.cu up
// to kFewTokens.  Up to kWideAny qc_int8_wide.cu reads them so; up to kWideInPlace if the
// weights are few and lie as TMA reads them (else they are copied first); and up to kWideMost
// if the whole product is small.  Beyond, both operands are widened in memory and this
// file's tiles multiply them.  Weights of 4096 x 4096: 16 tokens take 7 us against the next
// kernel's 10, 256 take 19.2 us against 22.7, 512 28.2 against 28.6, and 1024 34 against 52.
// 11000 x 4096: 384 tokens 55 us against 66, 512 74 against 67.  Copied, 4096 x 4097: 384
// tokens 29 us against 35, and 4096 x 1025 with 512 17 against 14.  Small: 1024 x 1024, 1024
// tokens 8.3 us against 11.1, 1531 x 2052 (copied) 640 tokens 15.3 against 19.4, but 2048 x
// 2048, 896 tokens 17.1 against 15.7.
constexpr uint64_t kFewTokens = 16, kWideAny = 384, kWideInPlace = 512, kWideMost = 2048;
constexpr uint64_t kFewWeights = 1u << 25, kSmallProduct = 2500000000;

bool wide_always(uint64_t T, uint64_t N, uint64_t K) { return T <= kWideAny || (T <= kWideMost && T * N * K <= kSmallProduct); }
bool wide_in_place(uint64_t T, uint64_t N, uint64_t K) { return T <= kWideInPlace && N * K <= kFewWeights; }

size_t int8_matmul_workspace(uint64_t T, uint64_t N, uint64_t K, bool readable) {
    if (T <= kFewTokens) return 0;
    if (wide_always(T, N, K) || (wide_in_place(T, N, K) && readable)) return wide_tokens_workspace(T, N, K, readable);
    return widened_bytes(T, K) + widened_bytes(N, K) + partial_bytes(T, N, K);
}
size_t int8_input_grad_workspace(uint64_t T, uint64_t N, uint64_t K) {
    return widened_bytes(N, K) + widened_bytes(T, N) + partial_bytes(T, K, N);
}
size_t int8_weight_grad_workspace(uint64_t T, uint64_t N, uint64_t K) {
    return widened_bytes(T, K) + widened_bytes(T, N) + partial_bytes(N, K, T);
}

cudaError_t launch_int8_matmul(const ProductParams &p, cudaStream_t stream) {
    if (p.T <= kFewTokens) return launch_int8_few(p, stream);
    if (wide_always(p.T, p.N, p.K) || (wide_in_place(p.T, p.N, p.K) && wide_tokens_readable(p.x_codes, p.w_codes, p.K))) return launch_int8_wide(p, stream);
    uint8_t *ws = static_cast<uint8_t *>(p.workspace);
    const Widen x{p.x_codes, nullptr, p.T, ws}, w{p.w_codes, nullptr, p.N, ws + widened_bytes(p.T, p.K)};
    const cudaError_t e = widen(p.K, x, w, stream);
    if (e != cudaSuccess) return e;
    GemmParams g = outputs(p, p.T, p.N, p.K);
    g.m_scale = p.x_scale;
    g.n_scale = p.w_scale;
    g.bias = p.bias;
    return launch_product<false, false, false>(x.op(p.K), w.op(p.K), g, ws + widened_bytes(p.T, p.K) + widened_bytes(p.N, p.K), stream);
}

cudaError_t launch_int8_input_grad(const ProductParams &p, cudaStream_t stream) {
    Operand dy;
    uint8_t *ws = static_cast<uint8_t *>(p.workspace);
    const Widen w{p.w_codes, p.w_scale, p.N, ws};
    cudaError_t e = widen(p.K, w, {}, stream);
    if (e == cudaSuccess) e = readable_dy(p, ws + widened_bytes(p.N, p.K), dy, stream);
    if (e != cudaSuccess) return e;
    return launch_product<false, true, false>(dy, w.op(p.K), outputs(p, p.T, p.K, p.N),
                                       ws + widened_bytes(p.N, p.K) + widened_bytes(p.T, p.N), stream);
}

cudaError_t launch_int8_weight_grad(const ProductParams &p, cudaStream_t stream) {
    cudaError_t e;
    if (p.T == 0) {  // not accumulating: the gradients are zero
        e = cudaMemsetAsync(p.out, 0, p.N * p.K * (p.out_bf16 ? 2 : 4), stream);
        if (e == cudaSuccess && p.dbias) e = cudaMemsetAsync(p.dbias, 0, p.N * 4, stream);
        return e;
    }
    Operand dy;
    uint8_t *ws = static_cast<uint8_t *>(p.workspace);
    const Widen x{p.x_codes, p.x_scale, p.T, ws};
    e = widen(p.K, x, {}, stream);
    if (e == cudaSuccess) e = readable_dy(p, ws + widened_bytes(p.T, p.K), dy, stream);
    if (e == cudaSuccess) e = launch_product<true, true, true>(dy, x.op(p.K), outputs(p, p.N, p.K, p.T),
                                       ws + widened_bytes(p.T, p.K) + widened_bytes(p.T, p.N), stream);
    if (e != cudaSuccess || !p.dbias) return e;
    return launch_column_sums(p, stream);
}

}  // namespace qc
