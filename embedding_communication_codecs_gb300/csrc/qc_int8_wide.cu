// qc_int8_wide.cu -- the product of the 8-bit layer for tens to hundreds of tokens, the
// weights read from memory once and as codes.
//
// The weights' N K bytes are what has to be read, and widening them in memory first
// would move five times that.  The product is turned round, y^T = W X^T: the weights
// are the tensor core's A operand, which may come from tensor memory, so a widened
// weight never passes through shared memory again:
//
//     TMA -> codes in shared memory -> registers -> f16 in tensor memory -> tcgen05.mma
//
// (f16 holds every int8 exactly.)  The tokens, B, go from codes to f16 in shared
// memory on the way.  A block owns 128 weight rows x BT tokens and a range of the
// contraction, in steps of 128 codes.  Warp 0 loads codes, warp 1 issues the matrix
// instructions, and warps 4 to 15 widen and, at the end, store: three groups of four
// (a warp reaches 32 lanes of tensor memory) take every third step, so that the
// latency of a step, several hundred cycles of waits and conversions, is paid three
// at a time.  Tensor memory (64 columns a step next to the columns of the sums) and shared
// memory bound the ring of kRing widened steps, and the waits its ratio to the stages.
// The lanes of a storing warp hold neighbouring outputs of one token, so its stores
// are whole lines wherever y's rows start.
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
constexpr int kRows = 128;
constexpr int kThreads = 512, kGroups = 3;
// All of tensor memory, so it starts at column 0: the sums there, the ring at the end.
constexpr int kACols = kStepK / 2, kTmemCols = 512;

constexpr int kPartSteps = 16;
constexpr uint64_t max_steps(int bt) { return bt == 48 || bt == 96 ? 48 : bt == 64 ? 64 : 32; }

template <int BT>
struct Wide {
    static constexpr int kBytesW = kRows * kStepK, kBytesX = BT * kStepK;  // codes of a step
    static constexpr int kCodes = kBytesW + kBytesX;
    static constexpr int kBytesF = BT * kStepK * 2;                       // widened tokens of a step
    static constexpr int kRing = BT == 32 ? 7 : BT == 48 ? 5 : BT == 64 ? 4 : 3;
    static constexpr int kStages = BT == 32 ? 8 : BT == 48 ? 7 : BT == 64 ? 6 : BT == 96 ? 5 : 4;
    static constexpr int kFirstA = kTmemCols - kRing * kACols;
    // The tensor core's running sum loses up to a unit in the last place per instruction,
    // always towards zero: codes of one sign are 5e-5 off after 16384 terms, 3e-6 after 4096.  A
    // sum is cut into parts of 16 steps = 2048 terms, each in columns of its own, added in
    // fp32 as they are stored; a unit has no more steps than there is room for parts.
    static constexpr int kSumCols = (BT + 31) / 32 * 32;
    static constexpr int kSums = kFirstA / kSumCols;
    static constexpr int kSmem = kStages * kCodes + kRing * kBytesF + 1024;
    static_assert(kSums >= 2 && kSums * kPartSteps == max_steps(BT), "the sums and the ring share tensor memory");
    // A barrier's wait tells a phase from the one before it, not from the one before
    // that.  A group at step i has passed step i - kGroups, whose slot was freed by step
    // i - kGroups - kRing, and the instructions go in order: so the slot's last phase but one
    // is over (i - 2 kRing <= i - kGroups - kRing), and once the slot of step i is free, step
    // i - kRing is done and with it the stage's last user (i - kStages <= i - kRing).
    static_assert(kRing >= kGroups && kStages >= kRing, "no wait may pass on an older phase");
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
    const uint32_t tiles_n = static_cast<uint32_t>((P.N + kRows - 1) / kRows);
    const uint32_t all = static_cast<uint32_t>((P.K + kStepK - 1) / kStepK);
    const uint32_t split = u / (tiles_t * tiles_n), first = split * P.split_steps;
    return {u / tiles_t % tiles_n, u % tiles_t, split, first, min(P.split_steps, all - first)};
}

// scaled_far() of a lane's eight sums, whose tokens' scales lanes `first` on hold.  One call for
// eight: unrolled into the stores, tiles of 128 tokens took 31.1 us (16384 x 4096) instead of 29.2.
struct Eight {
    uint32_t v[8];
};
__device__ __noinline__ Eight far_eight(Eight e, float xs, int first, float ws) {
#pragma unroll
    for (int j = 0; j < 8; ++j) e.v[j] = __float_as_uint(scaled_far(__uint_as_float(e.v[j]), __shfl_sync(kFull, xs, first + j), ws));
    return e;
}

template <int BT>
__global__ void __launch_bounds__(kThreads, 1)
    wide_tokens(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const WideParams P) {
    using C = Wide<BT>;
    constexpr int S = C::kStages, R = C::kRing;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[S], empty[S], ready[R], freed[R], sums_full, sums_empty;
    __shared__ uint32_t tmem_slot;
    uint8_t *const widened = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);  // tokens, R steps
    uint8_t *const codes = widened + R * C::kBytesF;                             // S steps
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const uint32_t units = static_cast<uint32_t>((P.T + BT - 1) / BT) * static_cast<uint32_t>((P.N + kRows - 1) / kRows) * P.splits;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 4);  // the warps that widen it
        }
        for (int r = 0; r < R; ++r) {
            mbar_init(&ready[r], 4);  // the same warps
            mbar_init(&freed[r], 1);  // the matrix instructions that read it
        }
        mbar_init(&sums_full, 1);
        mbar_init(&sums_empty, 4 * kGroups);
        fence_barrier_init();
        prefetch_map(&map_w);
        prefetch_map(&map_x);
    }
    if (warp == 1) tmem_alloc<kTmemCols>(&tmem_slot);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            for (uint32_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const WideUnit w = wide_unit<BT>(u, P);
                for (uint32_t k = 0; k < w.steps; ++k, ++it) {
                    const uint32_t s = it % S;
                    if (!mbar_wait(&empty[s], ((it / S) & 1) ^ 1)) {
                        ok = false;
                        break;
                    }
                    uint8_t *to = codes + s * C::kCodes;
                    const int k0 = static_cast<int>((w.first + k) * kStepK);
                    mbar_arrive_expect_tx(&full[s], C::kCodes);
                    tma_load(to, &map_w, k0, static_cast<int>(w.n * kRows), &full[s]);
                    tma_load(to + C::kBytesW, &map_x, k0, static_cast<int>(w.t * BT), &full[s]);
                }
            }
            // the block stays while a copy is in flight
            for (uint32_t i = it > S ? it - S : 0; i < it; ++i) ok &= mbar_wait(&full[i % S], (i / S) & 1);
        }
    } else if (warp == 1) {
        // the whole warp goes round, one lane issues
        constexpr uint32_t kInstr = f16_instruction(kRows, BT);
        const bool issues = one_lane();
        uint32_t it = 0, done = 0;
        for (uint32_t u = blockIdx.x; u < units && ok; u += gridDim.x, ++done) {
            const uint32_t steps = wide_unit<BT>(u, P).steps;
            ok = __all_sync(kFull, mbar_wait(&sums_empty, (done & 1) ^ 1));
            for (uint32_t k = 0; k < steps && ok; ++k, ++it) {
                const uint32_t r = it % R;
                ok = __all_sync(kFull, mbar_wait(&ready[r], (it / R) & 1));
                if (!ok) break;
                tc_fence_after();
                const uint8_t *x = widened + r * C::kBytesF;
                const uint64_t b0 = smem_operand(x, 0), b1 = smem_operand(x + C::kBytesF / 2, 0);
                if (issues) {
#pragma unroll
                    for (int j = 0; j < kStepK / 16; ++j)
                        mma_tmem(k / kPartSteps * C::kSumCols, C::kFirstA + r * kACols + 8 * j, (j < 4 ? b0 : b1) + (j & 3) * 2, kInstr,
                                 k % kPartSteps > 0 || j > 0);
                    mma_commit(&freed[r]);
                }
                __syncwarp();
            }
            if (issues && ok) mma_commit(&sums_full);
            __syncwarp();
        }
    } else if (warp >= 4) {
        const uint32_t group = (warp - 4) >> 2;
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t mine = static_cast<uint32_t>(quarter * 32) << 16;  // the warp's lanes of tensor memory
        uint32_t it = 0, done = 0;
        for (uint32_t u = blockIdx.x; u < units && ok; u += gridDim.x, ++done) {
            const WideUnit w = wide_unit<BT>(u, P);
            const uint64_t n = static_cast<uint64_t>(w.n) * kRows + row;
            const uint32_t t0 = w.t * BT, left = static_cast<uint32_t>(P.T) - t0;
            const bool live = n < P.N;
            // what the stores will need, asked for before the sums are there
            const float ws = live ? __ldg(P.w_scale + n) : 0.0f, bias = live && P.bias ? __ldg(P.bias + n) : 0.0f;
            float xs[(BT + 31) / 32];
#pragma unroll
            for (int i = 0; i < (BT + 31) / 32; ++i) xs[i] = 32 * i + lane < left ? __ldg(P.x_scale + t0 + 32 * i + lane) : 0.0f;
            for (uint32_t k = 0; k < w.steps; ++k, ++it) {
                if (it % kGroups != group) continue;
                const uint32_t s = it % S, r = it % R;
                ok = mbar_wait(&freed[r], ((it / R) & 1) ^ 1) && mbar_wait(&full[s], (it / S) & 1);
                const uint8_t *from = codes + s * C::kCodes;
                uint4 c[8], x[BT / 16];
#pragma unroll
                for (int i = 0; i < 8; ++i) c[i] = *reinterpret_cast<const uint4 *>(from + row * 128 + ((i ^ (row & 7)) << 4));
                // 16 codes of token t, piece p of its eight
#pragma unroll
                for (int i = 0; i < BT / 16; ++i) {
                    const int t = i * 16 + (row >> 3), p = row & 7;
                    x[i] = *reinterpret_cast<const uint4 *>(from + C::kBytesW + t * 128 + ((p ^ (t & 7)) << 4));
                }
                if (__any_sync(kFull, !ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t f[32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        widen4(c[4 * h + i].x, f[8 * i], f[8 * i + 1]);
                        widen4(c[4 * h + i].y, f[8 * i + 2], f[8 * i + 3]);
                        widen4(c[4 * h + i].z, f[8 * i + 4], f[8 * i + 5]);
                        widen4(c[4 * h + i].w, f[8 * i + 6], f[8 * i + 7]);
                    }
                    tmem_store32(mine + C::kFirstA + r * kACols + 32 * h, f);
                }
                uint8_t *to = widened + r * C::kBytesF;
#pragma unroll
                for (int i = 0; i < BT / 16; ++i) {
                    const int t = i * 16 + (row >> 3), p = row & 7;
                    uint4 lo, hi;
                    widen4(x[i].x, lo.x, lo.y);
                    widen4(x[i].y, lo.z, lo.w);
                    widen4(x[i].z, hi.x, hi.y);
                    widen4(x[i].w, hi.z, hi.w);
                    uint8_t *at = to + (p >> 2) * (C::kBytesF / 2) + t * 128;
                    *reinterpret_cast<uint4 *>(at + (((2 * (p & 3)) ^ (t & 7)) << 4)) = lo;
                    *reinterpret_cast<uint4 *>(at + (((2 * (p & 3) + 1) ^ (t & 7)) << 4)) = hi;
                }
                fence_proxy_async_shared();
                // The stage is given back only here, where its codes have been widened and stored: the
                // stores depend on the loaded values, so no load can come later.  Given back
                // right after the loads, it was refilled under some of them (measured: wrong
                // tokens in tiles of 64, none with volatile loads).  16384 x 4096 with 128 tokens takes
                // 29 us, 28 in the other order; with 64 tokens 21 either way.
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[s]);
                tmem_wait_store();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ready[r]);
            }
            if (ok) ok = mbar_wait(&sums_full, done & 1);
            if (__any_sync(kFull, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            bool far = far_scale(ws);
#pragma unroll
            for (int i = 0; i < (BT + 31) / 32; ++i) far |= far_scale(xs[i]);
            far = __any_sync(kFull, far);
            const uint64_t rows = (P.T + 31) / 32 * 32, pitch = (P.N + 31) / 32 * 32;
#pragma unroll
            for (int c = 0; c < BT; c += 8) {
                if (c >= left) break;
                if ((c / 8) % kGroups != group) continue;
                uint32_t v[8];
                tmem_load8(mine + c, v);
                tmem_wait_load();
                for (uint32_t part = 1; part * kPartSteps < w.steps; ++part) {
                    uint32_t more[8];
                    tmem_load8(mine + part * C::kSumCols + c, more);
                    tmem_wait_load();
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(__fadd_rn(__uint_as_float(v[j]), __uint_as_float(more[j])));
                }
                if (far && P.splits == 1) {
                    Eight e;
#pragma unroll
                    for (int j = 0; j < 8; ++j) e.v[j] = v[j];
                    e = far_eight(e, xs[c / 32], c & 31, ws);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = e.v[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float xt = __shfl_sync(kFull, xs[c / 32], (c + j) & 31);
                    if (c + j >= left || !live) continue;
                    const uint64_t t = t0 + c + j;
                    float y = __uint_as_float(v[j]);
                    if (P.splits > 1) {
                        P.partial[(w.split * rows + t) * pitch + n] = y;
                        continue;
                    }
                    if (!far) y = __fmul_rn(y, __fmul_rn(xt, ws));
                    if (P.bias) y = __fadd_rn(y, bias);
                    if (P.y_bf16)
                        static_cast<uint16_t *>(P.y)[t * P.y_stride + n] = to_bf16(y);
                    else
                        static_cast<float *>(P.y)[t * P.y_stride + n] = y;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sums_empty);
        }
    }
    if (!ok) report_failure(&g_wide_error, P.status, kErrPipelineTimeout);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tmem_free<kTmemCols>(0);
    }
}

struct WidePlan {
    int bt;
    uint32_t splits, split_steps;
};

// The token tile and the cuts of the contraction that cost least, in ns.  A step takes
// longer the wider the tile, as its tokens are widened with it; a unit starts and stores; a join is a launch and its sums written
// and read.  The figures were fitted to 1450 timed plans (1024 x 1024 to 16384 x 4096, 24 to
// 512 tokens): 5 % off on average, and the choice within 3 % of the best.  Small weights
// want many narrow tiles (1024 x 1024, 128 tokens: 6.5 us in tiles of 32, 11.4 in one of 128),
// large ones as few as there are (16384 x 4096: 30.5 us in one, 33.8 in two of 64).  The
// contraction is cut as far as two units for each SM, or as the parts of a sum need.
WidePlan wide_plan(uint64_t T, uint64_t N, uint64_t K) {
    constexpr uint64_t kBlocks = 152;
    const uint64_t steps = (K + kStepK - 1) / kStepK;
    WidePlan best{};
    double best_cost = 1e300;
    for (const int bt : {32, 48, 64, 96, 128}) {
        const uint64_t tiles = ((T + bt - 1) / bt) * ((N + kRows - 1) / kRows);
        const uint64_t least = (steps + max_steps(bt) - 1) / max_steps(bt);
        for (uint64_t s = least; s == least || (s <= 16 && steps / s >= 2 && tiles * s <= 2 * kBlocks); ++s) {
            const uint64_t per = (steps + s - 1) / s, splits = (steps + per - 1) / per;
            const uint64_t waves = (tiles * splits + kBlocks - 1) / kBlocks;
            double cost = static_cast<double>(waves) * (static_cast<double>(per) * (240 + 2.6 * bt) + 300 + 21.0 * bt);
            if (splits > 1) cost += 1800 + 0.0017 * static_cast<double>(splits) * static_cast<double>(T) * static_cast<double>(N);
            if (cost < best_cost) {
                best_cost = cost;
                best = {bt, static_cast<uint32_t>(splits), static_cast<uint32_t>(per)};
            }
        }
        if (static_cast<uint64_t>(bt) >= T) break;
    }
    return best;
}

// Rows of K codes, `pitch` bytes apart, as boxes of 128 codes under the 128-byte
// swizzle; zeros outside.
bool map_codes(CUtensorMap *map, const int8_t *p, uint64_t rows, uint64_t K, uint64_t pitch, uint32_t box_rows) {
    const cuuint64_t dims[2] = {K, rows}, strides[1] = {pitch};
    const cuuint32_t box[2] = {kStepK, box_rows}, unit[2] = {1, 1};
    EncodeTiled fn = encode_tiled();
    return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(p), dims, strides, box, unit,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Codes as TMA reads them: rows on 16-byte boundaries.
struct Codes {
    const int8_t *p;
    uint64_t pitch;
};
bool readable(const int8_t *p, uint64_t K) { return K % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
uint64_t pitch16(uint64_t K) { return (K + 15) / 16 * 16; }
uint64_t copied_bytes(uint64_t rows, uint64_t K) { return (rows * pitch16(K) + 255) / 256 * 256; }

template <int BT>
cudaError_t launch_wide(const ProductParams &p, const Codes &wc, const Codes &xc, const WideParams &w, cudaStream_t stream) {
    using C = Wide<BT>;
    const auto kernel = wide_tokens<BT>;
    CUtensorMap mw, mx;
    if (!map_codes(&mw, wc.p, p.N, p.K, wc.pitch, kRows) || !map_codes(&mx, xc.p, p.T, p.K, xc.pitch, BT)) return cudaErrorInvalidValue;
    const cudaError_t e = prepare_dynamic_smem(reinterpret_cast<const void *>(kernel), C::kSmem);
    if (e != cudaSuccess) return e;
    const uint64_t units = ((p.T + BT - 1) / BT) * ((p.N + kRows - 1) / kRows) * w.splits, most = sm_count();
    kernel<<<static_cast<unsigned>(units < most ? units : most), kThreads, C::kSmem, stream>>>(mw, mx, w);
    return cudaGetLastError();
}

}  // namespace

bool wide_tokens_readable(const int8_t *x_codes, const int8_t *w_codes, uint64_t K) {
    return readable(w_codes, K) && readable(x_codes, K);
}

// Room for the sums of a split contraction and, for codes that TMA cannot read where
// they lie, for copies of both matrices.
size_t wide_tokens_workspace(uint64_t T, uint64_t N, uint64_t K, bool readable) {
    const WidePlan plan = wide_plan(T, N, K);
    return (plan.splits > 1 ? plan.splits * ceil32(T) * ceil32(N) * 4 : 0) + (readable ? 0 : copied_bytes(N, K) + copied_bytes(T, K));
}

cudaError_t launch_int8_wide(const ProductParams &p, cudaStream_t stream) {
    const WidePlan plan = wide_plan(p.T, p.N, p.K);
    WideParams w{};
    w.T = p.T;
    w.N = p.N;
    w.K = p.K;
    w.splits = plan.splits;
    w.split_steps = plan.split_steps;
    w.partial = static_cast<float *>(p.workspace);
    w.y = p.out;
    w.y_stride = p.out_stride;
    w.y_bf16 = p.out_bf16;
    w.x_scale = p.x_scale;
    w.w_scale = p.w_scale;
    w.bias = p.bias;
    w.status = p.status;
    Codes wc{p.w_codes, p.K}, xc{p.x_codes, p.K};
    cudaError_t e = cudaSuccess;
    if (!wide_tokens_readable(p.x_codes, p.w_codes, p.K)) {
        int8_t *room = static_cast<int8_t *>(p.workspace) + (plan.splits > 1 ? plan.splits * ceil32(p.T) * ceil32(p.N) * 4 : 0);
        wc = {room, pitch16(p.K)};
        xc = {room + copied_bytes(p.N, p.K), pitch16(p.K)};
        e = launch_ragged_copy8(p.w_codes, p.N, room, p.x_codes, p.T, room + copied_bytes(p.N, p.K), static_cast<uint32_t>(p.K),
                                wc.pitch, stream);
        if (e != cudaSuccess) return e;
    }
    e = plan.bt == 32   ? launch_wide<32>(p, wc, xc, w, stream)
        : plan.bt == 48 ? launch_wide<48>(p, wc, xc, w, stream)
        : plan.bt == 96 ? launch_wide<96>(p, wc, xc, w, stream)
        : plan.bt == 64 ? launch_wide<64>(p, wc, xc, w, stream)
                        : launch_wide<128>(p, wc, xc, w, stream);
    if (e != cudaSuccess || w.splits == 1) return e;
    return launch_join({w.partial, w.splits, p.T, p.N, p.out, p.out_stride, p.out_bf16, 0, p.x_scale, p.w_scale, p.bias}, stream);
}

}  // namespace qc
