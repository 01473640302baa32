// wgrad.cu -- gradients of the weights of a product by group:
//
//   dW[g][n][k] = sum over g's rows t of dY[t][n] X[t][k],   bf16 rows, fp32 sums
//
// Rows are summed over as they lie: a TMA box of 64 rows and 64 columns (128 bytes) is
// an operand along M (dY) or N (X) of the tensor core, whose K runs down the rows; no
// transpose.  A tile is 128 columns of dY by 256 of X.  A group may end anywhere: the
// rows of a box past the last are the next group's, and those that share an MMA's step
// of 16 with it are overwritten with zeros in shared memory, on both sides.
//
// Warps: 0 copies (TMA) the boxes, 1 issues the MMAs (and clears the rows past the
// last), 2 to 5 empty one of two accumulators while the next tile is summed into the other.
#include "async.cuh"
#include "common.cuh"
#include "groups.cuh"
#include "internal.h"
#include "launch.cuh"
#include "lora.cuh"
#include "tc05.cuh"
#include "w4a16.h"

namespace w4a16 {

namespace {

constexpr int kRowStep = 64;                       // rows of a stage
constexpr int kTileN = 128, kTileK = 256;
constexpr int kBox = kRowStep * 128;               // bytes of 64 rows x 64 columns
constexpr int kWgStage = (kTileN + kTileK) / 64 * kBox, kWgStages = 4;
constexpr int kWgThreads = 192, kWgStore0 = 2, kWgStoreWarps = 4;
constexpr int kStoreBox = 32 * 128;                // bytes of 32 rows of dW, 128 bytes of each

struct GroupWgradArgs {
    const int32_t *m_sizes;
    int *status, *err;
    int M, N, K, groups, n_tiles, k_tiles;
};

constexpr int kWgOffStore = kWgStages * kWgStage, kWgOffBar = kWgOffStore + kWgStoreWarps * kStoreBox;
constexpr int kWgOffTab = kWgOffBar + (2 * kWgStages + 5) * 8 + 8;
inline size_t wgrad_smem(int groups) { return kWgOffTab + 2 * (groups + 1) * sizeof(int) + 1024; }

struct WgTile {
    int group, n0, k0, row0, rows;
};
__device__ __forceinline__ WgTile wg_tile(const GroupWgradArgs &a, const int *tab_rows, int id) {
    WgTile t;
    const int per = a.n_tiles * a.k_tiles;
    t.group = id / per;
    const int r = id - t.group * per;
    t.k0 = r / a.n_tiles * kTileK;
    t.n0 = r % a.n_tiles * kTileN;
    t.row0 = tab_rows[t.group];
    t.rows = tab_rows[t.group + 1] - t.row0;
    return t;
}

template <bool F32>
__global__ void __launch_bounds__(kWgThreads, 1)
grouped_wgrad_kernel(const __grid_constant__ CUtensorMap tmap_dy, const __grid_constant__ CUtensorMap tmap_x,
                     const __grid_constant__ CUtensorMap tmap_dw, const GroupWgradArgs a) {
    extern __shared__ unsigned char s_raw[];
    unsigned char *smem = s_raw + (-smem_u32(s_raw) & 1023);
    __shared__ int s_abort;
    __shared__ uint32_t s_tmem;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t ring = smem_u32(smem), full = ring + kWgOffBar, empty = full + 8 * kWgStages;
    const uint32_t dfull = empty + 8 * kWgStages, dempty = dfull + 16, drained = dempty + 16;
    int *tab_rows = reinterpret_cast<int *>(smem + kWgOffTab), *tab_tiles = tab_rows + a.groups + 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWgStages; ++i) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, 1);
        for (int i = 0; i < 2; ++i) mbar_init(dfull + 8 * i, 1), mbar_init(dempty + 8 * i, kWgStoreWarps);
        mbar_init(drained, 1);
        s_abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tc_alloc(smem_u32(&s_tmem), 2 * kTileK);
        tc_relinquish();
    }
    if (warp == 0 && lane == 0) tma_prefetch_desc(&tmap_dy), tma_prefetch_desc(&tmap_x), tma_prefetch_desc(&tmap_dw);
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0)
        scan_groups(a.m_sizes, a.groups, a.M, 1, 0, tab_rows, tab_tiles, blockIdx.x == 0 ? a.status : nullptr);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    volatile int *abort_flag = &s_abort;
    const int tiles = a.groups * a.n_tiles * a.k_tiles;
    bool lost = false;
    if (warp == 0) {
        int i = 0;
        for (int id = blockIdx.x; id < tiles && !lost; id += gridDim.x) {
            const WgTile t = wg_tile(a, tab_rows, id);
            const int boxes_n = min(kTileN, a.N - t.n0) > 64 ? 2 : 1, boxes_k = (min(kTileK, a.K - t.k0) + 63) / 64;
            for (int r = 0; r < t.rows; r += kRowStep, ++i) {
                const int s = i % kWgStages;
                const bool ok = i < kWgStages || mbar_wait(empty + 8 * s, (i / kWgStages - 1) & 1, abort_flag, a.err);
                lost = !__all_sync(0xffffffffu, ok);
                if (lost) break;
                if (elect_one()) {
                    const uint32_t dst = ring + s * kWgStage, bar = full + 8 * s;
                    mbar_arrive_expect_tx(bar, (boxes_n + boxes_k) * kBox);
                    for (int c = 0; c < boxes_n; ++c)
                        tma_load_2d(dst + c * kBox, &tmap_dy, t.n0 + 64 * c, t.row0 + r, bar);
                    for (int c = 0; c < boxes_k; ++c)
                        tma_load_2d(dst + (kTileN / 64 + c) * kBox, &tmap_x, t.k0 + 64 * c, t.row0 + r, bar);
                }
                __syncwarp();
            }
        }
        if (*abort_flag)
            for (int u = i > kWgStages ? i - kWgStages : 0; u < i; ++u)
                drain_wait(full + 8 * (u % kWgStages), (u / kWgStages) & 1);
    } else if (warp == 1) {
        int i = 0, n = 0;
        for (int id = blockIdx.x; id < tiles && !lost; id += gridDim.x) {
            const WgTile t = wg_tile(a, tab_rows, id);
            if (t.rows == 0) continue;
            const uint32_t idesc = tc_idesc_bf16(kTileN, (min(kTileK, a.K - t.k0) + 15) & ~15) | kTcAMajorM | kTcBMajorN;
            const int d = n & 1;
            const bool free = n < 2 || mbar_wait(dempty + 8 * d, (n / 2 - 1) & 1, abort_flag, a.err);
            lost = !__all_sync(0xffffffffu, free);
            if (lost) break;
            for (int r = 0; r < t.rows; r += kRowStep, ++i) {
                const int s = i % kWgStages;
                lost = !__all_sync(0xffffffffu, mbar_wait(full + 8 * s, (i / kWgStages) & 1, abort_flag, a.err));
                if (lost) break;
                const int rows = min(kRowStep, t.rows - r), steps = (rows + 15) / 16;
                if (rows % 16) {
                    // rows to the end of the last step, 128 bytes in each box
                    const int pad = 16 * steps - rows;
                    for (int m = lane; m < pad * 8 * (kTileN + kTileK) / 64; m += 32) {
                        const int box = m / (pad * 8), at = m % (pad * 8);
                        *reinterpret_cast<uint4 *>(smem + s * kWgStage + box * kBox + rows * 128 + at * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async();
                    __syncwarp();
                }
                tc_fence_after();
                const uint32_t st = ring + s * kWgStage;
                const uint64_t dn = tc_sdesc_sw128_mn(st, kBox), dk = tc_sdesc_sw128_mn(st + kTileN / 64 * kBox, kBox);
                if (elect_one()) {
                    for (int e = 0; e < steps; ++e)
                        tc_mma_ss(tmem + d * kTileK, dn + 128 * e, dk + 128 * e, idesc, r > 0 || e > 0);
                    tc_commit(empty + 8 * s);
                }
                __syncwarp();
            }
            if (lost) break;
            if (elect_one()) tc_commit(dfull + 8 * d);
            __syncwarp();
            ++n;
        }
        if (elect_one()) tc_commit(drained);
        __syncwarp();
        drain_wait(drained, 0);
    } else {
        // Lane l of a warp holds row 32 (warp % 4) + l of the tile; 32 rows and 128 bytes of
        // each leave as one box.
        const int sub = warp % 4;
        unsigned char *buf = smem + kWgOffStore + (warp - kWgStore0) * kStoreBox;
        constexpr int kCols = F32 ? 32 : 64;
        int n = 0;
        for (int id = blockIdx.x; id < tiles; id += gridDim.x) {
            const WgTile t = wg_tile(a, tab_rows, id);
            const int d = n & 1, width = min(kTileK, a.K - t.k0);
            if (t.rows && !lost) {
                lost = !__all_sync(0xffffffffu, mbar_wait(dfull + 8 * d, (n / 2) & 1, abort_flag, a.err));
                tc_fence_after();
            }
            for (int c = 0; c < width; c += kCols) {
                uint32_t v[kCols];
                if (t.rows && !lost) {
                    #pragma unroll
                    for (int e = 0; e < kCols; e += 16) {
                        uint32_t w[16];
                        tc_ld_32x32b_x16(tmem + (uint32_t(32 * sub) << 16) + d * kTileK + c + e, w);
                        tc_wait_ld_of(w);
                        #pragma unroll
                        for (int j = 0; j < 16; ++j) v[e + j] = w[j];
                    }
                } else {
                    #pragma unroll
                    for (int j = 0; j < kCols; ++j) v[j] = lost ? 0x7fffffffu : 0u;
                }
                if (lane == 0) bulk_wait_read<0>();      // the box before has left the buffer
                __syncwarp();
                #pragma unroll
                for (int q = 0; q < 8; ++q) {
                    uint4 p;
                    if (F32) {
                        p = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                    } else {
                        uint32_t h[4];
                        #pragma unroll
                        for (int j = 0; j < 4; ++j)
                            h[j] = pack_bf16x2_rn(__uint_as_float(v[(8 * q + 2 * j) % kCols]),
                                                  __uint_as_float(v[(8 * q + 2 * j + 1) % kCols]));
                        p = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                    *reinterpret_cast<uint4 *>(buf + lane * 128 + ((q ^ (lane & 7)) << 4)) = p;
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    if (t.n0 + 32 * sub < a.N)
                        tma_store_3d(&tmap_dw, t.k0 + c, t.n0 + 32 * sub, t.group, smem_u32(buf));
                    bulk_commit();
                }
                __syncwarp();                            // tcgen05.ld takes the whole warp
            }
            if (t.rows) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && !lost) mbar_arrive(dempty + 8 * d);
                ++n;
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tc_dealloc(tmem, 2 * kTileK);
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int ceil_div(long long x, long long y) { return int((x + y - 1) / y); }

template <bool F32>
cudaError_t launch_grouped_wgrad(const GroupWgradArgs &a, const uint16_t *dy, const uint16_t *x, void *dw, int sms,
                                 cudaStream_t s) {
    CUtensorMap ty, tx, tw;
    const cuuint32_t box[2] = {64, kRowStep};
    const cuuint64_t ydim[2] = {cuuint64_t(a.N), cuuint64_t(a.M)}, ystride[1] = {2 * ydim[0]};
    cudaError_t e = encode_tensor_map(&ty, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dy, ydim, ystride, box,
                                      CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    const cuuint64_t xdim[2] = {cuuint64_t(a.K), cuuint64_t(a.M)}, xstride[1] = {2 * xdim[0]};
    e = encode_tensor_map(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, xdim, xstride, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    const size_t each = F32 ? 4 : 2;
    const cuuint64_t wdim[3] = {cuuint64_t(a.K), cuuint64_t(a.N), cuuint64_t(a.groups)};
    const cuuint64_t wstride[2] = {a.K * each, a.K * each * a.N};
    const cuuint32_t wbox[3] = {cuuint32_t(128 / each), 32, 1};
    e = encode_tensor_map(&tw, F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, dw, wdim,
                          wstride, wbox, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    e = allow_smem<grouped_wgrad_kernel<F32>>(kTensorMaxSmem - 256);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)a.groups * a.n_tiles * a.k_tiles;
    return launch_chained(grouped_wgrad_kernel<F32>, dim3(unsigned(tiles < sms ? tiles : sms)), kWgThreads,
                          wgrad_smem(a.groups), 1, s, ty, tx, tw, a);
}

}  // namespace

}  // namespace w4a16

using namespace w4a16;

extern "C" w4a16_status w4a16_gemm_grouped_wgrad(const w4a16_bf16 *dY, const w4a16_bf16 *X,
                                                 const int32_t *M_sizes_dev, void *dW, int dw_bytes,
                                                 int num_groups, int M_total, int N, int K, int32_t *status_dev,
                                                 void *stream) {
    if (num_groups < 1 || num_groups > kMaxGroups || M_total < 0 || M_total > (1 << 24) || N < 1 || N > (1 << 24) ||
        K < 1 || K > (1 << 20))
        return W4A16_ERR_INVALID_ARG;
    if (dw_bytes != 4 && dw_bytes != 2) return W4A16_ERR_UNSUPPORTED;
    if (N % 8 || K % 8) return W4A16_ERR_UNSUPPORTED;
    if ((long long)num_groups * N > (1LL << 40) / K) return W4A16_ERR_INVALID_ARG;
    if (!M_sizes_dev || !dW || !status_dev || (M_total > 0 && (!dY || !X))) return W4A16_ERR_INVALID_ARG;
    if (!aligned(dY, 16) || !aligned(X, 16) || !aligned(dW, 16) || !aligned(M_sizes_dev, 4) ||
        !aligned(status_dev, 4))
        return W4A16_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M_total == 0) {
        if (cudaMemsetAsync(dW, 0, size_t(num_groups) * N * K * dw_bytes, s) != cudaSuccess) return W4A16_ERR_CUDA;
        return cudaMemsetAsync(status_dev, 0, sizeof *status_dev, s) == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA;
    }
    int sms = 0;
    if (device_sm_count(&sms) != 0 || sms < 1) return W4A16_ERR_CUDA;
    GroupWgradArgs a = {};
    a.m_sizes = M_sizes_dev, a.status = status_dev, a.err = device_error_word();
    if (!a.err) return W4A16_ERR_CUDA;
    a.M = M_total, a.N = N, a.K = K, a.groups = num_groups;
    a.n_tiles = ceil_div(N, kTileN), a.k_tiles = ceil_div(K, kTileK);
    const cudaError_t e = dw_bytes == 4 ? launch_grouped_wgrad<true>(a, dY, X, dW, sms, s)
                                        : launch_grouped_wgrad<false>(a, dY, X, dW, sms, s);
    return e == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA;
}
