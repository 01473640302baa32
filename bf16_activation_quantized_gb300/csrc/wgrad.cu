// wgrad.cu -- gradients of the weights of a product by group:
//
//   dW[g][n][k] = sum over g's rows t of dY[t][n] X[t][k],   bf16 rows, fp32 sums
//
// Rows are summed over as they lie: a TMA box of 64 rows and 64 columns (128 bytes) is
// an operand along M (dY) or N (X) of the tensor core, whose K runs down the rows; no
// transpose.  Two CTAs share a tile of 256 columns of each (cta_group::2): a CTA loads
// 128 columns of dY and 128 of X and holds the sums of its 128 rows of dW.
//
// A group may end anywhere.  Its last rows come in boxes of 16, 8, 4, 2 and 1 rows, and
// what they leave of an MMA's step of 16 in boxes past the last row of all, which TMA fills
// with zeros: 32 boxes at most, one a lane, counted with the others.  Rows of the next
// group are never loaded.
//
// With few tiles and many rows `split` pairs (a cluster of 2 split CTAs) share a tile's
// rows; the parts stand in shared memory and are added in the order of the pairs.
//
// The tensor core cuts its sums off instead of rounding them, so that those of many rows
// drift: with 16384 rows in one sum the result's error is 4.4e-6 of it, with 65536 1.9e-5.  A
// sum of 512 rows is therefore handed over and added in registers, in fp32: 4.8e-7 for both
// (256 rows: 2.4e-7, and 4 to 8 % of the time; sums of 32 bits in order have 4 to 6e-7).
//
// What bounds it: the tensor cores, 283 us for 4096 rows of 8192 and 8192 columns (1.03 of
// the measured cuBLAS rate; without pairs 356).  8 groups of 512 rows, 2048 x 4096 in fp32: 63
// us, where the results alone take 47 (groups of 64 rows) and the MMAs alone 36: the two
// overlap in part only.  4096 rows in uneven groups: 69 to 74 (tiles are dealt out by number,
// whatever their rows).  (Results stored by TMA in boxes of 4 KB: 107 us where 73 were.)
// Six stages: with five 73.
// Rows past a group's last cleared in shared memory instead take as long (70.8 us for
// 69.7 with groups of 511), with a hand-over between the CTAs for each group's last boxes.
//
// Warps: 0 copies (TMA) the boxes, 1 issues the MMAs, 4 to 11 empty one of two accumulators
// while the next rows are summed into the other.
#include "async.cuh"
#include "common.cuh"
#include "groups.cuh"
#include "internal.h"
#include "launch.cuh"
#include "lora.cuh"
#include "split_plan.h"
#include "stall.cuh"
#include "tc05.cuh"
#include "w4a16.h"

namespace w4a16 {

namespace {

constexpr int kRowStep = 64;                       // rows of a stage
constexpr int kSide = 256, kHalf = 128;            // columns of dY and of X of a tile, of a CTA
constexpr int kBox = kRowStep * 128;               // bytes of 64 rows x 64 columns
constexpr int kWgStage = 4 * kBox, kWgStages = 6;
constexpr int kWgThreads = 384, kAddWarp0 = 4, kAddWarps = 8;
// Registers a thread of the first four warps and of the adding ones: the launch's
// (168 x 384) are what the two shares draw on.
constexpr int kRegsIn = 72, kRegsAdd = 216;
static_assert(128 * kRegsIn + 256 * kRegsAdd <= 168 * kWgThreads, "registers");
constexpr int kStoreBox = 16 * 128;                // bytes of 16 rows of dW, 128 bytes of each
constexpr int kPart = 512;                         // rows that the tensor core sums before registers add

constexpr int kTailBoxes = 5;                      // heights 16, 8, 4, 2, 1

struct GroupWgradMaps {
    CUtensorMap full[2], tail[2][kTailBoxes];      // dY, X
};

struct GroupWgradArgs {
    const int32_t *m_sizes;
    int *status, *err;
    void *dw;
    int M, N, K, groups, n_tiles, k_tiles;
};

constexpr int kWgOffStore = kWgStages * kWgStage, kWgOffBar = kWgOffStore + kAddWarps * kStoreBox;
constexpr int kWgOffTab = kWgOffBar + (2 * kWgStages + 5) * 8 + 8;
inline size_t wgrad_smem(int groups) { return kWgOffTab + (groups + 1) * sizeof(int) + 1024; }
static_assert(kWgOffTab + (kMaxGroups + 1) * 4 + 1024 <= kTensorMaxSmem - 256, "shared memory");
static_assert(kHalf * kSide * 4 <= kWgOffStore, "a tile's sums lie over the ring");

struct WgTile {
    int group, n0, k0, row0, rows;                 // the tile's columns, the rows of this pair's part
};
__device__ __forceinline__ WgTile wg_tile(const GroupWgradArgs &a, const int *tab_rows, int id, int part, int split) {
    WgTile t;
    const int per = a.n_tiles * a.k_tiles;
    t.group = id / per;
    const int r = id - t.group * per;
    banded(r, a.n_tiles, a.k_tiles, t.n0, t.k0);
    t.n0 *= kSide, t.k0 *= kSide;
    const int first = tab_rows[t.group], rows = tab_rows[t.group + 1] - first;
    if (split == 1) {
        t.row0 = first, t.rows = rows;
    } else {
        const int steps = (rows + kRowStep - 1) / kRowStep;
        const int s0 = steps * part / split * kRowStep, s1 = steps * (part + 1) / split * kRowStep;
        t.row0 = first + s0, t.rows = min(rows, s1) - s0;
    }
    return t;
}

// Piece i of the rows below the last full step, `rows` of them: its first row and the
// height, 16 >> box; past the rows it is one of zeros.  False: there are no more.
__device__ __forceinline__ bool tail_piece(int rows, int i, int &first, int &box, bool &zeros) {
    first = 16 * i, box = 0, zeros = false;
    if (i < rows / 16) return true;
    const int rest = rows % 16;
    if (rest == 0) return false;
    i -= rows / 16;
    const int mine = __popc(rest);
    zeros = i >= mine;
    if (zeros) i -= mine;
    int bits = zeros ? 16 - rest : rest;               // a piece for each bit, the highest first
    first = rows / 16 * 16 + (zeros ? rest : 0);
    for (; i > 0 && bits; --i) {
        const int high = 1 << (31 - __clz(bits));
        first += high, bits -= high;
    }
    if (!bits) return false;
    box = 4 - (31 - __clz(bits));
    return true;
}

template <bool F32>
__global__ void __launch_bounds__(kWgThreads, 1)
grouped_wgrad_kernel(const __grid_constant__ GroupWgradMaps maps, const GroupWgradArgs a) {
    extern __shared__ unsigned char s_raw[];
    unsigned char *smem = s_raw + (-smem_u32(s_raw) & 1023);
    __shared__ int s_abort;
    __shared__ uint32_t s_tmem;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = cluster_rank(), split = cluster_size() / 2, half = rank & 1, part = rank / 2;
    const uint32_t ring = smem_u32(smem), full = ring + kWgOffBar, empty = full + 8 * kWgStages;
    // full: both CTAs' boxes have landed (counted in the even one)
    const uint32_t dfull = empty + 8 * kWgStages, dempty = dfull + 16, drained = dempty + 16;
    int *tab_rows = reinterpret_cast<int *>(smem + kWgOffTab);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWgStages; ++i) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, 1);
        for (int i = 0; i < 2; ++i) mbar_init(dfull + 8 * i, 1), mbar_init(dempty + 8 * i, 2 * kAddWarps);
        mbar_init(drained, 1);
        s_abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) tc_alloc_pair(smem_u32(&s_tmem), 2 * kSide);
    if (warp == 0 && lane == 0) tma_prefetch_desc(&maps.full[0]), tma_prefetch_desc(&maps.full[1]);
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0)
        scan_groups(a.m_sizes, a.groups, a.M, 1, 0, tab_rows, nullptr, blockIdx.x == 0 ? a.status : nullptr);
    tc_fence_before();
    __syncthreads();
    cluster_arrive();                                    // the others' barriers stand
    cluster_wait();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    volatile int *abort_flag = &s_abort;
    const int tiles = a.groups * a.n_tiles * a.k_tiles, id0 = int(blockIdx.x) / (2 * split);
    const int step = int(gridDim.x) / (2 * split);
    const uint16_t both = uint16_t(3u << (rank & ~1));
    bool lost = false;
    if (warp < kAddWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIn));
        if (warp == 0) {
            int i = 0;
            const uint32_t even = cluster_address(full, rank & ~1);
            // a lane's box of a part's last rows: dY or X, 64 columns
            const int side = lane / 2 % 2, c = lane % 2;
            for (int id = id0; id < tiles && !lost; id += step) {
                const WgTile t = wg_tile(a, tab_rows, id, part, split);
                for (int r = 0; r < t.rows; r += kRowStep, ++i) {
                    const int s = i % kWgStages;
                    const bool ok = i < kWgStages || mbar_wait(empty + 8 * s, (i / kWgStages - 1) & 1, abort_flag, a.err);
                    lost = !__all_sync(0xffffffffu, ok);
                    if (lost) break;
                    const uint32_t dst = ring + s * kWgStage, bar = even + 8 * s;
                    const int y = t.row0 + r, rows = t.rows - r, n0 = t.n0 + half * kHalf, k0 = t.k0 + half * kHalf;
                    if (stalled(i)) continue;
                    if (rows >= kRowStep) {
                        if (elect_one()) {
                            if (half == 0) mbar_arrive_expect_tx(full + 8 * s, 2 * kWgStage);
                            #pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                tma_load_2d_pair(dst + j * kBox, &maps.full[0], n0 + 64 * j, y, bar);
                                tma_load_2d_pair(dst + (2 + j) * kBox, &maps.full[1], k0 + 64 * j, y, bar);
                            }
                        }
                    } else {
                        if (half == 0 && lane == 0) mbar_arrive_expect_tx(full + 8 * s, 2 * 4 * 128 * ((rows + 15) & ~15));
                        __syncwarp();
                        int first, box;
                        bool zeros;
                        if (tail_piece(rows, lane / 4, first, box, zeros))
                            tma_load_2d_pair(dst + (2 * side + c) * kBox + first * 128, &maps.tail[side][box],
                                             (side ? k0 : n0) + 64 * c, zeros ? a.M : y + first, bar);
                    }
                    __syncwarp();
                }
            }
            // Every copy lands before the CTA ends (the pair's are counted in the even one).
            if (*abort_flag && half == 0)
                for (int u = i > kWgStages ? i - kWgStages : 0; u < i; ++u) drain_wait(full + 8 * (u % kWgStages), (u / kWgStages) & 1);
        } else if (warp == 1 && half == 0) {
            constexpr uint32_t idesc = tc_idesc_bf16(kSide, kSide) | kTcAMajorM | kTcBMajorN;
            int i = 0, n = 0;
            for (int id = id0; id < tiles && !lost; id += step) {
                const WgTile t = wg_tile(a, tab_rows, id, part, split);
                for (int r = 0; r < t.rows; r += kRowStep, ++i) {
                    const int s = i % kWgStages, d = n & 1, steps = (min(kRowStep, t.rows - r) + 15) / 16;
                    bool ok = r % kPart || n < 2 || mbar_wait(dempty + 8 * d, (n / 2 - 1) & 1, abort_flag, a.err);
                    ok = ok && mbar_wait(full + 8 * s, (i / kWgStages) & 1, abort_flag, a.err);
                    lost = !__all_sync(0xffffffffu, ok);
                    if (lost) break;
                    tc_fence_after();
                    const uint32_t st = ring + s * kWgStage;
                    const uint64_t dn = tc_sdesc_sw128_mn(st, kBox), dk = tc_sdesc_sw128_mn(st + 2 * kBox, kBox);
                    const bool ends = (r + kRowStep) % kPart == 0 || r + kRowStep >= t.rows;
                    if (elect_one()) {
                        #pragma unroll
                        for (int e = 0; e < kRowStep / 16; ++e)
                            if (e < steps)
                                tc_mma_ss_pair(tmem + d * kSide, dn + 128 * e, dk + 128 * e, idesc, r % kPart > 0 || e > 0);
                        tc_commit_pair(empty + 8 * s, both);
                        if (ends) tc_commit_pair(dfull + 8 * d, both);
                    }
                    __syncwarp();
                    n += ends;
                }
            }
            if (elect_one()) tc_commit_pair(drained, both);
            __syncwarp();
            drain_wait(drained, 0);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsAdd));
        // Lane l of a warp holds row 32 (warp % 4) + l of this CTA's half of the tile, 128 of its
        // columns; 16 rows and 128 bytes of each go through shared memory and leave as whole lines.
        const int sub = warp % 4, side = (warp - kAddWarp0) / 4;
        const uint32_t from = tmem + (uint32_t(32 * sub) << 16) + side * kHalf;
        const uint32_t done = cluster_address(dempty, rank & ~1);
        unsigned char *buf = smem + kWgOffStore + (warp - kAddWarp0) * kStoreBox;
        float *join = reinterpret_cast<float *>(smem) + (32 * sub + lane) * kSide;
        int n = 0;
        for (int id = id0; id < tiles; id += step) {
            const WgTile t = wg_tile(a, tab_rows, id, part, split);
            constexpr int kCols = 32;
            const int row = t.n0 + half * kHalf + 32 * sub, col0 = t.k0 + side * kHalf;
            // 32 columns: fp32 in two halves of 16 rows and 128 bytes of each, bf16 in 32 rows and 64
            // bytes; pieces of 16 bytes lie so that eight of them meet in no bank.
            auto put = [&](const uint32_t *v, int c) {
                if (F32) {
                    #pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (lane / 16 == h)
                            #pragma unroll
                            for (int q = 0; q < 8; ++q)
                                *reinterpret_cast<uint4 *>(buf + lane % 16 * 128 + ((q ^ (lane & 7)) << 4)) =
                                    make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                        __syncwarp();
                        #pragma unroll
                        for (int k = 0; k < 16; k += 4) {
                            const int r = k + lane / 8, q = lane % 8, col = col0 + c + 4 * q, at = row + 16 * h + r;
                            if (at < a.N && col < a.K)
                                *reinterpret_cast<uint4 *>(static_cast<float *>(a.dw) + ((long long)t.group * a.N + at) * a.K + col) =
                                    *reinterpret_cast<const uint4 *>(buf + r * 128 + ((q ^ (r & 7)) << 4));
                        }
                        __syncwarp();
                    }
                } else {
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t p[4];
                        #pragma unroll
                        for (int j = 0; j < 4; ++j)
                            p[j] = pack_bf16x2_rn(__uint_as_float(v[8 * q + 2 * j]), __uint_as_float(v[8 * q + 2 * j + 1]));
                        *reinterpret_cast<uint4 *>(buf + lane * 64 + ((q ^ (lane / 2 & 3)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
                    }
                    __syncwarp();
                    #pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        const int r = k + lane / 4, q = lane % 4, col = col0 + c + 8 * q, at = row + r;
                        if (at < a.N && col < a.K)
                            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.dw) + ((long long)t.group * a.N + at) * a.K + col) =
                                *reinterpret_cast<const uint4 *>(buf + r * 64 + ((q ^ (r / 2 & 3)) << 4));
                    }
                    __syncwarp();
                }
            };
            if (split == 1 && t.rows <= kPart) {
                // The tensor core has the whole sum: it leaves as it is read (8 groups of 64 rows, 2048 x
                // 4096 in fp32: 46.8 us, through the sums in registers 50.9).
                const int d = n & 1;
                if (t.rows && !lost) {
                    lost = !__all_sync(0xffffffffu, mbar_wait(dfull + 8 * d, (n / 2) & 1, abort_flag, a.err));
                    tc_fence_after();
                }
                #pragma unroll 1
                for (int c = 0; c < kHalf && col0 + c < a.K; c += kCols) {
                    uint32_t v[kCols];
                    if (t.rows && !lost) {
                        #pragma unroll
                        for (int e = 0; e < kCols; e += 16) {
                            uint32_t u[16];
                            tc_ld_32x32b_x16(from + d * kSide + c + e, u);
                            tc_wait_ld_of(u);
                            #pragma unroll
                            for (int j = 0; j < 16; ++j) v[e + j] = u[j];
                        }
                    } else {
                        #pragma unroll
                        for (int j = 0; j < kCols; ++j) v[j] = lost ? 0x7fffffffu : 0u;
                    }
                    put(v, c);
                }
                if (t.rows) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0 && !lost) mbar_arrive_cluster(done + 8 * d);
                    ++n;
                }
                continue;
            }
            float acc[kHalf];
            #pragma unroll
            for (int j = 0; j < kHalf; ++j) acc[j] = 0.f;
            for (int r = 0; r < t.rows && !lost; r += kPart, ++n) {
                const int d = n & 1;
                lost = !__all_sync(0xffffffffu, mbar_wait(dfull + 8 * d, (n / 2) & 1, abort_flag, a.err));
                if (lost) break;
                tc_fence_after();
                constexpr int kChunk = 16;
                #pragma unroll
                for (int c = 0; c < kHalf; c += kChunk) {
                    uint32_t v[kChunk];
                    tc_ld_32x32b_x16(from + d * kSide + c, v);
                    tc_wait_ld_of(v);
                    #pragma unroll
                    for (int e = 0; e < kChunk; ++e) acc[c + e] += __uint_as_float(v[e]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(done + 8 * d);
            }
            // A wait that ran out: this tile and the pair's later ones are NaN.
            if (lost) {
                #pragma unroll
                for (int j = 0; j < kHalf; ++j) acc[j] = __int_as_float(0x7fffffff);
            }
            if (split > 1) {
                // over the ring, whose boxes this tile's last MMAs have read; pieces of 16 bytes
                // placed so that eight rows' meet in no bank; a cluster has one tile
                #pragma unroll
                for (int q = 0; q < kHalf / 4; ++q)
                    *reinterpret_cast<float4 *>(join + 4 * ((side * (kHalf / 4) + q) ^ (lane & 7))) =
                        make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
                break;
            }
            #pragma unroll
            for (int c = 0; c < kHalf; c += kCols) {
                if (col0 + c >= a.K) break;
                uint32_t v[kCols];
                #pragma unroll
                for (int j = 0; j < kCols; ++j) v[j] = __float_as_uint(acc[c + j]);
                put(v, c);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive();                                    // the pair's MMAs have read both CTAs' memory
    cluster_wait();
    if (split > 1) {
        // Rows part, part + split, ... of this half of the tile, a warp a row, 8 columns a lane.
        int gone = 0;                                    // a wait ran out: copies may have landed on the sums
        for (int k = 0; k < 2 * split; ++k) gone |= ld_cluster1(&s_abort, k);
        const WgTile t = wg_tile(a, tab_rows, id0, part, split);
        for (int r = part + split * warp; r < min(kHalf, a.N - t.n0 - half * kHalf); r += split * (kWgThreads / 32)) {
            float4 s[2];
            for (int k = 0; k < split; ++k)
                #pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int q = 2 * lane + h;
                    const float4 v = ld_cluster4(reinterpret_cast<float *>(smem) + r * kSide + 4 * (q ^ (r & 7)), half + 2 * k);
                    if (k == 0) s[h] = v;
                    else s[h].x += v.x, s[h].y += v.y, s[h].z += v.z, s[h].w += v.w;
                }
            if (gone) s[0].x = s[0].y = s[0].z = s[0].w = s[1].x = s[1].y = s[1].z = s[1].w = __int_as_float(0x7fffffff);
            const int col = t.k0 + 8 * lane;
            if (col >= a.K) continue;
            const long long at = ((long long)t.group * a.N + t.n0 + half * kHalf + r) * a.K + col;
            if (F32) {
                float4 *w = reinterpret_cast<float4 *>(static_cast<float *>(a.dw) + at);
                w[0] = s[0], w[1] = s[1];
            } else {
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.dw) + at) =
                    make_uint4(pack_bf16x2_rn(s[0].x, s[0].y), pack_bf16x2_rn(s[0].z, s[0].w),
                               pack_bf16x2_rn(s[1].x, s[1].y), pack_bf16x2_rn(s[1].z, s[1].w));
            }
        }
        cluster_arrive();                                // the others have read this CTA's part
        cluster_wait();
    }
    tc_fence_after();
    if (warp == 1) tc_dealloc_pair(tmem, 2 * kSide);
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <bool F32>
cudaError_t launch_grouped_wgrad(const GroupWgradArgs &a, const uint16_t *dy, const uint16_t *x, int sms, cudaStream_t s) {
    GroupWgradMaps maps;
    for (int side = 0; side < 2; ++side) {
        const cuuint64_t dim[2] = {cuuint64_t(side ? a.K : a.N), cuuint64_t(a.M)}, stride[1] = {2 * dim[0]};
        for (int i = 0; i <= kTailBoxes; ++i) {
            const cuuint32_t box[2] = {64, cuuint32_t(i == kTailBoxes ? kRowStep : 16 >> i)};
            const cudaError_t e = encode_tensor_map(i == kTailBoxes ? &maps.full[side] : &maps.tail[side][i],
                                                    CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, side ? x : dy, dim, stride, box,
                                                    CU_TENSOR_MAP_SWIZZLE_128B);
            if (e != cudaSuccess) return e;
        }
    }
    const cudaError_t e = allow_smem<grouped_wgrad_kernel<F32>>(kTensorMaxSmem - 256);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)a.groups * a.n_tiles * a.k_tiles;
    const int pairs = sms / 2;
    const int split = wgrad_split(tiles, pairs, a.M, a.groups, kRowStep);
    const int clusters = int(split > 1 || tiles < pairs ? tiles : pairs);
    return launch_chained(grouped_wgrad_kernel<F32>, dim3(clusters * 2 * split), kWgThreads, wgrad_smem(a.groups),
                          2 * split, s, maps, a);
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
        return launch_group_status(M_sizes_dev, num_groups, status_dev, s) == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA;
    }
    int sms = 0;
    if (device_sm_count(&sms) != 0 || sms < 1) return W4A16_ERR_CUDA;
    GroupWgradArgs a = {};
    a.m_sizes = M_sizes_dev, a.status = status_dev, a.err = device_error_word(), a.dw = dW;
    if (!a.err) return W4A16_ERR_CUDA;
    a.M = M_total, a.N = N, a.K = K, a.groups = num_groups;
    a.n_tiles = ceil_div(N, kSide), a.k_tiles = ceil_div(K, kSide);
    const cudaError_t e = dw_bytes == 4 ? launch_grouped_wgrad<true>(a, dY, X, sms, s)
                                        : launch_grouped_wgrad<false>(a, dY, X, sms, s);
    return e == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA;
}

W4A16_STALL_ENTRY(w4a16_test_stall_wgrad)
