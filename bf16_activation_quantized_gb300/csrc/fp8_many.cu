// fp8_many.cu -- many rows: the products of fp8_gemm.cu with the rows of x along M.
//
// A tile is 128 rows of x by 256 output columns.  A block's sum (4 MMAs of K = 32)
// lands in one of two buffers of tensor memory; eight warps read it and add it to their
// sums in registers, in fp32, while the next block's MMAs run.  A lane holds one row of
// x and 128 columns of one block of the weights, so a block's scale is one number a
// lane, the product of its row's and the weights'.
//
// PAIR: two CTAs share a tile of 256 rows; each loads its rows of x and half of the
// weights, which the pair's MMAs (cta_group::2) read from both.  That halves what an SM
// has to fetch of the weights.
//
// With few tiles `split` CTAs (a cluster) share one, each a run of the blocks that are
// summed over; the parts stand in shared memory and are added in the order of the CTAs.
//
// A tile's rounded sums go through shared memory to two warps that store them while the
// next tile's blocks are added; the last tile's are stored by the adding warps too.
//
// What bounds it: a block takes 740 cycles in the kernel, where its MMAs take 512 and its loads
// from tensor memory and FMAs 360 by themselves, 570 with the handshakes over two buffers
// (tensor memory holds no third).  wgrad.cu brings as much to an SM, 32 KB, for MMAs as long (64
// bytes a clock would be needed to hide it) and takes 0.32 us a stage where this kernel takes 0.42, a
// tile's end included in both: the loads set three quarters of a block's time, the cause of
// the last is not known.  Sixteen adding warps, packed FMAs and MMAs of 128
// columns were slower (279, 320 and 278 us where this had 238, 273 and 238).  4096 x 8192 x
// 8192: 187 us, 2.9 PFLOP/s (without pairs 236); 2858 x 19456 x 2560: 113 us.
//
// Warps: 0 copies (TMA) the tiles, 1 issues the MMAs, 2 and 3 store, 4 to 11 add.
#include "async.cuh"
#include "common.cuh"
#include "fp8.cuh"
#include "groups.cuh"
#include "internal.h"
#include "launch.cuh"
#include "lora.cuh"
#include "stall.cuh"
#include "tc05.cuh"

namespace w4a16 {

namespace {

constexpr int kManyThreads = 384, kAddWarp0 = 4, kAddWarps = 8;
// Registers a thread of the first four warps and of the adding ones: the launch's
// (168 x 384) are what the two shares draw on.
constexpr int kRegsIn = 72, kRegsAdd = 216;
constexpr int kSumBytes = 128 * 256 * 4;           // a tile's fp32 sums
static_assert(128 * kRegsIn + 256 * kRegsAdd <= 168 * kManyThreads, "registers");

constexpr int kRows = 128, kCols = 256;
constexpr int kTile = kFp8Block * kFp8Block;       // bytes of 128 rows of x, of 128 columns' weights
constexpr int kAhead = 4;                          // blocks whose scales are fetched ahead

template <bool PAIR>
struct ManyShape {
    static constexpr int kStage = PAIR ? 2 * kTile : 3 * kTile;
    static constexpr int kStages = PAIR ? 4 : 3;
    static constexpr int kOffStore = kStages * kStage;                       // a tile's results: rows of 512 bytes
    static_assert(kSumBytes <= kOffStore, "a tile's sums lie over the ring");
    static constexpr int kOffBar = kOffStore + kRows * kCols * 2;
    static constexpr int kOffTab = kOffBar + (2 * kStages + 7) * 8 + 8;
    static_assert(kOffTab + 2 * (kMaxGroups + 1) * 4 + 1024 <= kTensorMaxSmem - 256, "shared memory");
    static size_t smem(int groups, bool grouped) { return kOffTab + (grouped ? 2 * (groups + 1) * 4 : 0) + 1024; }
};

struct ManyTile {
    int group, tile, row0, rows;                   // rows: of this CTA, none or negative past the group's end
};
template <bool PAIR>
__device__ __forceinline__ bool many_tile(const Fp8Args &a, const int *tab_rows, const int *tab_tiles, int id, int part,
                                          ManyTile &t) {
    int first_row = 0, rows = a.M, r = id;
    t.group = 0;
    if (a.m_sizes) {
        if (id >= tab_tiles[a.groups]) return false;
        int lo = 0, hi = a.groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tab_tiles[mid] <= id) lo = mid; else hi = mid;
        }
        t.group = lo;
        r = id - tab_tiles[lo];
        first_row = tab_rows[lo], rows = tab_rows[lo + 1] - first_row;
    }
    const int n = row_tiles(rows, (PAIR ? 2 : 1) * kRows);
    if (r >= n * a.out_tiles) return false;
    int tt;
    banded(r, n, a.out_tiles, tt, t.tile);
    const int at = tt * (PAIR ? 2 : 1) * kRows;
    t.row0 = first_row + at + part * kRows;
    t.rows = min(kRows, rows - at - part * kRows);
    return true;
}

template <int N>
__device__ __forceinline__ void load_sums(uint32_t addr, uint32_t (&v)[N]) {
    if constexpr (N == 16) tc_ld_32x32b_x16(addr, v); else tc_ld_32x32b_x32(addr, v);
}

// volatile: issued where it is written, so that a value fetched ahead is not fetched next
// to its use.
__device__ __forceinline__ float fetch(const float *p) {
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

// A tile's sums in shared memory: pieces of 16 bytes placed so that eight rows' meet in no bank.
__device__ __forceinline__ float *sum_at(unsigned char *smem, int row, int piece) {
    return reinterpret_cast<float *>(smem) + row * kCols + 4 * (piece ^ (row & 7));
}

// One warp: rows first, first + SPLIT * warps, ... of a tile that SPLIT CTAs share, eight
// columns a lane.
template <int SPLIT>
__device__ __forceinline__ void join_rows(const Fp8Args &a, const ManyTile &t, unsigned char *smem, int first, int lost) {
    constexpr int kParts = SPLIT < 4 ? SPLIT : 4;
    const int lane = threadIdx.x % 32, col = t.tile * kCols + 8 * lane;
    for (int r = first; r < t.rows; r += SPLIT * (kManyThreads / 32)) {
        float s[8];
        #pragma unroll
        for (int k0 = 0; k0 < SPLIT; k0 += kParts) {
            float4 v[kParts][2];
            #pragma unroll
            for (int k = 0; k < kParts; ++k)
                #pragma unroll
                for (int h = 0; h < 2; ++h) v[k][h] = ld_cluster4(sum_at(smem, r, 2 * lane + h), k0 + k);
            #pragma unroll
            for (int k = 0; k < kParts; ++k)
                #pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float u[4] = {v[k][h].x, v[k][h].y, v[k][h].z, v[k][h].w};
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) s[4 * h + e] = k0 + k == 0 ? u[e] : s[4 * h + e] + u[e];
                }
        }
        if (lost)
            #pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = __int_as_float(0x7fffffff);
        uint16_t *y = a.y + (long long)(t.row0 + r) * a.out + col;
        store_cols8(y, a.out - col, a.vec, make_uint4(pack_bf16x2_rn(s[0], s[1]), pack_bf16x2_rn(s[2], s[3]),
                                                      pack_bf16x2_rn(s[4], s[5]), pack_bf16x2_rn(s[6], s[7])));
    }
}

// One warp: rows first, first + step, ... of a tile from shared memory, a row of 512 bytes
// at a time.
__device__ __forceinline__ void store_rows(const Fp8Args &a, const ManyTile &t, const unsigned char *store, int first,
                                           int step, bool lost) {
    constexpr int kAtOnce = 8;
    const int lane = threadIdx.x % 32, col = t.tile * kCols + 8 * lane;
    uint16_t *y = a.y + (long long)t.row0 * a.out + col;
    #pragma unroll 1
    for (int r0 = first; r0 < t.rows; r0 += kAtOnce * step) {
        uint4 v[kAtOnce];
        #pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int r = (r0 + j * step) % kRows;
            v[j] = *reinterpret_cast<const uint4 *>(store + r * 512 + ((lane ^ (r & 7)) << 4));
            // a wait that ran out: this tile and the CTA's later ones are NaN
            if (lost) v[j] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
        }
        #pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (r0 + j * step < t.rows) store_cols8(y + (long long)(r0 + j * step) * a.out, a.out - col, a.vec, v[j]);
    }
}

template <bool TRANS, bool PAIR>
__global__ void __launch_bounds__(kManyThreads, 1)
fp8_many_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                const Fp8Args a) {
    using S = ManyShape<PAIR>;
    constexpr int NS = S::kStages;
    extern __shared__ unsigned char s_raw[];
    unsigned char *smem = s_raw + (-smem_u32(s_raw) & 1023);
    __shared__ int s_abort;
    __shared__ uint32_t s_tmem;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, part = PAIR ? cluster_rank() : 0;
    const int split = PAIR ? 1 : cluster_size(), share = PAIR ? 0 : cluster_rank();
    const int b0 = int((long long)a.blocks * share / split), b1 = int((long long)a.blocks * (share + 1) / split);
    const uint32_t ring = smem_u32(smem), full = ring + S::kOffBar, empty = full + 8 * NS;
    const uint32_t dfull = empty + 8 * NS, dempty = dfull + 16, sfull = dempty + 16, sempty = sfull + 8, drained = sempty + 8;
    int *tab_rows = reinterpret_cast<int *>(smem + S::kOffTab), *tab_tiles = tab_rows + a.groups + 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, 1);
        for (int i = 0; i < 2; ++i) mbar_init(dfull + 8 * i, 1), mbar_init(dempty + 8 * i, (PAIR ? 2 : 1) * kAddWarps);
        mbar_init(sfull, kAddWarps), mbar_init(sempty, 2), mbar_init(drained, 1);
        s_abort = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) tma_prefetch_desc(&tmap_x), tma_prefetch_desc(&tmap_w);
    if (warp == 1) {
        if (PAIR) {
            tc_alloc_pair(smem_u32(&s_tmem), 2 * kCols);
        } else {
            tc_alloc(smem_u32(&s_tmem), 2 * kCols);
            tc_relinquish();
        }
    }
    pdl_wait();
    pdl_launch_dependents();
    if (a.m_sizes && warp == 0)
        scan_groups(a.m_sizes, a.groups, a.M, (PAIR ? 2 : 1) * kRows, a.out_tiles, tab_rows, tab_tiles,
                    blockIdx.x == 0 ? a.status : nullptr);
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_arrive(), cluster_wait();          // the other CTA's barriers stand
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    volatile int *abort_flag = &s_abort;
    const int per = PAIR ? 2 : split, id0 = int(blockIdx.x) / per, step = int(gridDim.x) / per;
    ManyTile t;
    if (warp < kAddWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIn));
        bool lost = false;
        int i = 0;
        if (warp == 0) {
            for (int id = id0; !lost && many_tile<PAIR>(a, tab_rows, tab_tiles, id, part, t); id += step)
                for (int b = b0; b < b1; ++b, ++i) {
                    const int s = i % NS;
                    const bool ok = i < NS || mbar_wait(empty + 8 * s, (i / NS - 1) & 1, abort_flag, a.err);
                    lost = !__all_sync(0xffffffffu, ok);
                    if (lost) break;
                    if (!stalled(i) && elect_one()) {
                        const uint32_t dst = ring + s * S::kStage;
                        const int at = b * kFp8Block, col = t.tile * kCols + part * kFp8Block;
                        if (PAIR) {
                            const uint32_t bar = cluster_address(full + 8 * s, 0);
                            if (part == 0) mbar_arrive_expect_tx(full + 8 * s, 2 * S::kStage);
                            tma_load_2d_pair(dst, &tmap_x, at, t.row0, bar);
                            tma_load_3d_pair(dst + kTile, &tmap_w, TRANS ? col : at, TRANS ? at : col, t.group, bar);
                        } else {
                            mbar_arrive_expect_tx(full + 8 * s, S::kStage);
                            tma_load_2d(dst, &tmap_x, at, t.row0, full + 8 * s);
                            for (int h = 0; h < 2; ++h) {
                                const int c = col + h * kFp8Block;
                                tma_load_3d(dst + (1 + h) * kTile, &tmap_w, TRANS ? c : at, TRANS ? at : c, t.group, full + 8 * s);
                            }
                        }
                    }
                    __syncwarp();
                }
            // Every copy lands before the CTA ends (a pair's are counted in its even CTA).
            if (*abort_flag && part == 0)
                for (int u = i > NS ? i - NS : 0; u < i; ++u) drain_wait(full + 8 * (u % NS), (u / NS) & 1);
        } else if (warp == 1 && part == 0) {
            constexpr uint32_t idesc = tc_idesc_e4m3((PAIR ? 2 : 1) * kRows, kCols) | (TRANS ? kTcBMajorN : 0u);
            for (int id = id0; !lost && many_tile<PAIR>(a, tab_rows, tab_tiles, id, part, t); id += step)
                for (int b = b0; b < b1; ++b, ++i) {
                    const int s = i % NS, d = i & 1;
                    const bool ok = mbar_wait(full + 8 * s, (i / NS) & 1, abort_flag, a.err) &&
                                    (i < 2 || mbar_wait(dempty + 8 * d, (i / 2 - 1) & 1, abort_flag, a.err));
                    lost = !__all_sync(0xffffffffu, ok);
                    if (lost) break;
                    tc_fence_after();
                    const uint32_t xs = ring + s * S::kStage;
                    const uint64_t dx = tc_sdesc_sw128(xs);
                    const uint64_t dw = TRANS ? tc_sdesc_sw128_mn(xs + kTile, kTile) : tc_sdesc_sw128(xs + kTile);
                    if (elect_one()) {
                        #pragma unroll
                        for (int e = 0; e < 4; ++e) {     // 32 of the block's 128: 32 bytes along rows, 4096 down them
                            const uint64_t de = dw + (TRANS ? 256 : 2) * e;
                            if (PAIR) tc_mma_f8_ss_pair(tmem + d * kCols, dx + 2 * e, de, idesc, e > 0);
                            else tc_mma_f8_ss(tmem + d * kCols, dx + 2 * e, de, idesc, e > 0);
                        }
                        if (PAIR) tc_commit_pair(empty + 8 * s, 3), tc_commit_pair(dfull + 8 * d, 3);
                        else tc_commit(empty + 8 * s), tc_commit(dfull + 8 * d);
                    }
                    __syncwarp();
                }
            if (elect_one()) {
                if (PAIR) tc_commit_pair(drained, 3);
                else tc_commit(drained);
            }
            __syncwarp();
            drain_wait(drained, 0);
        } else if (warp >= 2 && split == 1) {
            for (int id = id0; many_tile<PAIR>(a, tab_rows, tab_tiles, id, part, t); ++i) {
                const ManyTile now = t;
                id += step;
                const bool last = !many_tile<PAIR>(a, tab_rows, tab_tiles, id, part, t);
                lost = lost || !__all_sync(0xffffffffu, mbar_wait(sfull, i & 1, abort_flag, a.err));
                store_rows(a, now, smem + S::kOffStore, warp - 2, last ? 2 + kAddWarps : 2, lost);
                __syncwarp();
                if (lane == 0) mbar_arrive(sempty);
                if (last) break;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsAdd));
        const int sub = warp % 4, half = (warp - kAddWarp0) / 4;
        const uint32_t from = tmem + (uint32_t(32 * sub) << 16) + half * kFp8Block;
        const uint32_t done = PAIR ? cluster_address(dempty, 0) : dempty;
        const int row = 32 * sub + lane;
        // This lane's scales of x and of the weights, fetched kAhead blocks before their use.
        float fx[kAhead], fw[kAhead];
        const float *xs = nullptr, *ws = nullptr;
        // Rows past the tile's and columns past the last are not stored: any scale does.
        auto enter = [&]() {
            const int wt = min(2 * t.tile + half, (a.out - 1) / kFp8Block);
            xs = a.xs + (long long)b0 * a.M + min(t.row0 + row, a.M - 1);
            ws = a.ws + t.group * a.ws_group + (long long)wt * a.ws_tile + (long long)b0 * a.ws_block;
            #pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (b0 + u < b1) fx[u] = fetch(xs), fw[u] = fetch(ws);
                xs += a.M, ws += a.ws_block;
            }
        };
        int i = 0, tiles = 0;
        bool lost = false, more = many_tile<PAIR>(a, tab_rows, tab_tiles, id0, part, t);
        if (more) enter();
        ManyTile now = t;
        for (int id = id0; more;) {
            now = t;
            float acc[kFp8Block];
            #pragma unroll
            for (int j = 0; j < kFp8Block; ++j) acc[j] = 0.f;
            for (int b = b0; b < b1 && !lost; b += kAhead) {
                #pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (b + u >= b1 || lost) break;
                    const int d = i & 1;
                    const float scale = fx[u] * fw[u];
                    if (b + u + kAhead < b1) fx[u] = fetch(xs), fw[u] = fetch(ws);
                    xs += a.M, ws += a.ws_block;
                    lost = !__all_sync(0xffffffffu, mbar_wait(dfull + 8 * d, (i / 2) & 1, abort_flag, a.err));
                    if (lost) break;
                    ++i;
                    tc_fence_after();
                    // A chunk's load is under way while the one before it is added.
                    constexpr int kChunk = 16, kChunks = kFp8Block / kChunk;
                    uint32_t v[2][kChunk];
                    load_sums(from + d * kCols, v[0]);
                    #pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        tc_wait_ld_of(v[c & 1]);
                        if (c + 1 < kChunks) {
                            load_sums(from + d * kCols + kChunk * (c + 1), v[(c + 1) & 1]);
                        } else {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) {
                                if (PAIR) mbar_arrive_cluster(done + 8 * d);
                                else mbar_arrive(done + 8 * d);
                            }
                        }
                        #pragma unroll
                        for (int e = 0; e < kChunk; ++e)
                            acc[kChunk * c + e] = fmaf(__uint_as_float(v[c & 1][e]), scale, acc[kChunk * c + e]);
                    }
                }
            }
            // The next tile's first scales come while this one is rounded.
            id += step;
            more = many_tile<PAIR>(a, tab_rows, tab_tiles, id, part, t);
            if (more) enter();
            if (!PAIR && split > 1) {
                // over the ring, whose tiles this one's last MMAs have read; a cluster has one tile
                // (where a wait ran out the join finds the flag)
                #pragma unroll
                for (int q = 0; q < kFp8Block / 4; ++q)
                    *reinterpret_cast<float4 *>(sum_at(smem, row, half * (kFp8Block / 4) + q)) =
                        make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
                break;
            }
            // This row's 128 columns to the store warps, in pieces of 16 bytes placed so that
            // eight rows' meet in no bank.  Where a wait ran out they write NaN.
            if (tiles > 0 && !lost)
                lost = !__all_sync(0xffffffffu, mbar_wait(sempty, (tiles - 1) & 1, abort_flag, a.err));
            ++tiles;
            if (lost) continue;
            #pragma unroll
            for (int q = 0; q < kFp8Block / 8; ++q) {
                uint32_t p[4];
                #pragma unroll
                for (int j = 0; j < 4; ++j) p[j] = pack_bf16x2_rn(acc[8 * q + 2 * j], acc[8 * q + 2 * j + 1]);
                *reinterpret_cast<uint4 *>(smem + S::kOffStore + row * 512 + (((half * 16 + q) ^ (row & 7)) << 4)) =
                    make_uint4(p[0], p[1], p[2], p[3]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(sfull);
        }
        // Nothing is left to add: these warps help to store the last tile.
        if (split == 1 && tiles > 0) {
            lost = lost || !__all_sync(0xffffffffu, mbar_wait(sfull, (tiles - 1) & 1, abort_flag, a.err));
            store_rows(a, now, smem + S::kOffStore, warp - kAddWarp0 + 2, 2 + kAddWarps, lost);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_arrive(), cluster_wait();          // the pair's MMAs have read both CTAs' memory
    if (!PAIR && split > 1) {
        cluster_arrive();
        cluster_wait();
        int lost = 0;                                    // a wait ran out: copies may have landed on the sums
        #pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
            if (k < split) lost |= ld_cluster1(&s_abort, k);
        if (many_tile<PAIR>(a, tab_rows, tab_tiles, id0, part, t)) {
            const int first = share + split * warp;
            if (split == 2) join_rows<2>(a, t, smem, first, lost);
            else if (split == 4) join_rows<4>(a, t, smem, first, lost);
            else join_rows<8>(a, t, smem, first, lost);
        }
        cluster_arrive();                                // the others have read this CTA's part
        cluster_wait();
    }
    tc_fence_after();
    if (warp == 1) {
        if (PAIR) tc_dealloc_pair(tmem, 2 * kCols);
        else tc_dealloc(tmem, 2 * kCols);
    }
}

template <bool TRANS, bool PAIR>
cudaError_t launch_many_form(const Fp8Plan &p, const Fp8Args &a, const CUtensorMap &tx, const CUtensorMap &tw,
                             cudaStream_t s) {
    const cudaError_t e = allow_smem<fp8_many_kernel<TRANS, PAIR>>(kTensorMaxSmem - 256);
    if (e != cudaSuccess) return e;
    return launch_chained(fp8_many_kernel<TRANS, PAIR>, dim3(p.ctas), kManyThreads,
                          ManyShape<PAIR>::smem(a.groups, a.m_sizes != nullptr), p.split, s, tx, tw, a);
}

}  // namespace

cudaError_t launch_fp8_many(const Fp8Plan &p, const Fp8Args &a, const CUtensorMap &tx, const CUtensorMap &tw,
                            bool trans, cudaStream_t s) {
    if (p.pair) return trans ? launch_many_form<true, true>(p, a, tx, tw, s) : launch_many_form<false, true>(p, a, tx, tw, s);
    return trans ? launch_many_form<true, false>(p, a, tx, tw, s) : launch_many_form<false, false>(p, a, tx, tw, s);
}

}  // namespace w4a16

W4A16_STALL_ENTRY(w4a16_test_stall_many)
