// fp8_gemm.cu -- few rows: products of e4m3 rows with e4m3 weights, a scale for 128 elements of a
// row and for a block of 128 x 128 of the weights:
//
//   Y[m][n]  = sum_b xs[b][m] ws[n / 128][b] sum_{k in block b} X[m][k] W[n][k]
//   dX[m][k] = sum_b ds[b][m] ws[b][k / 128] sum_{n in block b} dY[m][n] W[n][k]
//
// plain and by group, the second (TRANS) from the weights as they lie: a tile of W is
// the same box of 128 x 128 bytes in both, whose rows are the tensor core's M in the
// first and its K in the second.
//
// The weights are the MMA's A (M = 128 output columns), rows of x its N: any number of
// them down to 16 makes a tile, so one kernel serves a single token and a long prefill
// and a group's last tile multiplies what it holds.  A block's sum (4 MMAs of K = 32)
// lands in one of several buffers of tensor memory; eight warps read it, multiply by
// both scales and add in registers, in fp32, while the next block's MMAs run.
//
// With few tiles `split` CTAs (a cluster) share one, each a run of the blocks that are
// summed over; the parts stand in shared memory and are added in the order of the CTAs.
//
// What bounds it: memory, once enough CTAs run (a CTA takes a block of 128 x 128 weights
// in 0.2 to 0.36 us).  128 rows of 128 groups, 2048 x 4096: 103 us, 6.6 TB/s, 0.97 of the
// measured copy bandwidth.  One row, 8192 x 8192: 13.3 us, of which the weights take 9.5;
// the first bytes come 2 us after the launch, a cluster's sums and the exit take 2.
//
// Warps: 0 copies (TMA) the tiles, 1 and 2 issue the MMAs of every second block each (one
// warp takes 480 cycles for a block's waits, four MMAs and two commits), 3 forms the
// products of the scales, 4 to 11 add.
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

constexpr int kFp8Threads = 384, kAddWarp0 = 4, kAddWarps = 8;
constexpr int kWTile = kFp8Block * kFp8Block;      // bytes of a tile of W
constexpr int kSlots = 4;                          // blocks whose sums and scales are held

template <int BT>
struct Fp8Shape {
    static constexpr int kTmem = kSlots * BT;
    static constexpr int kChunk = BT == 128 ? 32 : BT == 32 ? 16 : 8;    // columns a load from tensor memory brings
    static constexpr int kChunks = BT / 2 / kChunk;            // per warp
    static constexpr int kAhead = 4;            // blocks whose scales a warp fetches ahead
    static constexpr int kOccupancy = BT <= 64 ? 2 : 1;
};

struct Fp8Smem {
    int stage, off_scale, off_store, off_bar, off_tab, total;
};
__host__ __device__ inline Fp8Smem fp8_smem(int size, int bt, int stages, int groups) {
    Fp8Smem L;
    L.stage = kWTile + bt * kFp8Block;
    L.off_scale = stages * L.stage;
    L.off_store = L.off_scale + kSlots * size * 4;
    L.off_bar = L.off_store + kAddWarps * 32 * 16 * 2;
    L.off_tab = L.off_bar + (2 * stages + 2 * kSlots + 1) * 8 + 16;
    L.total = (L.off_tab + 2 * (groups + 1) * 4 + 15) & ~15;
    return L;
}

struct Fp8Tile {
    int group, tile, row0, rows;      // output tile, first row of x, rows
};

// Output tiles fastest, so that CTAs that run together share rows of x.  A group's rows
// are cut evenly, in steps of 16.
__device__ __forceinline__ bool fp8_tile(const Fp8Args &a, const int *tab_rows, const int *tab_tiles, int id,
                                         Fp8Tile &t) {
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
    const int n = row_tiles(rows, a.bt), tt = r / a.out_tiles;
    if (tt >= n) return false;
    const int each = ((rows + n - 1) / n + 15) & ~15;
    t.tile = r - tt * a.out_tiles;
    t.row0 = first_row + tt * each;
    t.rows = min(each, rows - tt * each);
    return true;
}

// volatile: issued where it is written, so that a value fetched ahead is not fetched next
// to its use.
__device__ __forceinline__ float fetch(const float *p) {
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

template <int N>
__device__ __forceinline__ void load_sums(uint32_t addr, uint32_t (&v)[N]) {
    if constexpr (N == 8) tc_ld_32x32b_x8(addr, v);
    else if constexpr (N == 16) tc_ld_32x32b_x16(addr, v);
    else tc_ld_32x32b_x32(addr, v);
}

// One warp: rows first, first + SPLIT * warps, ... of a tile that SPLIT CTAs share, four
// columns a lane; several parts are under way at once, a row's are added in the order of
// the CTAs.
template <int SPLIT>
__device__ __forceinline__ void join_rows(const Fp8Args &a, const Fp8Tile &t, const float *join, int first, int lost) {
    constexpr int kParts = SPLIT < 4 ? SPLIT : 4, kAtOnce = 4 / kParts, kStep = SPLIT * (kFp8Threads / 32);
    const int lane = threadIdx.x % 32, col0 = t.tile * kFp8Block + 4 * lane, cols = a.out - col0;
    for (int r0 = first; r0 < t.rows; r0 += kAtOnce * kStep) {
        float4 s[kAtOnce];
        #pragma unroll
        for (int k0 = 0; k0 < SPLIT; k0 += kParts) {
            float4 v[kAtOnce][kParts];
            #pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
                #pragma unroll
                for (int k = 0; k < kParts; ++k)
                    if (r0 + j * kStep < t.rows)
                        v[j][k] = ld_cluster4(join + (r0 + j * kStep) * kFp8Block + 4 * lane, k0 + k);
            #pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
                #pragma unroll
                for (int k = 0; k < kParts; ++k) {
                    if (k0 + k == 0) s[j] = v[j][0];
                    else s[j].x += v[j][k].x, s[j].y += v[j][k].y, s[j].z += v[j][k].z, s[j].w += v[j][k].w;
                }
        }
        #pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            if (r0 + j * kStep >= t.rows) break;
            if (lost) s[j].x = s[j].y = s[j].z = s[j].w = __int_as_float(0x7fffffff);
            uint16_t *y = a.y + (long long)(t.row0 + r0 + j * kStep) * a.out + col0;
            const uint32_t lo = pack_bf16x2_rn(s[j].x, s[j].y), hi = pack_bf16x2_rn(s[j].z, s[j].w);
            if (a.vec) {
                if (cols > 0) *reinterpret_cast<uint2 *>(y) = make_uint2(lo, hi);
            } else {
                if (cols > 0) y[0] = uint16_t(lo);
                if (cols > 1) y[1] = uint16_t(lo >> 16);
                if (cols > 2) y[2] = uint16_t(hi);
                if (cols > 3) y[3] = uint16_t(hi >> 16);
            }
        }
    }
}

template <int BT, bool TRANS>
__global__ void __launch_bounds__(kFp8Threads, Fp8Shape<BT>::kOccupancy)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                const Fp8Args a) {
    using S = Fp8Shape<BT>;
    extern __shared__ unsigned char s_raw[];
    unsigned char *smem = s_raw + (-smem_u32(s_raw) & 1023);
    const int split = cluster_size(), part = cluster_rank();
    const int NS = a.stages;
    const Fp8Smem L = fp8_smem(BT, a.bt, NS, a.groups);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t ring = smem_u32(smem), full = smem_u32(smem + L.off_bar), empty = full + 8 * NS;
    const uint32_t dfull = empty + 8 * NS, dempty = dfull + 8 * kSlots, drained = dempty + 8 * kSlots;
    float *scales = reinterpret_cast<float *>(smem + L.off_scale);
    // fp32 sums of a tile that several CTAs share, over the ring: whoever has waited for a
    // tile's last MMAs finds its copies landed and read.
    float *join = reinterpret_cast<float *>(smem);
    int *tab_rows = reinterpret_cast<int *>(smem + L.off_tab), *tab_tiles = tab_rows + a.groups + 1;
    __shared__ int s_abort;
    __shared__ uint32_t s_tmem;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, 1);
        for (int i = 0; i < kSlots; ++i)                   // full: the MMAs' end and the scales
            mbar_init(dfull + 8 * i, 2), mbar_init(dempty + 8 * i, kAddWarps);
        mbar_init(drained, 2);
        s_abort = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) tma_prefetch_desc(&tmap_x), tma_prefetch_desc(&tmap_w);
    if (warp == 1) {
        tc_alloc(smem_u32(&s_tmem), S::kTmem);
        tc_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    volatile int *abort_flag = &s_abort;
    const int b0 = int((long long)a.blocks * part / split), b1 = int((long long)a.blocks * (part + 1) / split);
    const uint32_t stage_bytes = kWTile + a.bt * kFp8Block;

    // The first stages of weights that nothing on the stream still writes start at once;
    // others are brought to L2, where a later write replaces them.
    int early = 0;
    if (warp == 0 && !a.m_sizes) {
        const int tile = (int(blockIdx.x) / split) % a.out_tiles, n = min(NS, b1 - b0);
        early = a.resident ? n : 0;
        if (elect_one())
            for (int i = 0; i < n; ++i) {
                const int b = (b0 + i) * kFp8Block, o = tile * kFp8Block, x = TRANS ? o : b, y = TRANS ? b : o;
                if (a.resident) {
                    mbar_arrive_expect_tx(full + 8 * i, stage_bytes);
                    tma_load_3d(ring + i * L.stage, &tmap_w, x, y, 0, full + 8 * i);
                } else {
                    tma_prefetch_3d(&tmap_w, x, y, 0);
                }
            }
        __syncwarp();
    }
    pdl_wait();
    pdl_launch_dependents();
    if (a.m_sizes) {
        if (warp == 1)
            scan_groups(a.m_sizes, a.groups, a.M, a.bt, a.out_tiles, tab_rows, tab_tiles, blockIdx.x == 0 ? a.status : nullptr);
        __syncthreads();
    }
    const int id0 = int(blockIdx.x) / split, step = int(gridDim.x) / split;
    Fp8Tile t;

    if (warp == 0) {
        int i = 0, s = 0;
        uint32_t phase = 1;                              // of the slot's release (first lap: none)
        bool lost = false;
        for (int id = id0; !lost && fp8_tile(a, tab_rows, tab_tiles, id, t); id += step)
            for (int b = b0; b < b1; ++b, ++i) {
                const bool ok = i < NS || mbar_wait(empty + 8 * s, phase, abort_flag, a.err);
                lost = !__all_sync(0xffffffffu, ok);
                if (lost) break;
                if (!stalled(i) && elect_one()) {
                    const uint32_t dst = ring + s * L.stage;
                    if (i >= early) {
                        mbar_arrive_expect_tx(full + 8 * s, stage_bytes);
                        tma_load_3d(dst, &tmap_w, (TRANS ? t.tile : b) * kFp8Block, (TRANS ? b : t.tile) * kFp8Block,
                                    t.group, full + 8 * s);
                    }
                    tma_load_2d(dst + kWTile, &tmap_x, b * kFp8Block, t.row0, full + 8 * s);
                }
                __syncwarp();
                if (++s == NS) s = 0, phase ^= 1;
            }
        // Every copy lands before the CTA ends.
        if (*abort_flag)
            for (int u = i > NS ? i - NS : 0; u < i; ++u) drain_wait(full + 8 * (u % NS), (u / NS) & 1);
    } else if (warp <= 2) {
        // The slot is a counter: a division by the ring's depth would cost more than a block's MMAs.
        int i = 0, s = warp - 1;
        uint32_t phase = 0;
        bool lost = false;
        for (int id = id0; !lost && fp8_tile(a, tab_rows, tab_tiles, id, t); id += step) {
            const uint32_t idesc = tc_idesc_e4m3(kFp8Block, (t.rows + 15) & ~15) | (TRANS ? kTcAMajorM : 0u);
            for (int b = b0; b < b1; ++b, ++i) {
                if ((i & 1) != warp - 1) continue;
                const int d = i % kSlots;
                // The sums' slot first: with an odd ring this warp meets a ring slot every second lap,
                // and its parity would also fit two laps before.  The block that had the sums' slot
                // has been added, so the ring slot's lap before, kSlots blocks back at least, is over.
                bool ok = i < kSlots || mbar_wait(dempty + 8 * d, (i / kSlots - 1) & 1, abort_flag, a.err);
                ok = ok && mbar_wait(full + 8 * s, phase, abort_flag, a.err);
                lost = !__all_sync(0xffffffffu, ok);
                if (lost) break;
                tc_fence_after();
                const uint32_t ws = ring + s * L.stage;
                const uint64_t dx = tc_sdesc_sw128(ws + kWTile);
                const uint64_t dw = TRANS ? tc_sdesc_sw128_mn(ws, 1024) : tc_sdesc_sw128(ws);
                if (elect_one()) {
                    #pragma unroll
                    for (int e = 0; e < 4; ++e)       // 32 of the block's 128: 32 bytes along rows, 4096 down them
                        tc_mma_f8_ss(tmem + d * BT, dw + (TRANS ? 256 : 2) * e, dx + 2 * e, idesc, e > 0);
                    tc_commit(empty + 8 * s);
                    tc_commit(dfull + 8 * d);
                }
                __syncwarp();
                s += 2;
                if (s >= NS) s -= NS, phase ^= 1;
            }
        }
        if (elect_one()) tc_commit(drained);
        __syncwarp();
        drain_wait(drained, 0);
    } else if (warp < kAddWarp0) {
        // Products of the scales, fetched kAhead blocks before their use.
        constexpr int kEach = BT < 32 ? 1 : BT / 32, kAhead = S::kAhead;
        int i = 0;
        bool lost = false;
        for (int id = id0; !lost && fp8_tile(a, tab_rows, tab_tiles, id, t); id += step) {
            const float *ws = a.ws + t.group * a.ws_group + (long long)t.tile * a.ws_tile + (long long)b0 * a.ws_block;
            const float *xs = a.xs + (long long)b0 * a.M + t.row0;
            int r[kEach];
            #pragma unroll
            for (int j = 0; j < kEach; ++j) r[j] = min(lane + 32 * j, t.rows - 1);   // no row's scale: never used
            float v[kAhead][kEach], w[kAhead];
            auto load = [&](int u) {
                w[u] = fetch(ws);
                #pragma unroll
                for (int j = 0; j < kEach; ++j) v[u][j] = fetch(xs + r[j]);
            };
            #pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (b0 + u < b1) load(u);
                ws += a.ws_block, xs += a.M;
            }
            for (int b = b0; b < b1 && !lost; b += kAhead) {
                #pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (b + u >= b1) break;
                    const int k = i + b + u - b0, s = k % kSlots;
                    const bool ok = k < kSlots || mbar_wait(dempty + 8 * s, (k / kSlots - 1) & 1, abort_flag, a.err);
                    lost = !__all_sync(0xffffffffu, ok);
                    if (lost) break;
                    #pragma unroll
                    for (int j = 0; j < kEach; ++j)
                        if (BT >= 32 || lane < BT) scales[s * BT + lane + 32 * j] = v[u][j] * w[u];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(dfull + 8 * s);
                    if (b + u + kAhead < b1) load(u);
                    ws += a.ws_block, xs += a.M;
                }
            }
            i += b1 - b0;
        }
    } else {
        // Lane l of a warp holds output column 32 (warp % 4) + l of the tile, for half of
        // its rows of x.
        const int sub = warp % 4, half = (warp - kAddWarp0) / 4;
        const uint32_t lanes = tmem + (uint32_t(32 * sub) << 16);
        uint16_t *store = reinterpret_cast<uint16_t *>(smem + L.off_store) + (warp - kAddWarp0) * 32 * 16;
        int i = 0;
        bool lost = false;
        for (int id = id0; fp8_tile(a, tab_rows, tab_tiles, id, t); id += step) {
            const int c0 = half * ((((t.rows + 1) / 2) + S::kChunk - 1) / S::kChunk * S::kChunk);
            const int left = (half ? t.rows : min(t.rows, (((t.rows + 1) / 2) + S::kChunk - 1) / S::kChunk * S::kChunk)) - c0;
            float acc[BT / 2];
            #pragma unroll
            for (int j = 0; j < BT / 2; ++j) acc[j] = 0.f;
            for (int b = b0; b < b1 && !lost; ++b, ++i) {
                const int d = i % kSlots;
                lost = !__all_sync(0xffffffffu, mbar_wait(dfull + 8 * d, (i / kSlots) & 1, abort_flag, a.err));
                if (lost) break;
                tc_fence_after();
                const float *sc = scales + d * BT + c0;
                #pragma unroll
                for (int c = 0; c < S::kChunks; ++c) {
                    if (c * S::kChunk < left) {
                        uint32_t v[S::kChunk];
                        load_sums(lanes + d * BT + c0 + c * S::kChunk, v);
                        float4 f[S::kChunk / 4];
                        #pragma unroll
                        for (int e = 0; e < S::kChunk / 4; ++e)
                            f[e] = *reinterpret_cast<const float4 *>(sc + c * S::kChunk + 4 * e);
                        tc_wait_ld_of(v);
                        #pragma unroll
                        for (int e = 0; e < S::kChunk; e += 4) {
                            float *s = acc + c * S::kChunk + e;
                            s[0] = fmaf(__uint_as_float(v[e]), f[e / 4].x, s[0]);
                            s[1] = fmaf(__uint_as_float(v[e + 1]), f[e / 4].y, s[1]);
                            s[2] = fmaf(__uint_as_float(v[e + 2]), f[e / 4].z, s[2]);
                            s[3] = fmaf(__uint_as_float(v[e + 3]), f[e / 4].w, s[3]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(dempty + 8 * d);
            }
            // A wait that ran out: this tile and the CTA's later ones are NaN.
            if (lost) {
                #pragma unroll
                for (int j = 0; j < BT / 2; ++j) acc[j] = __int_as_float(0x7fffffff);
            }
            if (split > 1) {                             // a cluster has one tile
                #pragma unroll
                for (int j = 0; j < BT / 2; ++j)
                    if (j < left) join[(c0 + j) * kFp8Block + 32 * sub + lane] = acc[j];
                break;
            }
            const int col = t.tile * kFp8Block + 32 * sub;
            constexpr int kStoreCols = BT == 16 ? 8 : 16;
            #pragma unroll
            for (int c = 0; c < BT / 2; c += kStoreCols) {
                if (c < left) {
                    uint16_t *y = a.y + (long long)(t.row0 + c0 + c) * a.out + col;
                    if (a.vec) {
                        #pragma unroll
                        for (int e = 0; e < kStoreCols; e += 2) {
                            const uint32_t p = pack_bf16x2_rn(acc[c + e], acc[c + e + 1]);
                            store[e * 32 + lane] = uint16_t(p);
                            store[(e + 1) * 32 + lane] = uint16_t(p >> 16);
                        }
                        __syncwarp();
                        #pragma unroll
                        for (int k = 0; k < kStoreCols; k += 8) {
                            const int e = k + lane / 4, q = 8 * (lane % 4);
                            if (c + e < left && col + q < a.out)
                                *reinterpret_cast<uint4 *>(y + (long long)e * a.out + q) =
                                    *reinterpret_cast<const uint4 *>(store + e * 32 + q);
                        }
                    } else {
                        #pragma unroll
                        for (int e = 0; e < kStoreCols; ++e)
                            if (c + e < left && col + lane < a.out)
                                y[(long long)e * a.out + lane] =
                                    f32_to_bf16_rn(acc[c + e]);
                    }
                }
                __syncwarp();                            // tcgen05.ld takes the whole warp
            }
        }
    }
    if (split > 1) {
        // The tile's rows of x are shared out: this CTA adds the parts of rows part, part +
        // split, ..., a warp a row, four columns a lane, in the order of the CTAs.
        cluster_arrive();
        cluster_wait();
        if (fp8_tile(a, tab_rows, tab_tiles, id0, t)) {
            // Where a wait ran out, copies may have landed on the sums.
            int lost = 0;
            #pragma unroll
            for (int k = 0; k < kMaxCluster; ++k)
                if (k < split) lost |= ld_cluster1(&s_abort, k);
            const int first = part + split * warp;
            if (split == 2) join_rows<2>(a, t, join, first, lost);
            else if (split == 4) join_rows<4>(a, t, join, first, lost);
            else join_rows<8>(a, t, join, first, lost);
        }
        cluster_arrive();                                // the others have read this CTA's part
        cluster_wait();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tc_dealloc(tmem, S::kTmem);
}

static_assert(kMaxSplit == kMaxCluster, "CTAs that share a tile");

template <int BT, bool TRANS>
cudaError_t launch_size(const Fp8Plan &p, const Fp8Args &a, const CUtensorMap &tx, const CUtensorMap &tw, size_t smem,
                        cudaStream_t s) {
    cudaError_t e = allow_smem<fp8_gemm_kernel<BT, TRANS>>(kTensorMaxSmem - 256);
    if (e != cudaSuccess) return e;
    return launch_chained(fp8_gemm_kernel<BT, TRANS>, dim3(p.ctas), kFp8Threads, smem, p.split, s, tx, tw, a);
}

template <int BT>
cudaError_t launch_trans(const Fp8Plan &p, const Fp8Args &a, const CUtensorMap &tx, const CUtensorMap &tw, size_t smem,
                         bool trans, cudaStream_t s) {
    return trans ? launch_size<BT, true>(p, a, tx, tw, smem, s) : launch_size<BT, false>(p, a, tx, tw, smem, s);
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8Plan &p, Fp8Args a, const uint8_t *x, const uint8_t *w, int N, int K, bool trans,
                            cudaStream_t s) {
    CUtensorMap tx, tw;
    const cuuint64_t xdim[2] = {cuuint64_t(a.blocks) * kFp8Block, cuuint64_t(a.M)};
    const cuuint64_t xstride[1] = {xdim[0]};
    const cuuint32_t xbox[2] = {kFp8Block, cuuint32_t(p.bt)};
    cudaError_t e = encode_tensor_map(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, x, xdim, xstride, xbox,
                                      CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    const cuuint64_t wdim[3] = {cuuint64_t(K), cuuint64_t(N), cuuint64_t(a.groups)};
    const cuuint64_t wstride[2] = {cuuint64_t(K), cuuint64_t(N) * K};
    const cuuint32_t wbox[3] = {kFp8Block, kFp8Block, 1};
    e = encode_tensor_map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, w, wdim, wstride, wbox, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    a.bt = p.bt;
    if (p.size == 0) {
        a.out_tiles = ceil_div(a.out, 2 * kFp8Block);
        return launch_fp8_many(p, a, tx, tw, trans, s);
    }
    const int budget = (p.occupancy == 2 ? kSmemPerSm / 2 - kSmemReservedPerCta : kTensorMaxSmem) - 1024 - 256;
    const int rest = fp8_smem(p.size, p.bt, 0, a.groups).total + 64 * 16;
    a.stages = (budget - rest) / (kWTile + p.bt * kFp8Block);
    if (a.stages > 16) a.stages = 16;
    // An odd ring has to hold as many blocks as there are slots for sums (see the MMA warps).
    if (a.stages % 2 && a.stages < kSlots) --a.stages;
    if (a.stages < 2) return cudaErrorInvalidValue;
    const size_t smem = fp8_smem(p.size, p.bt, a.stages, a.groups).total + 1024;
    switch (p.size) {
        case 16: return launch_trans<16>(p, a, tx, tw, smem, trans, s);
        case 32: return launch_trans<32>(p, a, tx, tw, smem, trans, s);
        case 64: return launch_trans<64>(p, a, tx, tw, smem, trans, s);
        default: return launch_trans<128>(p, a, tx, tw, smem, trans, s);
    }
}

}  // namespace w4a16

W4A16_STALL_ENTRY(w4a16_test_stall_few)
