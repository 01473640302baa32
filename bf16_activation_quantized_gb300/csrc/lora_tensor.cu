// lora_tensor.cu -- adapters for many tokens, on the tensor cores.
//
// lora_down_kernel: partial sums of h = A x (or, with the weight read along its
// other axis, of B^T dy); lora_sum_kernel: h; lora_up_kernel: y = base + s B h (dx
// = dx_base + A^T g).  The formulas and the precision are in lora.cu.  The two
// products walk tiles of 128 sorted tokens of one adapter in steps of 128
// columns; the (tile, column step) pairs are cut into one even run per CTA, one
// CTA per SM, so every SM moves the same bytes whatever the adapters' sizes.  A
// run that covers part of a tile's input columns leaves its sum in a workspace
// slot (tile + CTA, unique along the walk), and a tile's slots are added in CTA
// order.  The three launches are chained: the second product's CTAs stream base
// and weights while the sums are made.
//
// In each CTA four producer warps gather rows of X (of base) and the weights
// with 16-byte asynchronous copies into a ring of stages, in the 128-byte
// swizzle that tcgen05.mma reads; one warp issues the MMAs; the other warps
// empty TMEM, and in the second kernel add base in shared memory and store
// whole 128-byte pieces of rows.  h enters the second product as three bf16 planes.
//
// What bounds them: HBM.  At rank 64 the legacy MMA pipe would need two thirds of
// the memory's time and left a 64-token mma.sync version waiting on MMA latency
// (78 us for 4096 tokens, 8192 x 8192); tcgen05 needs a tenth.
//
// lora_wgrad_kernel: dA = g^T X and dB = s dY^T h, with the tokens as the MMA's K.
// Rows of X or dY lie along M as they come; g and s h are kept with the tokens
// along K (the sums' kernel turns them, a few KB a tile).  wgrad_sum_kernel adds
// what several runs share.
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "w4a16.h"
#include "internal.h"
#include "launch.cuh"
#include "lora.cuh"
#include "tc05.cuh"

namespace w4a16 {
namespace {

constexpr int kEpiWarps = 8, kProducerWarps = 4, kMmaWarp = kEpiWarps + kProducerWarps;
constexpr int kEpiThreads = kEpiWarps * 32, kProducers = kProducerWarps * 32;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kTile = 128;             // tokens of a tile: the MMA's M
constexpr int kCols = 128;             // columns of a stage: two blocks of 64
constexpr int kBlock = kTile * 128;    // bytes of 128 rows x 64 columns
constexpr int kSmemMax = 226 * 1024;
constexpr int kTmemCols = 512;
constexpr int kPrefetch = 256 * 1024;  // bytes of X that a CTA prefetches
constexpr int kMaxRuns = 160;          // CTAs of the two products: one per SM (152)

// A wait that runs out ends the pipeline of its CTA: the abort flag is set, no warp
// takes a step after a wait of its own has failed (`lost`; a later phase's parity
// would no longer say anything), and the warps that store leave NaN in all that is
// left of the CTA's run.
//
// A test's build makes waits run out: from stage (or tile) g_stall_at of kernel
// g_stall_kernel on, the producers of every other CTA do not report theirs.
enum Stall { kStallDown = 1, kStallUp, kStallWgrad, kStallDownTile, kStallUpTile };
#ifdef W4A16_TEST_STALL
__device__ int g_stall_kernel, g_stall_at;
__device__ __forceinline__ bool stalled(int kernel, int at) {
    return kernel == g_stall_kernel && at >= g_stall_at && blockIdx.x % 2 == 0;
}
#else
__device__ __forceinline__ constexpr bool stalled(int, int) { return false; }
#endif

// All MMAs have ended: no CTA leaves, or gives its TMEM back, before.
__device__ __forceinline__ void drain_mmas(uint32_t bar) {
    if (elect_one()) tc_commit(bar);
    __syncwarp();
    drain_wait(bar, 0);
}

// Byte of piece p (16 bytes) of row `row` in a block of 128-byte rows.
__device__ __forceinline__ uint32_t sw128(int row, int p) { return uint32_t(row * 128 + ((p ^ (row & 7)) << 4)); }

// The walk: unit u = tile * per + step; CTA b of n takes units [run(b), run(b + 1)).
// (64-bit quotients take a few hundred cycles each: 32-bit ones where they do.)
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)(uint32_t(a) / uint32_t(b)) : a / b;
}
__device__ __forceinline__ long long run_start(long long units, int n, int b) { return quotient(units * b, n); }
// The CTA whose run holds unit u.
__device__ __forceinline__ int run_owner(long long units, int n, long long u) {
    return int(quotient((u + 1) * n - 1, units));
}
struct Walk {
    long long units;
    int per, ctas;          // steps of a tile; CTAs with a run
    long long u0, u1;       // this CTA's run
};
__device__ __forceinline__ Walk make_walk(int tiles, int per, int b, int ctas) {
    Walk w;
    w.units = (long long)tiles * per;
    w.per = per;
    w.ctas = int(w.units < ctas ? w.units : ctas);
    w.u0 = w.u1 = 0;
    if (b < w.ctas) w.u0 = run_start(w.units, w.ctas, b), w.u1 = run_start(w.units, w.ctas, b + 1);
    return w;
}

// Tiles of all adapters and, past those, of the tokens without one.  Every warp
// counts for itself.
struct TileCount {
    int with, without;
};
__device__ __forceinline__ TileCount count_tiles(const LoraArgs &p) {
    int tiles = 0, rows = 0;
    for (int a = threadIdx.x & 31; a < p.adapters; a += 32) {
        const int size = p.sizes[a];
        tiles += (size + kTile - 1) / kTile;
        rows += size;
    }
    tiles = __reduce_add_sync(0xffffffffu, tiles);
    rows = __reduce_add_sync(0xffffffffu, rows);
    return {tiles, (p.tokens - rows + kTile - 1) / kTile};
}

// Two tiles' tokens, filled by the first producer warp ahead of the others.
struct TileSlots {
    int rows[2][kTile];
    int info[2][3];         // adapter (-1: none), tokens, first place in the sort
};

// Bytes of a stage's weights: along, rows of RP ranks x 128 columns; across, rows
// of 128 columns x RP ranks (in blocks of 64 elements either way).
constexpr int weight_bytes(int RP, bool along) { return along ? 2 * RP * 128 : (RP + 63) / 64 * kBlock; }
// Of a tile's planes side by side, in blocks of 64 elements.
constexpr int planes_bytes(int RP) { return (kPlanes * RP + 63) / 64 * kBlock; }

// A producer thread's part of a stage: column piece `piece` of rows row0 + 8 j,
// whose swizzled places are 1024 bytes apart.
struct Producer {
    int piece, row0;
    uint32_t dst;
};
__device__ __forceinline__ Producer make_producer() {
    Producer t;
    const int pt = threadIdx.x - kEpiThreads;
    t.piece = pt % 16;
    t.row0 = pt / 16;
    t.dst = (t.piece / 8) * kBlock + sw128(t.row0, t.piece % 8);
    return t;
}

// Rows of x or base: src[j] is this thread's piece of column 0 of its row; columns
// past n are zeros.
__device__ __forceinline__ void stage_rows(const Producer &t, unsigned char *xs, const uint16_t *const (&src)[kTile / 8],
                                           int rows, long long col, int n, int vec) {
    const uint32_t dst = smem_u32(xs) + t.dst;
    const bool in = 8 * t.piece < n;
    if (vec) {
        const long long at = in ? col : 0;
        #pragma unroll
        for (int j = 0; j < kTile / 8; ++j)
            if (j < rows) cp_async16z(dst + 1024 * j, src[j] + at, in);
    } else {
        #pragma unroll
        for (int j = 0; j < kTile / 8; ++j)
            if (j < rows) *reinterpret_cast<uint4 *>(xs + t.dst + 1024 * j) = load_cols8(src[j] + col, n - 8 * t.piece, 0);
    }
}

// Weights of a stage.  [r][cols]: this thread's piece of the ranks row0 + 8 j;
// [cols][r]: pieces of the columns' rows.  Past the last rank or column: zeros
// (they are summed over).
template <int RP, bool ALONG>
__device__ __forceinline__ void stage_weights(const Producer &t, uint32_t ws, const uint16_t *w, int r, int cols, int col,
                                              int n) {
    if (ALONG) {
        const bool in = 8 * t.piece < n;
        const uint32_t dst = ws + (t.piece / 8) * (RP * 128) + sw128(t.row0, t.piece % 8);
        const uint16_t *src = w + (long long)t.row0 * cols + (in ? col + 8 * t.piece : 0);
        const long long step = 8LL * cols;
        #pragma unroll
        for (int j = 0; j < RP / 8; ++j) {
            const bool ok = in && 8 * j < r;             // r is a multiple of 8
            cp_async16z(dst + 1024 * j, ok ? src : w, ok);
            src += step;
        }
    } else {
        constexpr int kPieces = RP / 8, kRows = kProducers / kPieces;   // rows in one go
        const int pt = threadIdx.x - kEpiThreads, q = pt % kPieces, row0 = pt / kPieces;
        const uint16_t *src = w + (long long)(col + row0) * r + 8 * q;
        #pragma unroll
        for (int j = 0; j < kCols / kRows; ++j) {
            const int row = row0 + kRows * j;
            const bool ok = row < n && 8 * q < r;
            cp_async16z(ws + (q / 8) * kBlock + sw128(row, q % 8), ok ? src + kRows * j * r : w, ok);
        }
    }
}

// The first producer warp fills segment seg's slot; everyone waits for it.
__device__ __forceinline__ bool tile_ready(const LoraArgs &p, TileSlots &ts, int seg, int tile, uint32_t tfull,
                                           uint32_t tempty, bool writer, int stall, volatile int *abort_flag) {
    const int slot = seg & 1;
    bool ok = true;
    if (writer) {
        if (seg >= 2) ok = mbar_wait(tempty + 8 * slot, ((seg >> 1) - 1) & 1, abort_flag, p.err);
        if (__all_sync(0xffffffffu, ok) && !stalled(stall, seg)) {
            find_tile_sorted<kTile>(p, tile, ts.rows[slot], ts.info[slot]);
            __syncwarp();
            if ((threadIdx.x & 31) == 0) mbar_arrive(tfull + 8 * slot);
        }
    }
    ok = ok && mbar_wait(tfull + 8 * slot, (seg >> 1) & 1, abort_flag, p.err);
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void tile_done(int seg, uint32_t tempty) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(tempty + 8 * (seg & 1));
}

// ------------------------------------------------------------ first product
// h[t][rank] = sum over columns of x[t][col] A[rank][col] (g: of dy and B, whose
// columns lie along the weight's rows: an MN-major operand).  Tokens are the MMA's M,
// ranks its N.  Bound by HBM, the rows of X: a stage is 32 KB of them and its weights;
// six stages fit at padded rank 16, five at 32, four at 64, three at 128 (in the gradient
// four up to 64).  4096 tokens of 8192 columns at rank 64 (67 MB): 21 us behind the sort,
// of which time stamps put 11.5 from the first data to the last sum (5.8 TB/s); the rest
// is the start and the walk's set-up (sizes -> tile -> rows -> X, one load after the other).
template <int RP, bool TRANS>
struct DownShape {
    static constexpr int kW = weight_bytes(RP, !TRANS);
    static constexpr int kStage = 2 * kBlock + kW;
    static constexpr int kStages = (kSmemMax - 1024) / kStage < 6 ? (kSmemMax - 1024) / kStage : 6;
    static constexpr int kSmem = kStages * kStage + 1024;
    // A tile's sums go in turn into several accumulators, which the epilogue adds: the
    // MMA cuts off what each addition leaves below the accumulator's last bit.  h of 8192
    // columns: relative error 3.8e-7 with four, 1.7e-6 with one, at the same time.
    static constexpr int kAcc = RP <= 64 ? 4 : 2;
    static_assert(kStages >= 3 && 2 * kAcc * RP <= kTmemCols, "the ring does not fit");
};

template <int RP, bool TRANS>
__global__ void __launch_bounds__(kThreads, 1) lora_down_kernel(const LoraArgs p) {
    using S = DownShape<RP, TRANS>;
    constexpr int NS = S::kStages;
    extern __shared__ unsigned char s_raw[];
    __shared__ uint64_t s_bar[2 * NS + 9];
    __shared__ TileSlots s_tiles;
    __shared__ int s_abort;
    __shared__ uint32_t s_tmem;
    unsigned char *s_mem = s_raw + (-smem_u32(s_raw) & 1023);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t full = smem_u32(s_bar), empty = full + 8 * NS, tfull = empty + 8 * NS, tempty = tfull + 16;
    const uint32_t dfull = tempty + 16, dempty = dfull + 16, drained = dempty + 16;
    if (threadIdx.x == 0) {
        mbar_init(drained, 1);
        for (int i = 0; i < NS; ++i) mbar_init(full + 8 * i, kProducers), mbar_init(empty + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull + 8 * i, 1), mbar_init(tempty + 8 * i, kThreads / 32);
            mbar_init(dfull + 8 * i, 1), mbar_init(dempty + 8 * i, kEpiWarps);
        }
        s_abort = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tc_alloc(smem_u32(&s_tmem), kTmemCols);
        tc_relinquish();
    }
    // While the sort runs (whose CTAs had waited for what came before when they let
    // this kernel start): this CTA's share of X, the first 256 KB of it, into L2.
    if (threadIdx.x == 0 && p.vec_in) {
        const long long t0 = (long long)p.tokens * blockIdx.x / gridDim.x * p.in;
        const long long t1 = (long long)p.tokens * (blockIdx.x + 1) / gridDim.x * p.in;
        const long long most = kPrefetch / 2, n = t1 - t0 < most ? t1 - t0 : most;
        for (long long at = 0; at < n; at += 8192)
            bulk_prefetch_l2(p.x + t0 + at, uint32_t(n - at < 8192 ? n - at : 8192) * 2);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int r = p.rank;
    pdl_wait();
    pdl_launch_dependents();
    const Walk w = make_walk(count_tiles(p).with, (p.in + kCols - 1) / kCols, blockIdx.x, gridDim.x);
    volatile int *abort_flag = &s_abort;

    int i = 0, seg = 0;                              // steps and tiles so far
    bool lost = false;                               // a wait of this warp's has run out
    long long u = w.u0;                              // the first unit that is not done
    for (int n_steps; u < w.u1; ++seg, u += n_steps) {
        const int tile = int(quotient(u, w.per)), k0 = int(u - (long long)tile * w.per);
        n_steps = int(w.u1 - u < w.per - k0 ? w.u1 - u : w.per - k0);
        lost = !tile_ready(p, s_tiles, seg, tile, tfull, tempty, warp == kEpiWarps, kStallDownTile, abort_flag);
        if (lost) break;
        const int *rows = s_tiles.rows[seg & 1];
        const int adapter = s_tiles.info[seg & 1][0], count = s_tiles.info[seg & 1][1];
        if (warp >= kEpiWarps && warp < kMmaWarp) {
            const Producer t = make_producer();
            const uint16_t *wt = p.w1 + (long long)adapter * r * p.in, *src[kTile / 8];
            const int mine = (count - t.row0 + 7) / 8;
            #pragma unroll
            for (int j = 0; j < kTile / 8; ++j)
                src[j] = p.x + (long long)rows[j < mine ? t.row0 + 8 * j : 0] * p.in + 8 * t.piece;
            for (int k = 0; k < n_steps; ++k, ++i) {
                const int s = i % NS, col = (k0 + k) * kCols, n = min(kCols, p.in - col);
                const bool ok = i < NS || mbar_wait(empty + 8 * s, (i / NS - 1) & 1, abort_flag, p.err);
                lost = !__all_sync(0xffffffffu, ok);
                if (lost) break;
                unsigned char *xs = s_mem + s * S::kStage;
                stage_rows(t, xs, src, mine, col, n, p.vec_in);
                stage_weights<RP, !TRANS>(t, smem_u32(xs) + 2 * kBlock, wt, r, p.in, col, n);
                if (!stalled(kStallDown, i)) stage_done(full + 8 * s, p.vec_in);
            }
            if (lost) break;
        } else if (warp == kMmaWarp) {
            constexpr uint32_t idesc = tc_idesc_bf16(kTile, RP) | (TRANS ? kTcBMajorN : 0);
            const uint32_t d = tmem + (seg & 1) * (S::kAcc * RP);
            bool ok = seg < 2 || mbar_wait(dempty + 8 * (seg & 1), ((seg >> 1) - 1) & 1, abort_flag, p.err);
            ok = __all_sync(0xffffffffu, ok);
            for (int k = 0; k < n_steps && ok; ++k, ++i) {
                const int s = i % NS;
                ok = __all_sync(0xffffffffu, mbar_wait(full + 8 * s, (i / NS) & 1, abort_flag, p.err));
                if (!ok) break;
                fence_proxy_async();
                tc_fence_after();
                const uint32_t xs = smem_u32(s_mem) + s * S::kStage, ws = xs + 2 * kBlock;
                if (elect_one()) {
                    #pragma unroll
                    for (int m = 0; m < kCols / 16; ++m) {
                        const uint64_t a = tc_sdesc_sw128(xs + (m / 4) * kBlock + (m % 4) * 32);
                        const uint64_t b = TRANS ? tc_sdesc_sw128_mn(ws + m * 2048, kBlock)
                                                 : tc_sdesc_sw128(ws + (m / 4) * (RP * 128) + (m % 4) * 32);
                        tc_mma_ss(d + m % S::kAcc * RP, a, b, idesc, k > 0 || m >= S::kAcc);
                    }
                    tc_commit(empty + 8 * s);
                }
                __syncwarp();
            }
            lost = !ok;
            if (lost) break;
            if (elect_one()) tc_commit(dfull + 8 * (seg & 1));
            __syncwarp();
        } else {
            // this run's sum over the tile's columns, to its slot
            const int sub = warp % 4, half = warp / 4, row = 32 * sub + lane;
            lost = !__all_sync(0xffffffffu, mbar_wait(dfull + 8 * (seg & 1), (seg >> 1) & 1, abort_flag, p.err));
            if (lost) break;
            tc_fence_after();
            float *out = p.partial + ((long long)(tile + blockIdx.x) * kTile + row) * RP + half * (RP / 2);
            #pragma unroll
            for (int k = 0; k < RP / 16; ++k) {
                uint32_t v[8], w[S::kAcc - 1][8];
                const uint32_t at = tmem + (uint32_t(32 * sub) << 16) + (seg & 1) * (S::kAcc * RP) + half * (RP / 2) + 8 * k;
                tc_ld_32x32b_x8(at, v);
                #pragma unroll
                for (int n = 1; n < S::kAcc; ++n) {
                    tc_ld_32x32b_x8(at + n * RP, w[n - 1]);
                    __syncwarp();
                }
                tc_wait_ld();
                #pragma unroll
                for (int n = 1; n < S::kAcc; ++n)
                    #pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = __float_as_uint(__uint_as_float(v[e]) + __uint_as_float(w[n - 1][e]));
                if (row < count) {
                    *reinterpret_cast<uint4 *>(out + 8 * k) = make_uint4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<uint4 *>(out + 8 * k + 4) = make_uint4(v[4], v[5], v[6], v[7]);
                }
                __syncwarp();                        // tcgen05.ld takes the whole warp
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(dempty + 8 * (seg & 1));
        }
        tile_done(seg, tempty);
    }
    if (warp < kEpiWarps)                            // the tiles that a wait lost, this thread's part
        for (; u < w.u1; u += w.per - u % w.per) {
            const int tile = int(u / w.per), row = 32 * (warp % 4) + lane;
            float *out = p.partial + ((long long)(tile + blockIdx.x) * kTile + row) * RP + warp / 4 * (RP / 2);
            if (row < locate_tile<kTile>(p, tile).count)
                for (int k = 0; k < RP / 2; ++k) out[k] = __int_as_float(0x7fffffff);
            __syncwarp();
        }
    cp_async_wait_all();
    if (warp == kMmaWarp) drain_mmas(drained);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tc_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ its sums
// h of every tile: its slots in CTA order, to the planes (scaled) and p.hidden;
// in the gradient the planes of g, and of s h from p.hidden, by tile too.  Four
// ranks a thread, all of a tile's slots (5 of them at 4096 tokens) on their way
// at once.
constexpr int kSumThreads = 256;
// Blocks of a tile, four ranks of a row per thread: the kernel is a chain of
// latencies (a quarter of the blocks with four rows each took 7.6 us, these 3.5 when
// the sums are in L2: 4096 tokens at rank 64).
constexpr int sum_blocks(int RP) { return kTile * (RP / 4) / kSumThreads; }

template <int RP, bool TRANS>
__global__ void __launch_bounds__(kSumThreads) lora_sum_kernel(const LoraArgs p, int down_ctas) {
    constexpr int kPieces = RP / 4, kRows = kTile / sum_blocks(RP), kSlots = 8;
    static_assert(kRows * kPieces == kSumThreads, "one piece a thread");
    __shared__ int s_rows[kTile];
    __shared__ int s_info[3];
    __shared__ long long s_slots[2];                     // first slot, how many
    __shared__ uint16_t s_t[TRANS ? kPlanes * RP : 1][kRows + 2];   // g, then s h: [plane, rank][row]
    // The first product's CTAs let this kernel start after the sort had ended.
    pdl_launch_dependents();
    const int tile = blockIdx.x / sum_blocks(RP), row0 = blockIdx.x % sum_blocks(RP) * kRows;
    if (threadIdx.x < 32) {
        find_tile_sorted<kTile>(p, tile, s_rows, s_info);
        const Walk d = make_walk(count_tiles(p).with, (p.in + kCols - 1) / kCols, 0, down_ctas);
        __syncwarp();
        if (threadIdx.x == 0 && s_info[1] > 0 && s_info[0] >= 0) {
            const long long first = (long long)tile * d.per;
            const int b0 = run_owner(d.units, d.ctas, first);
            s_slots[0] = tile + b0;
            s_slots[1] = run_owner(d.units, d.ctas, first + d.per - 1) - b0 + 1;
        }
    }
    __syncthreads();
    const int adapter = s_info[0], count = s_info[1], r = p.rank;
    if (count == 0) return;
    const float scale = adapter >= 0 ? p.scale[adapter] : 0.f;
    const int slots = adapter >= 0 ? int(s_slots[1]) : 0;
    const int rank = 4 * (threadIdx.x % kPieces);
    pdl_wait();
    #pragma unroll
    for (int which = 0; which < (TRANS ? 2 : 1); ++which) {
        // first g (forward: h), then s h as it was kept
        {
            const int row = row0 + threadIdx.x / kPieces;
            const bool token = row < count, in = token && rank < r;
            float4 *hidden = reinterpret_cast<float4 *>(p.hidden + (in ? (long long)s_rows[row] * r + rank : 0));
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in && which) {
                v = *hidden;
            } else if (in) {
                const float *at = p.partial + (s_slots[0] * kTile + row) * RP + rank;
                for (int b = 0; b < slots; b += kSlots) {
                    float4 u[kSlots];
                    #pragma unroll
                    for (int k = 0; k < kSlots; ++k)
                        if (b + k < slots) u[k] = *reinterpret_cast<const float4 *>(at + (long long)(b + k) * kTile * RP);
                    #pragma unroll
                    for (int k = 0; k < kSlots; ++k)
                        if (b + k < slots) v.x += u[k].x, v.y += u[k].y, v.z += u[k].z, v.w += u[k].w;
                }
                if (!TRANS && p.hidden) *hidden = v;     // zeros without an adapter
            }
            if (adapter < 0) return;
            // ranks past r and rows past the tokens are zeros, also where x or the scale is
            // infinite (0 * inf)
            if (in) v = make_float4(scale * v.x, scale * v.y, scale * v.z, scale * v.w);
            uint32_t v01[kPlanes], v23[kPlanes];
            split3(v.x, v.y, v01), split3(v.z, v.w, v23);
            if (token && !which) {
                const long long out = (long long)(s_info[2] + row) * (plane_pitch(RP) / 2) + rank;
                #pragma unroll
                for (int k = 0; k < kPlanes; ++k)
                    *reinterpret_cast<uint2 *>(p.planes + out + k * RP) = make_uint2(v01[k], v23[k]);
            }
            if (TRANS) {
                #pragma unroll
                for (int k = 0; k < kPlanes; ++k)
                    #pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s_t[k * RP + rank + e][row - row0] = uint16_t((e < 2 ? v01[k] : v23[k]) >> (16 * (e & 1)));
            }
        }
        if (TRANS) {
            __syncthreads();
            uint16_t *out = (which ? p.th : p.tg) + (long long)tile * tile_planes(RP) + row0;
            for (int i = threadIdx.x; i < kPlanes * RP * kRows / 2; i += kSumThreads) {
                const int pair = i % (kRows / 2), line = i / (kRows / 2);
                *reinterpret_cast<uint32_t *>(out + line * kTile + 2 * pair) = *reinterpret_cast<const uint32_t *>(&s_t[line][2 * pair]);
            }
            __syncthreads();
        }
    }
}

// ----------------------------------------------------------- second product
// y[t][col] = base[t][col] + sum over ranks and planes of h[t][rank] B[col][rank] (dx: A,
// the weight's ranks along its rows, an MN-major operand).  Tokens are the MMA's M, the
// stage's 128 columns its N; the low plane first, all into one accumulator in TMEM.
// Bound by HBM: base in, y out.  The accumulators meet base in its swizzled place, and
// a warp stores four rows' 128 bytes in one instruction; pieces four at a time (one at a
// time the shared-memory round trips took 2 of 57.5 us below).  2858 tokens of 12 adapters,
// 17408 columns, rank 16: 38 of the call's 56 us, 5.2 TB/s with 200 MB of base and y.
template <int RP, bool TRANS>
struct UpShape {
    static constexpr int kW = weight_bytes(RP, TRANS);
    static constexpr int kStage = 2 * kBlock + kW;
    static constexpr int kH = planes_bytes(RP);
    static constexpr int kStages = (kSmemMax - 1024 - kH) / kStage < 5 ? (kSmemMax - 1024 - kH) / kStage : 5;
    static constexpr int kSmem = kStages * kStage + kH + 1024;
    static_assert(kStages >= 2, "the ring does not fit");
};

template <int RP, bool TRANS>
__global__ void __launch_bounds__(kThreads, 1) lora_up_kernel(const LoraArgs p) {
    using S = UpShape<RP, TRANS>;
    constexpr int NS = S::kStages, KS = RP / 16;
    extern __shared__ unsigned char s_raw[];
    __shared__ uint64_t s_bar[2 * NS + 15];
    __shared__ TileSlots s_tiles;
    __shared__ int s_abort;
    __shared__ uint32_t s_tmem;
    unsigned char *s_mem = s_raw + (-smem_u32(s_raw) & 1023);
    unsigned char *s_h = s_mem + NS * S::kStage;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t full = smem_u32(s_bar), empty = full + 8 * NS, tfull = empty + 8 * NS, tempty = tfull + 16;
    const uint32_t dfull = tempty + 16, dempty = dfull + 32, hready = dempty + 32;
    const uint32_t multiplied = hready + 8, drained = multiplied + 8;
    if (threadIdx.x == 0) {
        mbar_init(multiplied, kEpiWarps), mbar_init(drained, 1);
        for (int i = 0; i < NS; ++i) mbar_init(full + 8 * i, kProducers), mbar_init(empty + 8 * i, kEpiWarps / 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull + 8 * i, 1), mbar_init(tempty + 8 * i, kThreads / 32);
        }
        for (int i = 0; i < 4; ++i) mbar_init(dfull + 8 * i, 1), mbar_init(dempty + 8 * i, kEpiWarps / 2);
        mbar_init(hready, kEpiThreads);
        s_abort = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tc_alloc(smem_u32(&s_tmem), kTmemCols);
        tc_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int r = p.rank;
    // The first product's CTAs had waited for what came before them when they let
    // the next kernel start: the sort, base and the weights may be read at once.
    // h is waited for where the kernel before this one makes it (forward); in the
    // gradient that is the weight gradients', which had waited for it.
    const TileCount tiles = count_tiles(p);
    const Walk w = make_walk(tiles.with + tiles.without, (p.out + kCols - 1) / kCols, blockIdx.x, gridDim.x);
    volatile int *abort_flag = &s_abort;

    // steps, tiles, multiplied tiles; step i multiplies into buffer i % 4 of D2
    int i = 0, seg = 0, h_seg = 0;
    uint32_t uses = 0;                               // a bit per buffer: the parity of its next use
    uint32_t used = 0;
    bool lost = false;                               // a wait of this warp's has run out
    long long u = w.u0;                              // the first unit that is not done
    for (int n_steps; u < w.u1; ++seg, u += n_steps) {
        const int tile = int(quotient(u, w.per)), k0 = int(u - (long long)tile * w.per);
        n_steps = int(w.u1 - u < w.per - k0 ? w.u1 - u : w.per - k0);
        lost = !tile_ready(p, s_tiles, seg, tile, tfull, tempty, warp == kEpiWarps, kStallUpTile, abort_flag);
        if (lost) break;
        const int *rows = s_tiles.rows[seg & 1];
        const int adapter = s_tiles.info[seg & 1][0], count = s_tiles.info[seg & 1][1];
        const bool in_place = adapter < 0 && p.y == p.base;      // nothing to do
        if (warp >= kEpiWarps && warp < kMmaWarp) {
            const Producer t = make_producer();
            const uint16_t *wt = p.w2 + (long long)max(adapter, 0) * r * p.out, *src[kTile / 8];
            const int mine = p.base ? (count - t.row0 + 7) / 8 : 0;
            #pragma unroll
            for (int m = 0; m < kTile / 8; ++m)
                src[m] = p.base + (long long)rows[m < mine ? t.row0 + 8 * m : 0] * p.out + 8 * t.piece;
            for (int k = 0; k < n_steps && !in_place; ++k, ++i) {
                const int s = i % NS, col = (k0 + k) * kCols, n = min(kCols, p.out - col);
                const bool ok = i < NS || mbar_wait(empty + 8 * s, (i / NS - 1) & 1, abort_flag, p.err);
                lost = !__all_sync(0xffffffffu, ok);
                if (lost) break;
                unsigned char *xs = s_mem + s * S::kStage;
                stage_rows(t, xs, src, mine, col, n, p.vec_out);
                if (adapter >= 0) stage_weights<RP, TRANS>(t, smem_u32(xs) + 2 * kBlock, wt, r, p.out, col, n);
                if (!stalled(kStallUp, i)) stage_done(full + 8 * s, p.vec_out);
            }
            if (lost) break;
        } else if (warp == kMmaWarp) {
            constexpr uint32_t idesc = tc_idesc_bf16(kTile, kCols) | (TRANS ? kTcBMajorN : 0);
            if (adapter >= 0) {
                bool ok = __all_sync(0xffffffffu, mbar_wait(hready, h_seg & 1, abort_flag, p.err));
                ++h_seg;
                for (int k = 0; k < n_steps && ok; ++k, ++i) {
                    const int s = i % NS, buf = i & 3;
                    if ((used >> buf) & 1) ok = mbar_wait(dempty + 8 * buf, (~uses >> buf) & 1, abort_flag, p.err);
                    used |= 1u << buf;
                    uses ^= 1u << buf;
                    ok = ok && mbar_wait(full + 8 * s, (i / NS) & 1, abort_flag, p.err);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    fence_proxy_async();
                    tc_fence_after();
                    const uint32_t ws = smem_u32(s_mem) + s * S::kStage + 2 * kBlock;
                    if (elect_one()) {
                        #pragma unroll
                        for (int part = kPlanes - 1; part >= 0; --part)     // the low plane first
                            #pragma unroll
                            for (int m = 0; m < KS; ++m) {
                                const int k = part * KS + m;                 // 16 columns of the planes
                                const uint64_t a = tc_sdesc_sw128(smem_u32(s_h) + (k / 4) * kBlock + (k % 4) * 32);
                                const uint64_t b = TRANS ? tc_sdesc_sw128_mn(ws + m * 2048, RP * 128)
                                                         : tc_sdesc_sw128(ws + (m / 4) * kBlock + (m % 4) * 32);
                                tc_mma_ss(tmem + buf * kCols, a, b, idesc, part < kPlanes - 1 || m > 0);
                            }
                        tc_commit(dfull + 8 * buf);
                    }
                    __syncwarp();
                }
                lost = !ok;
                if (lost) break;
            } else if (!in_place) {
                i += n_steps;
            }
        } else {
            // Two groups of four warps take the steps in turn, two buffers of D2 each (with
            // one buffer 1100 to 1700 of a group's 5300 cycles a step went by waiting for
            // the MMAs); a warp has 32 rows.
            const int sub = warp % 4, group = warp / 4, my_row = 32 * sub + lane;
            if (seg == 0 && !TRANS) pdl_wait();
            if (seg > 0) {
                // the MMAs of the tile before have ended: every warp of these has waited for its own
                __syncwarp();
                if (lane == 0) mbar_arrive(multiplied);
                lost = !__all_sync(0xffffffffu, mbar_wait(multiplied, (seg - 1) & 1, abort_flag, p.err));
                if (lost) break;
            }
            if (adapter >= 0) {
                // h's planes of the tile; rows past its tokens are zeros
                const int start = s_tiles.info[seg & 1][2];
                constexpr int kPieces = kPlanes * RP / 8, kOnce = RP >= 64 ? 6 : kPlanes * RP / 16;
                static_assert(kTile * kPieces % (kOnce * kEpiThreads) == 0, "whole rounds");
                #pragma unroll 1
                for (int m0 = threadIdx.x; m0 < kTile * kPieces; m0 += kOnce * kEpiThreads) {
                    uint4 v[kOnce];
                    #pragma unroll
                    for (int e = 0; e < kOnce; ++e) {
                        const int m = m0 + e * kEpiThreads, row = m / kPieces, b = m % kPieces;
                        v[e] = make_uint4(0, 0, 0, 0);
                        if (row < count)
                            v[e] = *(reinterpret_cast<const uint4 *>(p.planes + (long long)(start + row) * (plane_pitch(RP) / 2)) + b);
                    }
                    #pragma unroll
                    for (int e = 0; e < kOnce; ++e) {
                        const int m = m0 + e * kEpiThreads, row = m / kPieces, b = m % kPieces;
                        *reinterpret_cast<uint4 *>(s_h + (b / 8) * kBlock + sw128(row, b % 8)) = v[e];
                    }
                }
                fence_proxy_async();
                mbar_arrive(hready);
            }
            for (int k = 0; k < n_steps && !in_place; ++k, ++i) {
                if ((i & 1) != group) continue;
                const int s = i % NS;
                const uint32_t lanes = tmem + (uint32_t(32 * sub) << 16) + (i & 3) * kCols;
                bool ok = mbar_wait(full + 8 * s, (i / NS) & 1, abort_flag, p.err);
                if (adapter >= 0) {
                    ok = ok && mbar_wait(dfull + 8 * (i & 3), (uses >> (i & 3)) & 1, abort_flag, p.err);
                    uses ^= 1u << (i & 3);
                    tc_fence_after();
                }
                lost = !__all_sync(0xffffffffu, ok);
                if (lost) {
                    u += k;
                    break;
                }
                #pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const int col = (k0 + k) * kCols + 64 * half;
                    if (col >= p.out || 32 * sub >= count) break;
                    unsigned char *bs = s_mem + s * S::kStage + half * kBlock;
                    // Four pieces of 16 bytes at once: the compiler cannot tell that a store of
                    // one leaves the next one's load alone.
                    if (adapter >= 0) {
                        uint32_t acc[2][32];
                        tc_ld_32x32b_x32(lanes + 64 * half, acc[0]);
                        tc_ld_32x32b_x32(lanes + 64 * half + 32, acc[1]);
                        uint4 v[4];
                        #pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            #pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                v[q] = make_uint4(0, 0, 0, 0);
                                if (p.base) v[q] = *reinterpret_cast<const uint4 *>(bs + sw128(my_row, 4 * h + q));
                            }
                            if (h == 0) tc_wait_ld();
                            #pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const uint32_t *d = &acc[h][8 * q];
                                const uint4 b = v[q];
                                v[q].x = pack_bf16x2_rn(bf16_lo_to_f32(b.x) + __uint_as_float(d[0]), bf16_hi_to_f32(b.x) + __uint_as_float(d[1]));
                                v[q].y = pack_bf16x2_rn(bf16_lo_to_f32(b.y) + __uint_as_float(d[2]), bf16_hi_to_f32(b.y) + __uint_as_float(d[3]));
                                v[q].z = pack_bf16x2_rn(bf16_lo_to_f32(b.z) + __uint_as_float(d[4]), bf16_hi_to_f32(b.z) + __uint_as_float(d[5]));
                                v[q].w = pack_bf16x2_rn(bf16_lo_to_f32(b.w) + __uint_as_float(d[6]), bf16_hi_to_f32(b.w) + __uint_as_float(d[7]));
                                *reinterpret_cast<uint4 *>(bs + sw128(my_row, 4 * h + q)) = v[q];
                            }
                        }
                    } else if (!p.base) {
                        #pragma unroll
                        for (int q = 0; q < 8; ++q)
                            *reinterpret_cast<uint4 *>(bs + sw128(my_row, q)) = make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                    const int q = lane % 8, left = p.out - col - 8 * q;
                    #pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint4 v[4];
                        uint16_t *y[4];
                        #pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const int row = 32 * sub + 16 * h + 4 * m + lane / 8;
                            v[m] = *reinterpret_cast<const uint4 *>(bs + sw128(row, q));
                            y[m] = p.y + (long long)rows[row < count ? row : 0] * p.out + col + 8 * q;
                        }
                        #pragma unroll
                        for (int m = 0; m < 4; ++m)
                            if (32 * sub + 16 * h + 4 * m + lane / 8 < count) store_cols8(y[m], left, p.vec_out, v[m]);
                    }
                    __syncwarp();                            // tcgen05.ld takes the whole warp
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (adapter >= 0) mbar_arrive(dempty + 8 * (i & 3));
                    mbar_arrive(empty + 8 * s);
                }
            }
            if (lost) break;
        }
        tile_done(seg, tempty);
    }
    pdl_wait();
    pdl_launch_dependents();
    if (warp < kEpiWarps)                            // the steps that a wait lost, this warp's rows
        for (; u < w.u1; ++u) {
            const int tile = int(u / w.per), col = int(u % w.per) * kCols, n = min(kCols, p.out - col);
            const Tile t = locate_tile<kTile>(p, tile);
            if (t.adapter < 0 && p.y == p.base) continue;
            if ((i++ & 1) != warp / 4) continue;
            for (int row = 32 * (warp % 4); row < min(t.count, 32 * (warp % 4) + 32); ++row)
                for (int c = lane; c < n; c += 32)
                    p.y[(long long)p.order[t.start + row] * p.out + col + c] = 0x7fffu;
        }
    cp_async_wait_all();
    if (warp == kMmaWarp) drain_mmas(drained);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tc_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------- weight gradients
constexpr int kStageTokens = 32;
// Warps: eight producers, four that empty TMEM, one that issues the MMAs.
constexpr int kWgradProducerWarps = 8, kWgradProducers = kWgradProducerWarps * 32, kWgradStore = 4;
constexpr int kWgradMma = kWgradProducerWarps + kWgradStore, kWgradThreads = (kWgradMma + 1) * 32;

template <int RP>
struct WgradShape {
    static constexpr int kCols = RP <= 64 ? 512 : 256;      // columns of a pair
    static constexpr int kQBlock = kStageTokens * 128;      // bytes of 32 tokens x 64 columns
    static constexpr int kQ = kCols / 64 * kQBlock;
    static constexpr int kP = kPlanes * RP * 64;            // the planes: rows of 32 tokens
    static constexpr int kStage = kQ + kP;
    static constexpr int kStages = (kSmemMax - 1024) / kStage < 6 ? (kSmemMax - 1024) / kStage : 6;
    static constexpr int kSmem = kStages * kStage + 1024;
    static constexpr int kD = kCols / 128 * 2 * RP;         // TMEM columns of a pair's sums: of the high plane, of the others
    static constexpr int kBufs = 2 * kD <= kTmemCols ? 2 : 1;
    static constexpr int kTileSums = kCols * RP;            // floats of a pair's sums
    static_assert(kStages >= 3 && kD <= kTmemCols, "the ring does not fit");
};

// The walk: a pair is an adapter with tokens and a slice of columns of x or dy; a
// unit is a block of 32 of its tokens; a CTA takes an even run of all units.
struct Pair {
    int adapter, slice, start, tile0, size, blocks;   // start, tile0: the adapter's first place and tile
    long long first;                                  // its first unit
};
// Every warp finds its pairs itself.
__device__ Pair find_pair(const WgradArgs &p, long long u) {
    const int lane = threadIdx.x & 31;
    Pair q = {};
    long long units = 0;
    int rows = 0, tiles = 0;
    for (int a0 = 0; a0 < p.adapters; a0 += 32) {
        const int size = a0 + lane < p.adapters ? p.sizes[a0 + lane] : 0;
        const int blocks = (size + kStageTokens - 1) / kStageTokens, my_tiles = (size + kTile - 1) / kTile;
        const long long mine = (long long)blocks * p.slices;
        long long u_end = mine;
        int r_end = size, t_end = my_tiles;
        #pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const long long x = __shfl_up_sync(0xffffffffu, u_end, d);
            const int y = __shfl_up_sync(0xffffffffu, r_end, d), z = __shfl_up_sync(0xffffffffu, t_end, d);
            if (lane >= d) u_end += x, r_end += y, t_end += z;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, u >= units + u_end - mine && u < units + u_end);
        if (hit) {
            const int src = __ffs(hit) - 1;
            q.adapter = a0 + src;
            q.size = __shfl_sync(0xffffffffu, size, src);
            q.blocks = __shfl_sync(0xffffffffu, blocks, src);
            q.start = __shfl_sync(0xffffffffu, rows + r_end - size, src);
            q.tile0 = __shfl_sync(0xffffffffu, tiles + t_end - my_tiles, src);
            const long long base = __shfl_sync(0xffffffffu, units + u_end - mine, src);
            q.slice = int(quotient(u - base, q.blocks));
            q.first = base + (long long)q.slice * q.blocks;
            return q;
        }
        units += __shfl_sync(0xffffffffu, u_end, 31);
        rows += __shfl_sync(0xffffffffu, r_end, 31);
        tiles += __shfl_sync(0xffffffffu, t_end, 31);
    }
    return q;
}
__device__ __forceinline__ long long count_units(const WgradArgs &p) {
    int blocks = 0;
    for (int a = threadIdx.x & 31; a < p.adapters; a += 32) blocks += (p.sizes[a] + kStageTokens - 1) / kStageTokens;
    return (long long)__reduce_add_sync(0xffffffffu, blocks) * p.slices;
}

// D[column][plane, rank] of a pair is summed in TMEM in blocks of 128 columns: x or
// dy lies along M as it comes, the planes of g or s h along N: one MMA for the upper
// two, one that adds the lowest to the middle's sums (TMEM holds no third).
// A run that covers all of a pair's tokens stores the gradient, the others their
// sums ([rank][column], slot 0: the pair began before the run, slot 1: it goes on
// after it) for wgrad_sum_kernel.
//
// What bounds it: the MMAs, with the rows along M: 142 cycles for 128 x 128 x 16 (the
// upper two planes at rank 64), 90 for 128 x 64 x 16 (the lowest plane; its MMAs are 6 of
// the 42 us below).  x or dy as the MMA's 256 columns took 375; one MMA for all three
// planes, whose sums leave room for slices of 256 columns only, 2 us more.  4096 tokens
// of 8192 and 8192 columns at rank 64: 42 us behind g, 3.2 TB/s of x and dy (dy from L2)
// besides three eighths of that in planes.
template <int RP>
__global__ void __launch_bounds__(kWgradThreads, 1) lora_wgrad_kernel(const WgradArgs p) {
    using S = WgradShape<RP>;
    constexpr int NS = S::kStages;
    extern __shared__ unsigned char s_raw[];
    __shared__ uint64_t s_bar[2 * NS + 5];
    __shared__ int s_abort;
    __shared__ uint32_t s_tmem;
    unsigned char *s_mem = s_raw + (-smem_u32(s_raw) & 1023);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t ring = smem_u32(s_mem), full = smem_u32(s_bar), empty = full + 8 * NS;
    const uint32_t dfull = empty + 8 * NS, dempty = dfull + 16, drained = dempty + 16;
    if (threadIdx.x == 0) {
        mbar_init(drained, 1);
        for (int i = 0; i < NS; ++i) mbar_init(full + 8 * i, kWgradProducers), mbar_init(empty + 8 * i, 1);
        for (int i = 0; i < 2; ++i) mbar_init(dfull + 8 * i, 1), mbar_init(dempty + 8 * i, kWgradStore);
        s_abort = 0;
        fence_barrier_init();
    }
    if (warp == kWgradMma) {
        tc_alloc(smem_u32(&s_tmem), kTmemCols);
        tc_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    // The sort had ended when the kernel before let this one start.
    const long long units = count_units(p);
    const int ctas = int(units < gridDim.x ? units : gridDim.x), b = blockIdx.x;
    const long long u0 = b < ctas ? run_start(units, ctas, b) : 0, u1 = b < ctas ? run_start(units, ctas, b + 1) : 0;
    const int r = p.rank;
    pdl_wait();
    pdl_launch_dependents();
    volatile int *abort_flag = &s_abort;
    int i = 0, seg = 0;                                          // stages, pairs
    bool lost = false;                                           // a wait of this warp's has run out
    for (long long u = u0; u < u1; ++seg) {
        const Pair q = find_pair(p, u);
        const int block0 = int(u - q.first);
        const int n_blocks = int(u1 - u < q.blocks - block0 ? u1 - u : q.blocks - block0);
        u += n_blocks;
        const bool db = q.slice >= p.slices_x;
        const int cols = db ? p.N : p.K, col0 = (db ? q.slice - p.slices_x : q.slice) * S::kCols;
        const int width = min(S::kCols, cols - col0), buf = seg % S::kBufs;
        if (warp < kWgradProducerWarps) {
            // Rows row0 + 16 j, column pieces piece + 16 e: their places are 2048 bytes and
            // 2 blocks apart.  The rows of the next stage are looked up one stage ahead.
            const uint16_t *src_q = db ? p.dy : p.x;
            const uint16_t *src_p = (db ? p.th : p.tg) + (long long)q.tile0 * tile_planes(RP);
            const int vec = db ? p.vec_dy : 1, *rows = p.order + q.start;
            const int pt = threadIdx.x, piece = pt % 16, row0 = pt / 16;
            constexpr int kRows = kWgradProducers / 16, kJ = kStageTokens / kRows, kE = S::kCols / 128;
            const uint32_t dst = (piece / 8) * S::kQBlock + sw128(row0, piece % 8);
            int next[kJ];
            #pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const int t = block0 * kStageTokens + row0 + kRows * j;
                next[j] = t < q.size ? rows[t] : -1;
            }
            for (int k = 0; k < n_blocks; ++k, ++i) {
                const int s = i % NS, tok = (block0 + k) * kStageTokens;
                int row[kJ];
                #pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    const int t = tok + kStageTokens + row0 + kRows * j;
                    row[j] = next[j];
                    next[j] = t < q.size ? rows[t] : -1;
                }
                const bool ok = i < NS || mbar_wait(empty + 8 * s, (i / NS - 1) & 1, abort_flag, p.err);
                lost = !__all_sync(0xffffffffu, ok);
                if (lost) break;
                const uint32_t qs = ring + s * S::kStage, ps = qs + S::kQ;
                // tokens past the last are zeros on both sides: they are summed over
                #pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    const bool in = row[j] >= 0;
                    const uint16_t *src = src_q + (long long)max(row[j], 0) * cols + col0 + 8 * piece;
                    #pragma unroll
                    for (int e = 0; e < kE; ++e) {
                        const int left = width - 8 * piece - 128 * e;
                        const uint32_t at = dst + kRows * 128 * j + 2 * S::kQBlock * e;
                        if (left <= 0) continue;
                        if (vec) cp_async16z(qs + at, in ? src + 128 * e : src_q, in);
                        else *reinterpret_cast<uint4 *>(s_mem + s * S::kStage + at) =
                                 load_cols8(src + 128 * e, in ? left : 0, 0);
                    }
                }
                // rows of 64 bytes (32 tokens of a plane's rank) in the 64-byte swizzle
                const uint16_t *src = src_p + (long long)(tok / kTile) * tile_planes(RP) + tok % kTile;
                #pragma unroll 1
                for (int m = pt; m < kPlanes * RP * 4; m += kWgradProducers) {
                    const int line = m / 4, e = m % 4;
                    cp_async16(ps + line * 64 + ((e ^ ((line >> 1) & 3)) << 4), src + line * kTile + 8 * e);
                }
                if (!stalled(kStallWgrad, i)) stage_done(full + 8 * s, vec);
            }
            if (lost) break;
        } else if (warp == kWgradMma) {
            constexpr uint32_t idesc = tc_idesc_bf16(128, 2 * RP) | kTcAMajorM, idesc1 = tc_idesc_bf16(128, RP) | kTcAMajorM;
            bool ok = seg < S::kBufs || mbar_wait(dempty + 8 * buf, (seg / S::kBufs - 1) & 1, abort_flag, p.err);
            ok = __all_sync(0xffffffffu, ok);
            for (int k = 0; k < n_blocks && ok; ++k, ++i) {
                const int s = i % NS;
                ok = __all_sync(0xffffffffu, mbar_wait(full + 8 * s, (i / NS) & 1, abort_flag, p.err));
                if (!ok) break;
                fence_proxy_async();
                tc_fence_after();
                const uint32_t qs = ring + s * S::kStage, ps = qs + S::kQ;
                if (elect_one()) {
                    #pragma unroll
                    for (int m = 0; m < S::kCols / 128; ++m)
                        #pragma unroll
                        for (int e = 0; e < kStageTokens / 16; ++e) {
                            const uint64_t dq = tc_sdesc_sw128_mn(qs + m * 2 * S::kQBlock + e * 2048, S::kQBlock);
                            const uint32_t d = tmem + buf * S::kD + m * 2 * RP;
                            tc_mma_ss(d, dq, tc_sdesc_sw64(ps + e * 32), idesc, k > 0 || e > 0);
                            tc_mma_ss(d + RP, dq, tc_sdesc_sw64(ps + 2 * RP * 64 + e * 32), idesc1, 1);
                        }
                    tc_commit(empty + 8 * s);
                }
                __syncwarp();
            }
            lost = !ok;
            if (lost) break;
            if (elect_one()) tc_commit(dfull + 8 * buf);
            __syncwarp();
        } else {
            const int sub = warp % 4;
            const bool ok = !lost && mbar_wait(dfull + 8 * buf, (seg / S::kBufs) & 1, abort_flag, p.err);
            lost = !__all_sync(0xffffffffu, ok);
            tc_fence_after();
            const bool whole = n_blocks == q.blocks;
            float *slot = p.partial + (long long)(2 * b + (block0 == 0)) * S::kTileSums;
            for (int m = 0; m < S::kCols / 128; ++m) {
                const int col = 128 * m + 32 * sub + lane;
                if (128 * m + 32 * sub >= width) break;
                #pragma unroll 1
                for (int rank = 0; rank < RP; rank += 8) {
                    uint32_t v[8], w[8];
                    const uint32_t at = tmem + (uint32_t(32 * sub) << 16) + buf * S::kD + m * 2 * RP + rank;
                    tc_ld_32x32b_x8(at, v);
                    tc_ld_32x32b_x8(at + RP, w);
                    tc_wait_ld();
                    // an infinity of x or dy: the upper plane's sum has it, the lower planes may
                    // hold zeros (0 * inf)
                    float f[8];
                    #pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        f[e] = __uint_as_float(v[e]);
                        if (!isinf(f[e])) f[e] += __uint_as_float(w[e]);
                        if (lost) f[e] = __int_as_float(0x7fffffff);
                    }
                    if (!whole) {
                        #pragma unroll
                        for (int e = 0; e < 8; ++e) __stcg(slot + (rank + e) * S::kCols + col, f[e]);
                    } else if (col < width && rank < r) {
                        if (db) {
                            *reinterpret_cast<uint4 *>(p.db + ((long long)q.adapter * cols + col0 + col) * r + rank) =
                                make_uint4(pack_bf16x2_rn(f[0], f[1]), pack_bf16x2_rn(f[2], f[3]),
                                           pack_bf16x2_rn(f[4], f[5]), pack_bf16x2_rn(f[6], f[7]));
                        } else {
                            uint16_t *d = p.da + ((long long)q.adapter * r + rank) * cols + col0 + col;
                            #pragma unroll
                            for (int e = 0; e < 8; ++e) d[(long long)e * cols] = f32_to_bf16_rn(f[e]);
                        }
                    }
                    __syncwarp();                                // tcgen05.ld takes the whole warp
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && !lost) mbar_arrive(dempty + 8 * buf);
        }
    }
    cp_async_wait_all();
    if (warp == kWgradMma) drain_mmas(drained);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWgradMma) tc_dealloc(tmem, kTmemCols);
}

// The gradients of pairs that several runs share: of a pair that n runs share the
// n blocks of these CTAs each add a part, in CTA order; so a block has a part of
// the pair its run began inside of and a part of the pair its run left unfinished.
// All blocks clear the gradients of adapters without tokens.  Bound by latency and
// L2: two tiles of sums per run at most (40 MB at rank 64), 9 us behind dX for 4096
// tokens of one adapter with 8192 and 8192 columns.
constexpr int kWgradSumThreads = 512;

template <int RP>
__device__ __forceinline__ void wgrad_sum_part(const WgradArgs &p, const Pair &q, int b0, int slots, int part) {
    using S = WgradShape<RP>;
    constexpr int kSlots = 8;
    const int r = p.rank;
    const bool db = q.slice >= p.slices_x;
    const int cols = db ? p.N : p.K, col0 = (db ? q.slice - p.slices_x : q.slice) * S::kCols;
    const int width = min(S::kCols, cols - col0);
    // the first CTA's slot 1, then the others' slot 0, which lie two apart
    const float *sum0 = p.partial + (long long)(2 * b0 + 1) * S::kTileSums, *rest = sum0 + S::kTileSums;
    const int items = db ? S::kCols * (r / 8) : r * width / 4;
    const int i0 = int((long long)items * part / slots), i1 = int((long long)items * (part + 1) / slots);
    for (int i = i0 + threadIdx.x; i < i1; i += kWgradSumThreads) {
        if (!db) {
            const int rank = i / (width / 4), col = 4 * (i % (width / 4)), at = rank * S::kCols + col;
            float4 v = *reinterpret_cast<const float4 *>(sum0 + at);
            for (int k0 = 1; k0 < slots; k0 += kSlots) {
                float4 u[kSlots];
                #pragma unroll
                for (int k = 0; k < kSlots; ++k)
                    if (k0 + k < slots)
                        u[k] = *reinterpret_cast<const float4 *>(rest + (long long)(2 * (k0 + k - 1)) * S::kTileSums + at);
                #pragma unroll
                for (int k = 0; k < kSlots; ++k)
                    if (k0 + k < slots) v.x += u[k].x, v.y += u[k].y, v.z += u[k].z, v.w += u[k].w;
            }
            *reinterpret_cast<uint2 *>(p.da + ((long long)q.adapter * r + rank) * cols + col0 + col) =
                make_uint2(pack_bf16x2_rn(v.x, v.y), pack_bf16x2_rn(v.z, v.w));
        } else {
            // one column, eight ranks: neighbouring threads read neighbouring columns
            const int col = i % S::kCols, rank = 8 * (i / S::kCols);
            if (col >= width) continue;
            float v[8];
            #pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = sum0[(rank + e) * S::kCols + col];
            for (int k0 = 1; k0 < slots; k0 += 4) {
                float u[4][8];
                #pragma unroll
                for (int k = 0; k < 4; ++k)
                    #pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (k0 + k < slots)
                            u[k][e] = rest[(long long)(2 * (k0 + k - 1)) * S::kTileSums + (rank + e) * S::kCols + col];
                #pragma unroll
                for (int k = 0; k < 4; ++k)
                    #pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (k0 + k < slots) v[e] += u[k][e];
            }
            *reinterpret_cast<uint4 *>(p.db + ((long long)q.adapter * cols + col0 + col) * r + rank) =
                make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]), pack_bf16x2_rn(v[4], v[5]),
                           pack_bf16x2_rn(v[6], v[7]));
        }
    }
}

template <int RP>
__global__ void __launch_bounds__(kWgradSumThreads, 2) wgrad_sum_kernel(const WgradArgs p) {
    __shared__ Pair s_pair;
    __shared__ int s_b0, s_slots;                        // 0 slots: no part
    pdl_launch_dependents();
    // blockIdx.y 0: the pair that the run began inside of; 1: the one that goes on
    const int r = p.rank, b = blockIdx.x, which = blockIdx.y;
    if (threadIdx.x < 32) {
        const long long units = count_units(p);
        const int ctas = int(units < gridDim.x ? units : gridDim.x);
        int b0 = 0, slots = 0;
        Pair q = {};
        if (b < ctas) {
            const long long u0 = run_start(units, ctas, b), u1 = run_start(units, ctas, b + 1);
            q = find_pair(p, which ? u1 - 1 : u0);
            const long long end = q.first + q.blocks;
            if (which ? (q.first >= u0 && end > u1) : q.first < u0) {
                b0 = run_owner(units, ctas, q.first);
                slots = run_owner(units, ctas, end - 1) - b0 + 1;
            }
        }
        if (threadIdx.x == 0) s_pair = q, s_b0 = b0, s_slots = slots;
    }
    __syncthreads();
    pdl_wait();
    if (s_slots) wgrad_sum_part<RP>(p, s_pair, s_b0, s_slots, b - s_b0);
    const long long na = (long long)r * p.K / 8, nb = (long long)r * p.N / 8, step = 2LL * gridDim.x * kWgradSumThreads;
    for (int a = 0; a < p.adapters; ++a) {
        if (p.sizes[a] != 0) continue;
        uint4 *da = reinterpret_cast<uint4 *>(p.da) + a * na, *db = reinterpret_cast<uint4 *>(p.db) + a * nb;
        for (long long i = (2LL * b + which) * kWgradSumThreads + threadIdx.x; i < na + nb; i += step)
            (i < na ? da[i] : db[i - na]) = make_uint4(0, 0, 0, 0);
    }
}

// ---------------------------------------------------------------- host side
int ceil_div(long long a, long long b) { return int((a + b - 1) / b); }

}  // namespace

// Tiles at most: the adapters' and the adapterless tokens' last may be part empty.
int lora_max_tiles(int tokens, int adapters) {
    return ceil_div(tokens, kTile) + (adapters < tokens ? adapters : tokens);
}

namespace {

template <int RP, bool TRANS>
cudaError_t launch_tensor_rank(const LoraArgs &p, LoraStep step, int sms, cudaStream_t s) {
    using D = DownShape<RP, TRANS>;
    using U = UpShape<RP, TRANS>;
    cudaError_t e = allow_smem<lora_down_kernel<RP, TRANS>>(D::kSmem);
    if (e == cudaSuccess) e = allow_smem<lora_up_kernel<RP, TRANS>>(U::kSmem);
    if (e != cudaSuccess) return e;
    const int ctas = sms < kMaxRuns ? sms : kMaxRuns;
    if (step == kLoraUp)
        return launch_chained(lora_up_kernel<RP, TRANS>, dim3(ctas), kThreads, U::kSmem, 1, s, p);
    e = launch_chained(lora_down_kernel<RP, TRANS>, dim3(ctas), kThreads, D::kSmem, 1, s, p);
    if (e != cudaSuccess) return e;
    const int blocks = lora_max_tiles(p.tokens, p.adapters) * sum_blocks(RP);
    return launch_chained(lora_sum_kernel<RP, TRANS>, dim3(blocks), kSumThreads, 0, 1, s, p, ctas);
}

template <int RP>
cudaError_t launch_wgrad_rank(WgradArgs p, WgradStep step, int sms, cudaStream_t s) {
    using S = WgradShape<RP>;
    cudaError_t e = allow_smem<lora_wgrad_kernel<RP>>(S::kSmem);
    if (e != cudaSuccess) return e;
    p.slices_x = ceil_div(p.K, S::kCols);
    p.slices = p.slices_x + ceil_div(p.N, S::kCols);
    const int ctas = sms < kMaxRuns ? sms : kMaxRuns;
    if (step == kWgradRuns)
        return launch_chained(lora_wgrad_kernel<RP>, dim3(ctas), kWgradThreads, S::kSmem, 1, s, p);
    return launch_chained(wgrad_sum_kernel<RP>, dim3(ctas, 2), kWgradSumThreads, 0, 1, s, p);
}

}  // namespace

size_t lora_partial_bytes(int tokens, int adapters, int rank, bool backward) {
    const int rp = padded_rank(rank);
    const size_t h = (size_t(lora_max_tiles(tokens, adapters)) + kMaxRuns) * kTile * rp * sizeof(float);
    const size_t grads = backward ? size_t(2) * kMaxRuns * (rp <= 64 ? 512 : 256) * rp * sizeof(float) : 0;
    return h > grads ? h : grads;
}

cudaError_t launch_lora_tensor(const LoraArgs &p, bool trans, LoraStep step, int sms, cudaStream_t s) {
    switch (padded_rank(p.rank)) {
        case 16: return trans ? launch_tensor_rank<16, true>(p, step, sms, s) : launch_tensor_rank<16, false>(p, step, sms, s);
        case 32: return trans ? launch_tensor_rank<32, true>(p, step, sms, s) : launch_tensor_rank<32, false>(p, step, sms, s);
        case 64: return trans ? launch_tensor_rank<64, true>(p, step, sms, s) : launch_tensor_rank<64, false>(p, step, sms, s);
        default: return trans ? launch_tensor_rank<128, true>(p, step, sms, s) : launch_tensor_rank<128, false>(p, step, sms, s);
    }
}

cudaError_t launch_wgrad(const WgradArgs &p, WgradStep step, int sms, cudaStream_t s) {
    switch (padded_rank(p.rank)) {
        case 16: return launch_wgrad_rank<16>(p, step, sms, s);
        case 32: return launch_wgrad_rank<32>(p, step, sms, s);
        case 64: return launch_wgrad_rank<64>(p, step, sms, s);
        default: return launch_wgrad_rank<128>(p, step, sms, s);
    }
}

}  // namespace w4a16

#ifdef W4A16_TEST_STALL
extern "C" int w4a16_test_stall(int kernel, int at) {
    const cudaError_t e = cudaMemcpyToSymbol(w4a16::g_stall_kernel, &kernel, sizeof kernel);
    return e != cudaSuccess ? int(e) : int(cudaMemcpyToSymbol(w4a16::g_stall_at, &at, sizeof at));
}
#endif
