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
// whole 128-byte pieces of rows.  h enters the second product as two bf16 planes.
//
// What bounds them: HBM.  At rank 64 the legacy MMA pipe would need two thirds of
// the memory's time and left a 64-token mma.sync version waiting on MMA latency
// (78 us for 4096 tokens, 8192 x 8192); tcgen05 needs a tenth.
//
// lora_wgrad_kernel: dA = g^T X and dB = s dY^T h.  The tokens are the MMA's K;
// rows of X or dY lie along M, rows of g or s h along N, as they come, so nothing
// is transposed.
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
constexpr int kMaxRuns = 160;          // CTAs of the two products: one per SM (152)

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory"); }

// Byte of piece p (16 bytes) of row `row` in a block of 128-byte rows.
__device__ __forceinline__ uint32_t sw128(int row, int p) { return uint32_t(row * 128 + ((p ^ (row & 7)) << 4)); }

// The walk: unit u = tile * per + step; CTA b of n takes units [run(b), run(b + 1)).
__device__ __forceinline__ long long run_start(long long units, int n, int b) { return units * b / n; }
// The CTA whose run holds unit u.
__device__ __forceinline__ int run_owner(long long units, int n, long long u) {
    return int(((u + 1) * n - 1) / units);
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

// One warp: tiles of all adapters and, past those, of the tokens without one.
__device__ void count_tiles(const LoraArgs &p, int *out) {
    const int lane = threadIdx.x & 31;
    int tiles = 0, rows = 0;
    for (int a = lane; a < p.adapters; a += 32) {
        const int size = p.sizes[a];
        tiles += (size + kTile - 1) / kTile;
        rows += size;
    }
    tiles = __reduce_add_sync(0xffffffffu, tiles);
    rows = __reduce_add_sync(0xffffffffu, rows);
    if (lane == 0) out[0] = tiles, out[1] = (p.tokens - rows + kTile - 1) / kTile;
}

// Two tiles' tokens, filled by the first producer warp ahead of the others.
struct TileSlots {
    int rows[2][kTile];
    int info[2][3];         // adapter (-1: none), tokens, first place in the sort
};

// Bytes of a stage's weights: along, rows of RP ranks x 128 columns; across, rows
// of 128 columns x RP ranks (in blocks of 64 elements either way).
constexpr int weight_bytes(int RP, bool along) { return along ? 2 * RP * 128 : (RP + 63) / 64 * kBlock; }
constexpr int plane_bytes(int RP) { return (RP + 63) / 64 * kBlock; }

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

// Rows of x or base: src[j] points at this thread's piece of column 0 of its
// row; columns past n are zeros.
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
                                           uint32_t tempty, bool writer, volatile int *abort_flag) {
    const int slot = seg & 1;
    bool ok = true;
    if (writer) {
        if (seg >= 2) ok = mbar_wait(tempty + 8 * slot, ((seg >> 1) - 1) & 1, abort_flag, p.err);
        if (__all_sync(0xffffffffu, ok)) {
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
template <int RP, bool TRANS>
struct DownShape {
    static constexpr int kW = weight_bytes(RP, !TRANS);
    static constexpr int kStage = 2 * kBlock + kW;
    static constexpr int kStages = (kSmemMax - 1024) / kStage < 6 ? (kSmemMax - 1024) / kStage : 6;
    static constexpr int kSmem = kStages * kStage + 1024;
    static_assert(kStages >= 3, "the ring does not fit");
};

template <int RP, bool TRANS>
__global__ void __launch_bounds__(kThreads, 1) lora_down_kernel(const LoraArgs p) {
    using S = DownShape<RP, TRANS>;
    constexpr int NS = S::kStages;
    extern __shared__ unsigned char s_raw[];
    __shared__ uint64_t s_bar[2 * NS + 8];
    __shared__ TileSlots s_tiles;
    __shared__ int s_count[2];
    __shared__ int s_abort;
    __shared__ uint32_t s_tmem;
    unsigned char *s_mem = s_raw + (-smem_u32(s_raw) & 1023);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t full = smem_u32(s_bar), empty = full + 8 * NS, tfull = empty + 8 * NS, tempty = tfull + 16;
    const uint32_t dfull = tempty + 16, dempty = dfull + 16;
    if (threadIdx.x == 0) {
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
    pdl_wait();
    if (warp == 0) count_tiles(p, s_count);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = s_tmem;
    const int r = p.rank;
    const Walk w = make_walk(s_count[0], (p.in + kCols - 1) / kCols, blockIdx.x, gridDim.x);
    volatile int *abort_flag = &s_abort;

    int i = 0, seg = 0;                              // steps and tiles so far
    for (long long u = w.u0; u < w.u1; ++seg) {
        const int tile = int(u / w.per), k0 = int(u - (long long)tile * w.per);
        const int n_steps = int(w.u1 - u < w.per - k0 ? w.u1 - u : w.per - k0);
        u += n_steps;
        if (!tile_ready(p, s_tiles, seg, tile, tfull, tempty, warp == kEpiWarps, abort_flag)) break;
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
                if (!__all_sync(0xffffffffu, ok)) break;
                unsigned char *xs = s_mem + s * S::kStage;
                stage_rows(t, xs, src, mine, col, n, p.vec_in);
                stage_weights<RP, !TRANS>(t, smem_u32(xs) + 2 * kBlock, wt, r, p.in, col, n);
                stage_done(full + 8 * s, p.vec_in);
            }
        } else if (warp == kMmaWarp) {
            constexpr uint32_t idesc = tc_idesc_bf16(kTile, RP) | (TRANS ? kTcBMajorN : 0);
            const uint32_t d = tmem + (seg & 1) * 128;
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
                        tc_mma_ss(d, a, b, idesc, k > 0 || m > 0);
                    }
                    tc_commit(empty + 8 * s);
                }
                __syncwarp();
            }
            if (elect_one()) tc_commit(dfull + 8 * (seg & 1));
            __syncwarp();
        } else {
            // this run's sum over the tile's columns, to its slot
            const int sub = warp % 4, half = warp / 4, row = 32 * sub + lane;
            const bool ok = __all_sync(0xffffffffu, mbar_wait(dfull + 8 * (seg & 1), (seg >> 1) & 1, abort_flag, p.err));
            tc_fence_after();
            float *out = p.partial + ((long long)(tile + blockIdx.x) * kTile + row) * RP + half * (RP / 2);
            #pragma unroll
            for (int k = 0; k < RP / 16; ++k) {
                uint32_t v[8];
                tc_ld_32x32b_x8(tmem + (uint32_t(32 * sub) << 16) + (seg & 1) * 128 + half * (RP / 2) + 8 * k, v);
                tc_wait_ld();
                if (!ok || *abort_flag) {
                    #pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = 0x7fffffffu;
                }
                if (row < count) {
                    *reinterpret_cast<uint4 *>(out + 8 * k) = make_uint4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<uint4 *>(out + 8 * k + 4) = make_uint4(v[4], v[5], v[6], v[7]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(dempty + 8 * (seg & 1));
        }
        tile_done(seg, tempty);
    }
    cp_async_wait_all();
    if (warp == kMmaWarp && seg > 0) drain_wait(dfull + 8 * ((seg - 1) & 1), ((seg - 1) >> 1) & 1);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tc_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ its sums
// h of every tile: its slots in CTA order, to the planes p.pg (scaled) and
// p.hidden; in the gradient also s h's planes from p.hidden.  Four ranks a
// thread, all of a tile's slots (5 of them at 4096 tokens) on their way at once.
constexpr int kSumThreads = 256;

template <int RP, bool TRANS>
__global__ void __launch_bounds__(kSumThreads) lora_sum_kernel(const LoraArgs p, int down_ctas) {
    constexpr int kPieces = RP / 4, kRows = kSumThreads / kPieces, kBlocks = kTile / kRows, kSlots = 8;
    __shared__ int s_rows[kTile];
    __shared__ int s_info[3], s_count[2];
    // The first product's CTAs let this kernel start after the sort had ended.
    pdl_launch_dependents();
    const int tile = blockIdx.x / kBlocks, row0 = blockIdx.x % kBlocks * kRows;
    if (threadIdx.x < 32) {
        count_tiles(p, s_count);
        find_tile_sorted<kTile>(p, tile, s_rows, s_info);
    }
    __syncthreads();
    const int adapter = s_info[0], count = s_info[1], r = p.rank;
    const int row = row0 + threadIdx.x / kPieces, rank = 4 * (threadIdx.x % kPieces);
    pdl_wait();
    if (row >= count) return;
    float4 *hidden = reinterpret_cast<float4 *>(p.hidden + (long long)s_rows[row] * r + rank);
    if (adapter < 0) {
        if (!TRANS && p.hidden && rank < r) *hidden = make_float4(0.f, 0.f, 0.f, 0.f);
        return;
    }
    const Walk d = make_walk(s_count[0], (p.in + kCols - 1) / kCols, 0, down_ctas);
    const long long first = (long long)tile * d.per;
    const int b0 = run_owner(d.units, d.ctas, first), b1 = run_owner(d.units, d.ctas, first + d.per - 1);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f), w = v;
    if (TRANS && rank < r) w = *hidden;
    const float *at = p.partial + ((long long)(tile + b0) * kTile + row) * RP + rank;
    for (int b = b0; b <= b1; b += kSlots) {
        float4 u[kSlots];
        #pragma unroll
        for (int k = 0; k < kSlots; ++k)
            if (b + k <= b1) u[k] = *reinterpret_cast<const float4 *>(at + (long long)(b - b0 + k) * kTile * RP);
        #pragma unroll
        for (int k = 0; k < kSlots; ++k)
            if (b + k <= b1) v.x += u[k].x, v.y += u[k].y, v.z += u[k].z, v.w += u[k].w;
    }
    if (!TRANS && p.hidden && rank < r) *hidden = v;
    if (rank >= r) v = make_float4(0.f, 0.f, 0.f, 0.f);  // also where x holds infinities (0 * inf)
    const float scale = p.scale[adapter];
    const long long out = (long long)(s_info[2] + row) * (plane_pitch(RP) / 2) + rank;
    uint2 hi, lo;
    split2(scale * v.x, scale * v.y, hi.x, lo.x), split2(scale * v.z, scale * v.w, hi.y, lo.y);
    *reinterpret_cast<uint2 *>(p.pg + out) = hi, *reinterpret_cast<uint2 *>(p.pg + out + RP) = lo;
    if (TRANS) {
        split2(scale * w.x, scale * w.y, hi.x, lo.x), split2(scale * w.z, scale * w.w, hi.y, lo.y);
        *reinterpret_cast<uint2 *>(p.ph + out) = hi, *reinterpret_cast<uint2 *>(p.ph + out + RP) = lo;
    }
}

// ----------------------------------------------------------- second product
template <int RP, bool TRANS>
struct UpShape {
    static constexpr int kW = weight_bytes(RP, TRANS);
    static constexpr int kStage = 2 * kBlock + kW;
    static constexpr int kH = 2 * plane_bytes(RP);
    static constexpr int kStages = (kSmemMax - 1024 - kH) / kStage < 5 ? (kSmemMax - 1024 - kH) / kStage : 5;
    static constexpr int kSmem = kStages * kStage + kH + 1024;
    static_assert(kStages >= 2, "the ring does not fit");
};

template <int RP, bool TRANS>
__global__ void __launch_bounds__(kThreads, 1) lora_up_kernel(const LoraArgs p) {
    using S = UpShape<RP, TRANS>;
    constexpr int NS = S::kStages, KS = RP / 16;
    extern __shared__ unsigned char s_raw[];
    __shared__ uint64_t s_bar[2 * NS + 13];
    __shared__ TileSlots s_tiles;
    __shared__ int s_count[2];
    __shared__ int s_abort;
    __shared__ uint32_t s_tmem;
    unsigned char *s_mem = s_raw + (-smem_u32(s_raw) & 1023);
    unsigned char *s_hi = s_mem + NS * S::kStage, *s_lo = s_hi + plane_bytes(RP);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t full = smem_u32(s_bar), empty = full + 8 * NS, tfull = empty + 8 * NS, tempty = tfull + 16;
    const uint32_t dfull = tempty + 16, dempty = dfull + 32, hready = dempty + 32;
    if (threadIdx.x == 0) {
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
    // The first product's CTAs had waited for what came before them when they let
    // the sums start, and those this kernel: the sort, base and the weights may be
    // read at once; only h (read by the epilogue) and what overwrites anything wait.
    if (warp == 0) count_tiles(p, s_count);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int r = p.rank;
    const Walk w = make_walk(s_count[0] + s_count[1], (p.out + kCols - 1) / kCols, blockIdx.x, gridDim.x);
    volatile int *abort_flag = &s_abort;

    // steps, tiles, multiplied tiles; step i multiplies into buffer i % 4 of D2
    int i = 0, seg = 0, h_seg = 0;
    uint32_t uses = 0;                               // a bit per buffer: the parity of its next use
    uint32_t used = 0;
    for (long long u = w.u0; u < w.u1; ++seg) {
        const int tile = int(u / w.per), k0 = int(u - (long long)tile * w.per);
        const int n_steps = int(w.u1 - u < w.per - k0 ? w.u1 - u : w.per - k0);
        u += n_steps;
        if (!tile_ready(p, s_tiles, seg, tile, tfull, tempty, warp == kEpiWarps, abort_flag)) break;
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
                if (!__all_sync(0xffffffffu, ok)) break;
                unsigned char *xs = s_mem + s * S::kStage;
                stage_rows(t, xs, src, mine, col, n, p.vec_out);
                if (adapter >= 0) stage_weights<RP, TRANS>(t, smem_u32(xs) + 2 * kBlock, wt, r, p.out, col, n);
                stage_done(full + 8 * s, p.vec_out);
            }
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
                        for (int part = 0; part < 2; ++part)     // the low plane first
                            #pragma unroll
                            for (int m = 0; m < KS; ++m) {
                                const uint32_t at = (m / 4) * kBlock + (m % 4) * 32;
                                const uint64_t a = tc_sdesc_sw128(smem_u32(part ? s_hi : s_lo) + at);
                                const uint64_t b = TRANS ? tc_sdesc_sw128_mn(ws + m * 2048, RP * 128)
                                                         : tc_sdesc_sw128(ws + at);
                                tc_mma_ss(tmem + buf * kCols, a, b, idesc, part > 0 || m > 0);
                            }
                        tc_commit(dfull + 8 * buf);
                    }
                    __syncwarp();
                }
            } else if (!in_place) {
                i += n_steps;
            }
        } else {
            // Two groups of four warps take the steps in turn, two buffers of D2 each (with
            // one the MMA's latency stood in the way: 2650 cycles a step, with two 2300 --
            // see the figures above); a warp has 32 rows.
            const int sub = warp % 4, group = warp / 4, my_row = 32 * sub + lane;
            bool bad = false;
            if (seg == 0) pdl_wait();
            else epi_sync();                         // the MMAs of the tile before have ended
            if (adapter >= 0) {
                // h's planes of the tile; rows past its tokens are zeros
                const int start = s_tiles.info[seg & 1][2];
                constexpr int kPieces = RP / 4, kOnce = RP >= 64 ? 8 : RP / 8;
                #pragma unroll 1
                for (int m0 = threadIdx.x; m0 < kTile * kPieces; m0 += kOnce * kEpiThreads) {
                    uint4 v[kOnce];
                    #pragma unroll
                    for (int e = 0; e < kOnce; ++e) {
                        const int m = m0 + e * kEpiThreads, row = m / kPieces, b = m % kPieces;
                        v[e] = make_uint4(0, 0, 0, 0);
                        if (row < count)
                            v[e] = *(reinterpret_cast<const uint4 *>(p.pg + (long long)(start + row) * (plane_pitch(RP) / 2)) + b);
                    }
                    #pragma unroll
                    for (int e = 0; e < kOnce; ++e) {
                        const int m = m0 + e * kEpiThreads, row = m / kPieces, b = m % kPieces, q = b % (RP / 8);
                        *reinterpret_cast<uint4 *>((b < RP / 8 ? s_hi : s_lo) + (q / 8) * kBlock + sw128(row, q % 8)) = v[e];
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
                bad |= !__all_sync(0xffffffffu, ok);
                #pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const int col = (k0 + k) * kCols + 64 * half;
                    if (col >= p.out || 32 * sub >= count) break;
                    unsigned char *bs = s_mem + s * S::kStage + half * kBlock;
                    if (adapter >= 0 && !bad) {
                        uint32_t acc[2][32];
                        tc_ld_32x32b_x32(lanes + 64 * half, acc[0]);
                        tc_ld_32x32b_x32(lanes + 64 * half + 32, acc[1]);
                        tc_wait_ld();
                        #pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            uint4 *at = reinterpret_cast<uint4 *>(bs + sw128(my_row, q));
                            uint4 b = make_uint4(0, 0, 0, 0);
                            if (p.base) b = *at;
                            const uint32_t *d = &acc[q / 4][8 * (q % 4)];
                            uint4 v;
                            v.x = pack_bf16x2_rn(bf16_lo_to_f32(b.x) + __uint_as_float(d[0]), bf16_hi_to_f32(b.x) + __uint_as_float(d[1]));
                            v.y = pack_bf16x2_rn(bf16_lo_to_f32(b.y) + __uint_as_float(d[2]), bf16_hi_to_f32(b.y) + __uint_as_float(d[3]));
                            v.z = pack_bf16x2_rn(bf16_lo_to_f32(b.z) + __uint_as_float(d[4]), bf16_hi_to_f32(b.z) + __uint_as_float(d[5]));
                            v.w = pack_bf16x2_rn(bf16_lo_to_f32(b.w) + __uint_as_float(d[6]), bf16_hi_to_f32(b.w) + __uint_as_float(d[7]));
                            *at = v;
                        }
                    } else if (bad || !p.base) {
                        const uint32_t fill = bad ? 0x7fff7fffu : 0u;
                        #pragma unroll
                        for (int q = 0; q < 8; ++q)
                            *reinterpret_cast<uint4 *>(bs + sw128(my_row, q)) = make_uint4(fill, fill, fill, fill);
                    }
                    __syncwarp();
                    #pragma unroll
                    for (int m = 0; m < 8; ++m) {
                        const int row = 32 * sub + 4 * m + lane / 8, q = lane % 8;
                        if (row < count) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(bs + sw128(row, q));
                            store_cols8(p.y + (long long)rows[row] * p.out + col + 8 * q, p.out - col - 8 * q, p.vec_out, v);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (adapter >= 0) mbar_arrive(dempty + 8 * (i & 3));
                    mbar_arrive(empty + 8 * s);
                }
            }
        }
        tile_done(seg, tempty);
    }
    pdl_wait();
    pdl_launch_dependents();
    cp_async_wait_all();
    if (warp == kMmaWarp)
        for (int buf = 0; buf < 4; ++buf)
            if ((used >> buf) & 1) drain_wait(dfull + 8 * buf, (~uses >> buf) & 1);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tc_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------- weight gradients
constexpr int kStageTokens = 32;
// Eight warps produce and then store; the ninth issues the MMAs.
constexpr int kWgradWarps = 8, kWgradProducers = kWgradWarps * 32, kWgradThreads = kWgradProducers + 32;

template <int RP>
struct WgradShape {
    static constexpr int kCols = RP <= 64 ? 512 : 256;      // columns of a CTA
    static constexpr int kQBlock = kStageTokens * 128;      // bytes of 32 tokens x 64 columns
    static constexpr int kQ = kCols / 64 * kQBlock;
    static constexpr int kP = (2 * RP + 63) / 64 * kQBlock; // both planes: rows of 2 RP, in blocks of 64
    static constexpr int kStage = kQ + kP;
    static constexpr int kSumsA = RP * (kCols + 4) * 4, kSumsB = kCols * (RP + 4) * 4;
    static constexpr int kSums = kSumsA > kSumsB ? kSumsA : kSumsB;
    static constexpr int kStages = (kSmemMax - 1024) / kStage;
    static constexpr int kSmem = kStages * kStage + 1024;
    static_assert(kStages >= 2 && kSums <= kStages * kStage, "the ring does not fit");
};

// Grid (slices * cluster, adapters): a cluster owns kCols columns of one
// adapter's dA (or rows of dB), D[column][rank] in TMEM in blocks of 128
// columns, once for each plane of g or s h (one MMA takes both as its N; two of
// half the N took twice the time); its CTAs split the adapter's tokens, 32 to a stage, and add their
// sums through distributed shared memory, in CTA order.
template <int RP, bool DB>
__device__ __forceinline__ void wgrad_tile(const WgradArgs &p, int slice, int adapter, unsigned char *s_mem,
                                           uint64_t *s_bar, int *s_abort, uint32_t tmem) {
    using S = WgradShape<RP>;
    constexpr int NS = S::kStages;
    const uint16_t *q = DB ? p.dy : p.x, *planes = DB ? p.ph : p.pg;
    const int cols = DB ? p.N : p.K, vec = DB ? p.vec_dy : p.vec_x, r = p.rank;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int C = cluster_size(), c = cluster_rank();
    const uint32_t ring = smem_u32(s_mem), full = smem_u32(s_bar), empty = full + 8 * NS, dfull = empty + 8 * NS;
    int start = 0;
    for (int a = lane; a < adapter; a += 32) start += p.sizes[a];
    start = __reduce_add_sync(0xffffffffu, start);
    const int size = p.sizes[adapter];
    const int blocks = (size + kStageTokens - 1) / kStageTokens;
    const int t0 = kStageTokens * int((long long)blocks * c / C);
    const int t1 = min(size, kStageTokens * int((long long)blocks * (c + 1) / C));
    const int stages = t1 > t0 ? (t1 - t0 + kStageTokens - 1) / kStageTokens : 0;
    const int col0 = slice * S::kCols, width = min(S::kCols, cols - col0);
    const int *rows = p.order + start;
    volatile int *abort_flag = s_abort;

    if (warp < kWgradWarps) {
        // Rows row0 + 16 j, column pieces piece + 16 e: their places are 2048 bytes and
        // 2 blocks apart.  The rows of the next stage are looked up one stage ahead.
        const int pt = threadIdx.x, piece = pt % 16, row0 = pt / 16;
        constexpr int kRows = kWgradProducers / 16, kJ = kStageTokens / kRows, kE = S::kCols / 128;
        const uint32_t dst = (piece / 8) * S::kQBlock + sw128(row0, piece % 8);
        int next[kJ];
        #pragma unroll
        for (int j = 0; j < kJ; ++j) next[j] = t0 + row0 + kRows * j < t1 ? rows[t0 + row0 + kRows * j] : -1;
        for (int i = 0; i < stages; ++i) {
            const int s = i % NS, tok = t0 + i * kStageTokens, n = min(kStageTokens, t1 - tok);
            int row[kJ];
            #pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const int t = tok + kStageTokens + row0 + kRows * j;
                row[j] = next[j];
                next[j] = t < t1 ? rows[t] : -1;
            }
            const bool ok = i < NS || mbar_wait(empty + 8 * s, (i / NS - 1) & 1, abort_flag, p.err);
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint32_t qs = ring + s * S::kStage, ps = qs + S::kQ;
            // tokens past the end are zeros on both sides: they are summed over
            #pragma unroll
            for (int j = 0; j < kJ; ++j) {
                const bool in = row[j] >= 0;
                const uint16_t *src = q + (long long)max(row[j], 0) * cols + col0 + 8 * piece;
                #pragma unroll
                for (int e = 0; e < kE; ++e) {
                    const int left = width - 8 * piece - 128 * e;
                    const uint32_t at = dst + kRows * 128 * j + 2 * S::kQBlock * e;
                    if (left <= 0) continue;
                    if (vec) cp_async16z(qs + at, in ? src + 128 * e : q, in);
                    else *reinterpret_cast<uint4 *>(s_mem + s * S::kStage + at) = load_cols8(src + 128 * e, in ? left : 0, 0);
                }
            }
            constexpr int kPieces = RP / 4, kAll = kStageTokens * kPieces;   // both planes' pieces
            const uint16_t *src = planes + (long long)(start + tok) * (plane_pitch(RP) / 2);
            #pragma unroll
            for (int k = pt; k < kAll; k += kWgradProducers) {
                const int tk = k / kPieces, b = k % kPieces;
                const bool in = tk < n;
                cp_async16z(ps + (b / 8) * S::kQBlock + sw128(tk, b % 8), in ? src + 8 * k : planes, in);
            }
            stage_done(full + 8 * s, vec);
        }
        cp_async_wait_all();
    } else {
        constexpr uint32_t idesc = tc_idesc_bf16(128, 2 * RP) | kTcAMajorM | kTcBMajorN;
        bool ok = true;
        for (int i = 0; i < stages; ++i) {
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
                    for (int k = 0; k < kStageTokens / 16; ++k) {
                        const uint64_t a = tc_sdesc_sw128_mn(qs + m * 2 * S::kQBlock + k * 2048, S::kQBlock);
                        const uint64_t b = tc_sdesc_sw128_mn(ps + k * 2048, S::kQBlock);
                        tc_mma_ss(tmem + m * 2 * RP, a, b, idesc, i > 0 || k > 0);
                    }
                tc_commit(empty + 8 * s);
            }
            __syncwarp();
        }
        if (elect_one()) tc_commit(dfull);
        __syncwarp();
        drain_wait(dfull, 0);
    }
    // ---- sums: the tile as it will be stored, in fp32, where the ring was
    tc_fence_before();
    __syncthreads();                                             // every copy and MMA has ended
    tc_fence_after();
    const bool bad = *abort_flag != 0;
    float *s_sum = reinterpret_cast<float *>(s_mem);
    constexpr int kPitch = DB ? RP + 4 : S::kCols + 4;
    if (warp < kWgradWarps) {
        const int sub = warp % 4;
        for (int m = warp / 4; m < S::kCols / 128; m += 2) {
            const int col = 128 * m + 32 * sub + lane;
            #pragma unroll 2
            for (int k = 0; k < RP / 8; ++k) {
                uint32_t v[8], w[8];
                if (stages > 0 && !bad) {
                    const uint32_t at = tmem + (uint32_t(32 * sub) << 16) + m * 2 * RP + 8 * k;
                    tc_ld_32x32b_x8(at, v);
                    tc_ld_32x32b_x8(at + RP, w);
                    tc_wait_ld();
                    #pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) + __uint_as_float(w[e]));
                } else {
                    #pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = bad ? 0x7fffffffu : 0u;
                }
                if (DB) {
                    float *d = s_sum + col * kPitch + 8 * k;
                    *reinterpret_cast<uint4 *>(d) = make_uint4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<uint4 *>(d + 4) = make_uint4(v[4], v[5], v[6], v[7]);
                } else {
                    #pragma unroll
                    for (int e = 0; e < 8; ++e) s_sum[(8 * k + e) * kPitch + col] = __uint_as_float(v[e]);
                }
            }
        }
    }
    __syncthreads();
    if (C > 1) {
        cluster_arrive();
        cluster_wait();
    }
    const int n_rows = DB ? width : r, per = (DB ? r : width) / 8;   // rows, 8-element pieces of one
    const int items = n_rows * per;
    const int i0 = int((long long)items * c / C), i1 = int((long long)items * (c + 1) / C);
    for (int i = i0 + threadIdx.x; i < i1; i += kWgradThreads) {
        const int row = i / per, col = 8 * (i % per);
        const float *at = s_sum + row * kPitch + col;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (C > 1) {
            for (int k0 = 0; k0 < C; k0 += 4) {          // clusters of 2, 4 or 8
                float4 x[4], y[4];
                #pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k0 + k < C) x[k] = ld_cluster4(at, k0 + k), y[k] = ld_cluster4(at + 4, k0 + k);
                #pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k0 + k < C) {
                        a.x += x[k].x, a.y += x[k].y, a.z += x[k].z, a.w += x[k].w;
                        b.x += y[k].x, b.y += y[k].y, b.z += y[k].z, b.w += y[k].w;
                    }
            }
        } else {
            a = *reinterpret_cast<const float4 *>(at), b = *reinterpret_cast<const float4 *>(at + 4);
        }
        uint4 o;
        o.x = pack_bf16x2_rn(a.x, a.y), o.y = pack_bf16x2_rn(a.z, a.w);
        o.z = pack_bf16x2_rn(b.x, b.y), o.w = pack_bf16x2_rn(b.z, b.w);
        uint16_t *d = DB ? p.db + ((long long)adapter * cols + col0 + row) * r + col
                         : p.da + ((long long)adapter * r + row) * cols + col0 + col;
        *reinterpret_cast<uint4 *>(d) = o;
    }
    if (C > 1) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    }
}

template <int RP>
__global__ void __launch_bounds__(kWgradThreads, 1) lora_wgrad_kernel(const WgradArgs p) {
    using S = WgradShape<RP>;
    constexpr int NS = S::kStages;
    extern __shared__ unsigned char s_raw[];
    __shared__ uint64_t s_bar[2 * NS + 1];
    __shared__ int s_abort;
    __shared__ uint32_t s_tmem;
    unsigned char *s_mem = s_raw + (-smem_u32(s_raw) & 1023);
    const int warp = threadIdx.x / 32;
    if (threadIdx.x == 0) {
        const uint32_t bar = smem_u32(s_bar);
        for (int i = 0; i < NS; ++i) mbar_init(bar + 8 * i, kWgradProducers), mbar_init(bar + 8 * (NS + i), 1);
        mbar_init(bar + 16 * NS, 1);
        s_abort = 0;
        fence_barrier_init();
    }
    if (warp == kWgradWarps) {
        tc_alloc(smem_u32(&s_tmem), kTmemCols);
        tc_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    pdl_launch_dependents();
    pdl_wait();
    const int slice = blockIdx.x / cluster_size();
    if (slice < p.slices_x) wgrad_tile<RP, false>(p, slice, blockIdx.y, s_mem, s_bar, &s_abort, tmem);
    else wgrad_tile<RP, true>(p, slice - p.slices_x, blockIdx.y, s_mem, s_bar, &s_abort, tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWgradWarps) tc_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------- host side
int ceil_div(long long a, long long b) { return int((a + b - 1) / b); }

// Tiles at most: the adapters' and the adapterless tokens' last may be part empty.
int lora_max_tiles(int tokens, int adapters) {
    return ceil_div(tokens, kTile) + (adapters < tokens ? adapters : tokens);
}

template <int RP, bool TRANS>
cudaError_t launch_tensor_rank(const LoraArgs &p, int sms, cudaStream_t s) {
    using D = DownShape<RP, TRANS>;
    using U = UpShape<RP, TRANS>;
    cudaError_t e = allow_smem<lora_down_kernel<RP, TRANS>>(D::kSmem);
    if (e == cudaSuccess) e = allow_smem<lora_up_kernel<RP, TRANS>>(U::kSmem);
    if (e != cudaSuccess) return e;
    const int ctas = sms < kMaxRuns ? sms : kMaxRuns;
    e = launch_chained(lora_down_kernel<RP, TRANS>, dim3(ctas), kThreads, D::kSmem, 1, s, p);
    if (e != cudaSuccess) return e;
    const int blocks = lora_max_tiles(p.tokens, p.adapters) * (kTile * (RP / 4) / kSumThreads);
    e = launch_chained(lora_sum_kernel<RP, TRANS>, dim3(blocks), kSumThreads, 0, 1, s, p, ctas);
    if (e != cudaSuccess) return e;
    return launch_chained(lora_up_kernel<RP, TRANS>, dim3(ctas), kThreads, U::kSmem, 1, s, p);
}

template <int RP>
cudaError_t launch_wgrad_rank(WgradArgs p, int adapters, int sms, cudaStream_t s) {
    using S = WgradShape<RP>;
    const cudaError_t e = allow_smem<lora_wgrad_kernel<RP>>(S::kSmem);
    if (e != cudaSuccess) return e;
    p.slices_x = ceil_div(p.K, S::kCols);
    const int slices = p.slices_x + ceil_div(p.N, S::kCols);
    int cluster = 1;
    while (cluster < kMaxCluster && 2LL * slices * adapters * cluster <= sms) cluster *= 2;
    return launch_chained(lora_wgrad_kernel<RP>, dim3(slices * cluster, adapters), kWgradThreads, S::kSmem, cluster, s, p);
}

}  // namespace

size_t lora_partial_bytes(int tokens, int adapters, int rank) {
    return (size_t(lora_max_tiles(tokens, adapters)) + kMaxRuns) * kTile * padded_rank(rank) * sizeof(float);
}

cudaError_t launch_lora_tensor(const LoraArgs &p, bool trans, int sms, cudaStream_t s) {
    switch (padded_rank(p.rank)) {
        case 16: return trans ? launch_tensor_rank<16, true>(p, sms, s) : launch_tensor_rank<16, false>(p, sms, s);
        case 32: return trans ? launch_tensor_rank<32, true>(p, sms, s) : launch_tensor_rank<32, false>(p, sms, s);
        case 64: return trans ? launch_tensor_rank<64, true>(p, sms, s) : launch_tensor_rank<64, false>(p, sms, s);
        default: return trans ? launch_tensor_rank<128, true>(p, sms, s) : launch_tensor_rank<128, false>(p, sms, s);
    }
}

cudaError_t launch_wgrad(const WgradArgs &p, int adapters, int sms, cudaStream_t s) {
    switch (padded_rank(p.rank)) {
        case 16: return launch_wgrad_rank<16>(p, adapters, sms, s);
        case 32: return launch_wgrad_rank<32>(p, adapters, sms, s);
        case 64: return launch_wgrad_rank<64>(p, adapters, sms, s);
        default: return launch_wgrad_rank<128>(p, adapters, sms, s);
    }
}

}  // namespace w4a16
