// lora.cu -- low-rank adapters of many requests beside a shared projection.
//
// Token t with adapter a = ids[t] (outside [0, L): none):
//   h[t] = A_a x[t],  y[t] = base[t] + s_a B_a h[t]          A [r][K], B [N][r]
// and the gradients, with g[t] = s_a B_a^T dy[t],
//   dx[t] = dx_base[t] + A_a^T g[t],  dA_a = sum_t g[t] x[t]^T,
//   dB_a = s_a sum_t dy[t] h[t]^T     (sums over the adapter's tokens).
// y and dx are one computation: a product down to the rank, then one up to the
// output, with the weights read along the other axis.  lora_kernel does both in
// one launch: a cluster of CTAs owns a tile of tokens of one adapter, its CTAs
// split the input columns, add their partial h through distributed shared
// memory in CTA order, and split the output columns.  A producer warp streams
// everything (rows of X and base, wherever the tokens stand, and the weights)
// through one ring of bulk copies, running ahead across the turn from the first
// product to the second.  In the first product the order of k inside an MMA is
// free as long as both operands agree, so a lane takes 16 bytes of a row, and
// 32 columns of a row feed two MMAs; where a weight lies along the wrong axis
// its 8 x 8 blocks are transposed in registers.
//
// Precision: products of bf16 are exact in the MMA and summed in fp32; h (and g)
// stay in fp32 and enter the second product as a sum of two bf16 terms, which
// holds them to 2^-17.  The outputs are rounded once.
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "w4a16.h"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "lora.cuh"

namespace w4a16 {
namespace {

constexpr int kLoraWarps = 8;                       // consumer warps
constexpr int kLoraConsumers = kLoraWarps * 32;
constexpr int kLoraProducers = 128;                 // threads of the four producer warps
constexpr int kLoraThreads = kLoraConsumers + kLoraProducers;
constexpr int kLoraCols = 32;          // columns of a step: 16 bytes per lane of a quad
constexpr int kChunkCols = 128;        // columns of a ring stage
constexpr int kRowBytes = kChunkCols * 2 + 64;   // of a staged row: two rows fill the banks
constexpr int kManyTile = 64;          // tokens of a cluster's tile
constexpr int kFewTile = 16;
constexpr int kFewTokens = 128;        // up to this many tokens clusters find their tiles in the ids
constexpr int kMaxRank = 128;

__device__ __forceinline__ uint32_t movm(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ void mma_acc(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    mma_16816_c(c, a, b0, b1, c);
}

// Moves registers from the producers to the consumers of a kernel launched
// with 168 a thread: 128 x 40 + 256 x 232 = 384 x 168.
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 40;"); }
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 232;"); }

__device__ __forceinline__ void consumer_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kLoraConsumers) : "memory");
}

__device__ __forceinline__ uint4 lds16(const unsigned char *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ uint2 lds8(const unsigned char *p) { return *reinterpret_cast<const uint2 *>(p); }

// How lora_kernel<RP, TM> divides its work and its shared memory.
template <int RP, int TM>
struct LoraShape {
    // Each ring stage is consumed by one group of four warps, the stages in
    // turn by the two groups.  First product: a group has RG row blocks of
    // 16 MT rows x KG warps that share the stage's four column steps.
    static constexpr int RG = TM == 64 && RP == 128 ? 2 : 1, KG = 4 / RG;
    static constexpr int MT = TM / 16 / RG;
    static constexpr int KW = 2 * KG;                   // partial sums of h
    static constexpr int NBUF = RP >= 64 && TM == 64 ? 2 : 4;   // held at once
    static constexpr int PS = RP + 4;                   // floats of a row of h
    static constexpr int kStage = (TM + RP) * kRowBytes;
    static constexpr int kSums = (NBUF + 1) * TM * PS * 4;
    // One CTA per SM for the 64-token tile, two (where that leaves three
    // stages) for the 16-token one.
    static constexpr int kRoom = (TM == 64 || RP >= 64 ? 226 : 112) * 1024 - kSums - 1024;
    static constexpr int kStages = kRoom / kStage < 12 ? kRoom / kStage : 12;
    static constexpr int kSmem = kStages * kStage + kSums;
    static_assert(kStages >= 2, "the ring does not fit");
};

// TRANS: weights along the other axis (the gradient).  RP: the rank rounded up
// to 16, 32, 64 or 128.  Staged rows past the tile's tokens and ranks past
// p.rank hold whatever the ring held: such rows are never stored, such ranks of h
// are set to zero and their weights in the second product too.
template <int RP, int TM, bool TRANS, bool FEW>
__global__ void __launch_bounds__(kLoraThreads, TM == 16 && RP <= 32 ? 2 : 1) lora_kernel(const LoraArgs p) {
    using S = LoraShape<RP, TM>;
    constexpr int MT = S::MT, RG = S::RG, KG = S::KG, PS = S::PS, NS = S::kStages;
    constexpr int NT = RP / 8;                           // 8-rank blocks
    constexpr int QN = RP >= 32 ? RP / 32 : 1;           // 32-rank blocks (one of 16)
    constexpr int JN = RP >= 32 ? 4 : 2;                 // 8-rank blocks of one
    extern __shared__ __align__(128) unsigned char s_mem[];
    float *s_part = reinterpret_cast<float *>(s_mem + NS * S::kStage);   // [NBUF][TM][PS]
    float *s_h = s_part + S::NBUF * TM * PS;                             // [TM][PS]
    __shared__ uint64_t s_bar[2 * NS + 2];               // full, empty, sums ready, sums read
    __shared__ int s_rows[TM];
    __shared__ int s_tile[3];
    __shared__ int s_abort;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int C = cluster_size(), c = cluster_rank();
    const uint32_t ring = smem_u32(s_mem), full = smem_u32(s_bar), empty = full + 8 * NS;
    const uint32_t ready = empty + 8 * NS, done = ready + 8;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) mbar_init(full + 8 * i, kLoraProducers), mbar_init(empty + 8 * i, 4);
        mbar_init(ready, C);
        mbar_init(done, C);
        s_abort = 0;
        fence_barrier_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) {
        if (FEW) find_tile_few<TM>(p, blockIdx.x / C, s_rows, s_tile);
        else find_tile_sorted<TM>(p, blockIdx.x / C, s_rows, s_tile);
    }
    __syncthreads();
    const int adapter = s_tile[0], count = s_tile[1];
    if (count == 0) return;                              // the same in every CTA of the cluster
    if (adapter < 0) {
        // no adapter: y = base, h = 0
        if (p.y != p.base) {
            const int items = (p.out + 7) / 8;
            const int i0 = int((long long)items * c / C), i1 = int((long long)items * (c + 1) / C);
            for (int r = warp; r < count; r += kLoraThreads / 32) {
                const long long at = (long long)s_rows[r] * p.out;
                #pragma unroll 4
                for (int i = i0 + lane; i < i1; i += 32) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (p.base) v = load_cols8(p.base + at + 8 * i, p.out - 8 * i, p.vec_out);
                    store_cols8(p.y + at + 8 * i, p.out - 8 * i, p.vec_out, v);
                }
            }
        }
        if (!TRANS && p.hidden && c == 0)
            for (int i = threadIdx.x; i < count * p.rank; i += kLoraThreads)
                p.hidden[(long long)s_rows[i / p.rank] * p.rank + i % p.rank] = 0.f;
        return;
    }
    if (C > 1) cluster_arrive();                         // barriers initialised

    const int r = p.rank;
    const int kin = (p.in + kChunkCols - 1) / kChunkCols, kout = (p.out + kChunkCols - 1) / kChunkCols;
    const int in0 = int((long long)kin * c / C), out0 = int((long long)kout * c / C);
    const int nin = int((long long)kin * (c + 1) / C) - in0;
    const int nall = nin + int((long long)kout * (c + 1) / C) - out0;
    volatile int *abort_flag = &s_abort;

    if (warp >= kLoraWarps) {
        // ---- producers: the stages of both products in order
        if (RP >= 64 && TM == 64) regs_down();
        const uint16_t *w1 = p.w1 + (long long)adapter * r * p.in, *w2 = p.w2 + (long long)adapter * r * p.out;
        const int pt = threadIdx.x - kLoraConsumers, piece = pt % (kChunkCols / 8), row0 = pt / (kChunkCols / 8);
        constexpr int kRows = kLoraProducers / (kChunkCols / 8);   // rows in one go
        for (int i = 0; i < nall; ++i) {
            const int s = i % NS;
            const bool ok = i < NS || mbar_wait(empty + 8 * s, (i / NS - 1) & 1, abort_flag, p.err);
            if (!__all_sync(0xffffffffu, ok)) break;
            const bool first = i < nin;
            const int cols = first ? p.in : p.out, col = (first ? in0 + i : out0 + i - nin) * kChunkCols;
            const int n = min(kChunkCols, cols - col), vec = first ? p.vec_in : p.vec_out;
            const uint16_t *rows = first ? p.x : p.base, *w = first ? w1 : w2;
            unsigned char *xs = s_mem + s * S::kStage, *ws = xs + TM * kRowBytes;
            if (8 * piece < n) {
                if (rows) {
                    #pragma unroll 4
                    for (int k = row0; k < count; k += kRows)
                        stage_piece(xs + k * kRowBytes + 16 * piece,
                                    rows + (long long)s_rows[k] * cols + col + 8 * piece, n - 8 * piece, vec);
                }
                if (first != TRANS) {                    // [r][cols]: a piece of each rank's row
                    #pragma unroll 4
                    for (int k = row0; k < r; k += kRows)
                        cp_async16(smem_u32(ws + k * kRowBytes + 16 * piece),
                                   w + (long long)k * cols + col + 8 * piece);
                }
            }
            if (first == TRANS) {                        // [cols][r]: contiguous
                const uint16_t *src = w + (long long)col * r;
                #pragma unroll 4
                for (int k = pt; k < n * r / 8; k += kLoraProducers) cp_async16(smem_u32(ws + 16 * k), src + 8 * k);
            }
            stage_done(full + 8 * s, vec);
        }
        cp_async_wait_all();
        __syncwarp();
        if (C > 1) cluster_wait();
        return;
    }
    if (RP >= 64 && TM == 64) regs_up();

    bool bad = false;
    const int group = warp / 4, gw = warp % 4;
    const float scale = p.scale[adapter];
    // ---- h: row block rg of 16 MT rows, steps kg, kg + KG, ... of the group's stages
    {
        const int rg = gw % RG, kg = gw / RG;
        float acc[MT][NT][4];
        #pragma unroll
        for (int m = 0; m < MT; ++m)
            #pragma unroll
            for (int n = 0; n < NT; ++n)
                #pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
        for (int i = group; i < nin; i += 2) {
            const int s = i % NS;
            bad |= !__all_sync(0xffffffffu, mbar_wait(full + 8 * s, (i / NS) & 1, abort_flag, p.err));
            const unsigned char *xs = s_mem + s * S::kStage, *ws = xs + TM * kRowBytes;
            const int col = (in0 + i) * kChunkCols;
            #pragma unroll
            for (int st = kg; st < kChunkCols / kLoraCols; st += KG) {
                const int c0 = col + st * kLoraCols;
                if (TRANS && c0 >= p.in) break;
                if (16 * MT * rg >= count) break;
                uint32_t w[TRANS ? RP / 2 : 1];
                if (TRANS) {
                    // B's rows of columns {8 (i/2) + 2 sh + i%2}, i = 0..7: the k slots
                    // of the MMAs (sh / 2) that x's 16-byte pieces fill
                    #pragma unroll
                    for (int sh = 0; sh < 4; ++sh) {
                        const int row = st * kLoraCols + 8 * (g >> 1) + 2 * sh + (g & 1);
                        const bool in = col + row < p.in;
                        #pragma unroll
                        for (int q = 0; q < QN; ++q) {
                            uint32_t *d = &w[(sh * QN + q) * JN];
                            if (RP >= 32) {
                                const uint4 v = lds16(ws + (row * r + 32 * q + 8 * t) * 2);
                                d[0] = in ? v.x : 0, d[1] = in ? v.y : 0, d[2] = in ? v.z : 0, d[3] = in ? v.w : 0;
                            } else {
                                const uint2 v = lds8(ws + (row * r + 4 * t) * 2);
                                d[0] = in ? v.x : 0, d[1] = in ? v.y : 0;
                            }
                        }
                    }
                }
                uint4 xv[MT][2];
                #pragma unroll
                for (int m = 0; m < MT; ++m)
                    #pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int row = 16 * (rg * MT + m) + 8 * h + g;
                        xv[m][h] = lds16(xs + row * kRowBytes + (st * kLoraCols + 8 * t) * 2);
                        if (TRANS && c0 + 8 * t >= p.in) xv[m][h] = make_uint4(0, 0, 0, 0);
                    }
                #pragma unroll
                for (int n = 0; n < NT; ++n) {
                    // A's row of rank 8n + g, columns 8t..8t+7
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (!TRANS) v = lds16(ws + (8 * n + g) * kRowBytes + (st * kLoraCols + 8 * t) * 2);
                    #pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t f0 = k ? v.z : v.x, f1 = k ? v.w : v.y;
                        if (TRANS) {
                            f0 = movm(w[(2 * k * QN + n / JN) * JN + n % JN]);
                            f1 = movm(w[((2 * k + 1) * QN + n / JN) * JN + n % JN]);
                        }
                        #pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const uint32_t a[4] = {k ? xv[m][0].z : xv[m][0].x, k ? xv[m][1].z : xv[m][1].x,
                                                   k ? xv[m][0].w : xv[m][0].y, k ? xv[m][1].w : xv[m][1].y};
                            mma_acc(acc[m][n], a, f0, f1);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * s);
        }
        // columns 2t, 2t+1 of block n hold these two neighbouring ranks; NBUF of the
        // KW partial sums are written at a time, the later ones added
        const int kw = group * KG + kg;
        #pragma unroll
        for (int round = 0; round < S::KW / S::NBUF; ++round) {
            if (kw / S::NBUF == round) {
                #pragma unroll
                for (int m = 0; m < MT; ++m)
                    #pragma unroll
                    for (int n = 0; n < NT; ++n)
                        #pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int rank = !TRANS ? 8 * n + 2 * t
                                                    : RP >= 32 ? 32 * (n / JN) + 8 * t + 2 * (n % JN) : 4 * t + 2 * n;
                            float2 *d = reinterpret_cast<float2 *>(
                                s_part + ((kw % S::NBUF) * TM + 16 * (rg * MT + m) + 8 * h + g) * PS + rank);
                            float2 v = make_float2(acc[m][n][2 * h], acc[m][n][2 * h + 1]);
                            if (round) {
                                const float2 u = *d;
                                v.x += u.x, v.y += u.y;
                            }
                            *d = v;
                        }
            }
            consumer_sync();
        }
    }
    constexpr int kQuads = RP / 4;
    for (int i = threadIdx.x; i < TM * kQuads; i += kLoraConsumers) {
        float *d = s_part + (i / kQuads) * PS + 4 * (i % kQuads);
        float4 v = *reinterpret_cast<const float4 *>(d);
        #pragma unroll
        for (int k = 1; k < S::NBUF; ++k) {
            const float4 u = *reinterpret_cast<const float4 *>(d + k * TM * PS);
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
        *reinterpret_cast<float4 *>(d) = v;
    }
    if (C > 1) {
        consumer_sync();
        cluster_wait();
        if (threadIdx.x < C) mbar_arrive_cluster(ready, threadIdx.x);
        bad |= !mbar_wait_cluster(ready, 0, abort_flag, p.err);
    }
    for (int i = threadIdx.x; i < TM * kQuads; i += kLoraConsumers) {
        const int row = i / kQuads, rank = 4 * (i % kQuads);
        const float *d = s_part + row * PS + rank;
        float4 v;
        if (C > 1) {
            v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < C; ++k) {
                const float4 u = ld_cluster4(d, k);
                v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
            }
        } else {
            v = *reinterpret_cast<const float4 *>(d);
        }
        // a rank past r is 0 also where x holds infinities (0 * inf)
        if (rank >= r) v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (bad) v.x = v.y = v.z = v.w = __int_as_float(0x7fffffff);
        const float4 s = make_float4(scale * v.x, scale * v.y, scale * v.z, scale * v.w);
        *reinterpret_cast<float4 *>(s_h + row * PS + rank) = s;
        if (c == 0 && row < count) {
            if (!TRANS && p.hidden && rank < r)
                *reinterpret_cast<float4 *>(p.hidden + (long long)s_rows[row] * r + rank) = v;
            if (TRANS) {
                // g and s h of the sorted token, for the weight gradients
                float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
                if (rank < r) h = *reinterpret_cast<const float4 *>(p.hidden + (long long)s_rows[row] * r + rank);
                const long long at = (long long)(s_tile[2] + row) * (plane_pitch(RP) / 2) + rank;
                uint2 hi, lo;
                split2(s.x, s.y, hi.x, lo.x), split2(s.z, s.w, hi.y, lo.y);
                *reinterpret_cast<uint2 *>(p.pg + at) = hi, *reinterpret_cast<uint2 *>(p.pg + at + RP) = lo;
                split2(scale * h.x, scale * h.y, hi.x, lo.x), split2(scale * h.z, scale * h.w, hi.y, lo.y);
                *reinterpret_cast<uint2 *>(p.ph + at) = hi, *reinterpret_cast<uint2 *>(p.ph + at + RP) = lo;
            }
        }
    }
    consumer_sync();
    if (C > 1 && threadIdx.x < C) mbar_arrive_cluster(done, threadIdx.x);   // has read the others' sums

    // ---- y: 16 rows x 32 columns at a time
    {
        constexpr int RG2 = TM / 16, CG2 = 4 / RG2, KS = RP / 16;
        const int rg = gw % RG2, cg = gw / RG2;
        uint32_t hi[KS][4], lo[KS][4];
        #pragma unroll
        for (int k = 0; k < KS; ++k)
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                // slots (2t, 2t+1) for i < 2, (2t+8, 2t+9) for i >= 2
                const int rank = TRANS ? 16 * k + 2 * t + 8 * (i / 2)
                                       : RP >= 32 ? 32 * (k / 2) + 8 * t + 4 * (k % 2) + 2 * (i / 2)
                                                  : 4 * t + 2 * (i / 2);
                const float2 v = *reinterpret_cast<const float2 *>(s_h + (16 * rg + g + 8 * (i % 2)) * PS + rank);
                split2(v.x, v.y, hi[k][i], lo[k][i]);
            }
        const int i0 = 16 * rg + g, i1 = i0 + 8;
        const long long row0 = i0 < count ? (long long)s_rows[i0] * p.out : -1;
        const long long row1 = i1 < count ? (long long)s_rows[i1] * p.out : -1;
        for (int i = nin + ((nin ^ group) & 1); i < nall; i += 2) {
            const int s = i % NS;
            bad |= !__all_sync(0xffffffffu, mbar_wait(full + 8 * s, (i / NS) & 1, abort_flag, p.err));
            const unsigned char *bs = s_mem + s * S::kStage, *ws = bs + TM * kRowBytes;
            const int col = (out0 + i - nin) * kChunkCols;
            #pragma unroll 1
            for (int st = cg; st < kChunkCols / kLoraCols; st += CG2) {
                const int mine = col + st * kLoraCols + 8 * t;
                if (col + st * kLoraCols >= p.out || 16 * rg >= count) break;
                uint4 base0 = make_uint4(0, 0, 0, 0), base1 = base0;
                if (p.base) {
                    base0 = lds16(bs + i0 * kRowBytes + (st * kLoraCols + 8 * t) * 2);
                    base1 = lds16(bs + i1 * kRowBytes + (st * kLoraCols + 8 * t) * 2);
                }
                uint32_t w[RP / 2];
                if (!TRANS) {
                    // B's rows of columns {8 (i/2) + 2 j + i%2}: a lane's results are 8 neighbours
                    #pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int row = st * kLoraCols + 8 * (g >> 1) + 2 * j + (g & 1);
                        #pragma unroll
                        for (int q = 0; q < QN; ++q) {
                            if (RP >= 32) {
                                const uint4 v = lds16(ws + (row * r + 32 * q + 8 * t) * 2);
                                const bool in = 32 * q + 8 * t < r;
                                uint32_t *d = &w[(j * QN + q) * 4];
                                d[0] = in ? v.x : 0, d[1] = in ? v.y : 0, d[2] = in ? v.z : 0, d[3] = in ? v.w : 0;
                            } else {
                                const uint2 v = lds8(ws + (row * r + 4 * t) * 2);
                                const bool in = 4 * t < r;
                                w[2 * j] = in ? v.x : 0, w[2 * j + 1] = in ? v.y : 0;
                            }
                        }
                    }
                } else {
                    #pragma unroll
                    for (int k = 0; k < 2 * KS; ++k) {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (8 * k < r) v = lds16(ws + (8 * k + g) * kRowBytes + (st * kLoraCols + 8 * t) * 2);
                        w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
                    }
                }
                float acc[4][4];
                #pragma unroll
                for (int j = 0; j < 4; ++j)
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
                #pragma unroll
                for (int k = 0; k < KS; ++k)
                    #pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t f0, f1;
                        if (TRANS) {
                            f0 = movm(w[4 * (2 * k) + j]), f1 = movm(w[4 * (2 * k + 1) + j]);
                        } else if (RP >= 32) {
                            f0 = w[(j * QN + k / 2) * 4 + 2 * (k % 2)];
                            f1 = w[(j * QN + k / 2) * 4 + 2 * (k % 2) + 1];
                        } else {
                            f0 = w[2 * j], f1 = w[2 * j + 1];
                        }
                        mma_acc(acc[j], lo[k], f0, f1);
                        mma_acc(acc[j], hi[k], f0, f1);
                    }
                #pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const long long row = h ? row1 : row0;
                    const uint4 b = h ? base1 : base0;
                    if (row < 0) continue;
                    uint4 v;
                    v.x = pack_bf16x2_rn(bf16_lo_to_f32(b.x) + acc[0][2 * h], bf16_hi_to_f32(b.x) + acc[0][2 * h + 1]);
                    v.y = pack_bf16x2_rn(bf16_lo_to_f32(b.y) + acc[1][2 * h], bf16_hi_to_f32(b.y) + acc[1][2 * h + 1]);
                    v.z = pack_bf16x2_rn(bf16_lo_to_f32(b.z) + acc[2][2 * h], bf16_hi_to_f32(b.z) + acc[2][2 * h + 1]);
                    v.w = pack_bf16x2_rn(bf16_lo_to_f32(b.w) + acc[3][2 * h], bf16_hi_to_f32(b.w) + acc[3][2 * h + 1]);
                    if (bad) v = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
                    store_cols8(p.y + row + mine, p.out - mine, p.vec_out, v);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * s);
        }
    }
    if (C > 1) mbar_wait_cluster(done, 0, abort_flag, p.err);   // no CTA leaves while its sums are read
}

// ---------------------------------------------------------------- host side
bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int ceil_div(long long a, long long b) { return int((a + b - 1) / b); }

// One lora_kernel launch over `tiles` tiles of TM tokens.
template <int RP, int TM, bool TRANS, bool FEW>
cudaError_t launch_lora_tiles(const LoraArgs &p, int tiles, int cluster, cudaStream_t s) {
    constexpr size_t smem = LoraShape<RP, TM>::kSmem;
    const cudaError_t e = allow_smem<lora_kernel<RP, TM, TRANS, FEW>>(smem);
    if (e != cudaSuccess) return e;
    return launch_chained(lora_kernel<RP, TM, TRANS, FEW>, dim3(unsigned(tiles) * cluster), kLoraThreads,
                          smem, cluster, s, p);
}

// The mma.sync kernel: few tokens, and ranks above 64.
template <int RP>
cudaError_t launch_few(const LoraArgs &p, cudaStream_t s) {
    return launch_lora_tiles<RP, kFewTile, false, true>(p, p.tokens, kMaxCluster, s);
}

// CTAs per tile: as many as leave one CTA per SM, so that few tiles use every
// SM and many tiles split nothing.
int tile_cluster(int tokens, int adapters, int sms) {
    const int full = ceil_div(tokens, kManyTile);
    const int tiles = full + (adapters < full ? adapters : full) / 2;
    int c = kMaxCluster;
    while (c > 1 && tiles * c > sms) c /= 2;
    return c;
}

cudaError_t launch_lora_few(const LoraArgs &p, cudaStream_t s) {
    switch (padded_rank(p.rank)) {
        case 16: return launch_few<16>(p, s);
        case 32: return launch_few<32>(p, s);
        case 64: return launch_few<64>(p, s);
        default: return launch_few<128>(p, s);
    }
}

template <bool TRANS>
cudaError_t launch_lora_many(const LoraArgs &p, int sms, cudaStream_t s) {
    if (padded_rank(p.rank) <= 64) return launch_lora_tensor(p, TRANS, sms, s);
    // the adapters' and the adapterless tokens' last tiles may be part empty
    const int extra = p.adapters + 1 < p.tokens ? p.adapters + 1 : p.tokens;
    return launch_lora_tiles<128, kManyTile, TRANS, false>(p, ceil_div(p.tokens, kManyTile) + extra,
                                                           tile_cluster(p.tokens, p.adapters, sms), s);
}

size_t round16(size_t b) { return (b + 15) / 16 * 16; }

// Workspace: order [tokens], sizes [adapters], the sort's counts, and for the
// gradient the planes of g and of s h.
struct LoraWorkspace {
    size_t order, sizes, counts, g, h, total;
};
LoraWorkspace lora_workspace(int tokens, int adapters, int rank, bool backward) {
    LoraWorkspace w;
    w.order = 0;
    w.sizes = round16(size_t(tokens) * 4);
    w.counts = w.sizes + round16(size_t(adapters) * 4);
    w.g = w.counts + round16(sort_bytes(tokens, adapters));
    w.h = w.g + size_t(tokens) * plane_pitch(padded_rank(rank));
    w.total = backward ? w.h + size_t(tokens) * plane_pitch(padded_rank(rank)) : w.g;
    if (!backward && tokens <= kFewTokens) w.total = 0;
    return w;
}

w4a16_status check_lora(int tokens, int adapters, int rank, int N, int K) {
    if (tokens < 0 || tokens > (1 << 24) || adapters < 1 || adapters > kMaxGroups) return W4A16_ERR_INVALID_ARG;
    if (rank < 8 || rank > kMaxRank || rank % 8) return W4A16_ERR_UNSUPPORTED;
    if (N < 1 || N > (1 << 24) || K < kGroup || K % kGroup || K > (1 << 20)) return W4A16_ERR_INVALID_ARG;
    return W4A16_OK;
}

w4a16_status from_cuda(cudaError_t e) { return e == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA; }

w4a16_status check_workspace(const LoraWorkspace &w, const void *ws, size_t bytes) {
    if (w.total == 0) return W4A16_OK;
    if (!ws || bytes < w.total) return W4A16_ERR_WORKSPACE_TOO_SMALL;
    return aligned(ws, 16) ? W4A16_OK : W4A16_ERR_INVALID_ARG;
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

w4a16_status w4a16_lora_workspace_bytes(int tokens, int num_adapters, int rank, int backward, size_t *bytes) {
    if (!bytes) return W4A16_ERR_INVALID_ARG;
    const w4a16_status st = check_lora(tokens, num_adapters, rank, 1, kGroup);
    if (st != W4A16_OK) return st;
    *bytes = tokens == 0 ? 0 : lora_workspace(tokens, num_adapters, rank, backward != 0).total;
    return W4A16_OK;
}

w4a16_status w4a16_lora_add(const w4a16_bf16 *X, const w4a16_bf16 *A, const w4a16_bf16 *B,
                            const void *adapters_dev, int id_bytes, const float *lora_scales,
                            const w4a16_bf16 *base, w4a16_bf16 *Y, float *hidden, int tokens,
                            int num_adapters, int rank, int N, int K, void *workspace,
                            size_t workspace_bytes, void *stream) {
    w4a16_status st = check_lora(tokens, num_adapters, rank, N, K);
    if (st != W4A16_OK) return st;
    if (id_bytes != 4 && id_bytes != 8) return W4A16_ERR_UNSUPPORTED;
    if (tokens == 0) return W4A16_OK;
    if (!X || !A || !B || !adapters_dev || !lora_scales || !Y) return W4A16_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(adapters_dev, id_bytes) ||
        !aligned(lora_scales, 4) || !aligned(base, 2) || !aligned(Y, 2) || !aligned(hidden, 16))
        return W4A16_ERR_INVALID_ARG;
    const LoraWorkspace w = lora_workspace(tokens, num_adapters, rank, false);
    st = check_workspace(w, workspace, workspace_bytes);
    if (st != W4A16_OK) return st;
    int sms = 0;
    if (device_sm_count(&sms) != 0 || sms < 1) return W4A16_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LoraArgs p = {};
    p.x = X, p.w1 = A, p.w2 = B, p.ids = adapters_dev, p.id_bytes = id_bytes, p.scale = lora_scales;
    p.base = base, p.y = Y, p.hidden = hidden, p.err = device_error_word();
    p.tokens = tokens, p.adapters = num_adapters, p.rank = rank, p.in = K, p.out = N;
    p.vec_in = 1;
    p.vec_out = N % 8 == 0 && aligned(base, 16) && aligned(Y, 16);
    if (tokens <= kFewTokens) return from_cuda(launch_lora_few(p, s));
    char *ws = static_cast<char *>(workspace);
    int *order = reinterpret_cast<int *>(ws + w.order), *sizes = reinterpret_cast<int *>(ws + w.sizes);
    cudaError_t e = launch_sort(adapters_dev, id_bytes, tokens, num_adapters,
                                reinterpret_cast<int *>(ws + w.counts), sizes, order, s);
    if (e != cudaSuccess) return W4A16_ERR_CUDA;
    p.order = order, p.sizes = sizes;
    return from_cuda(launch_lora_many<false>(p, sms, s));
}

w4a16_status w4a16_lora_add_backward(const w4a16_bf16 *dY, const w4a16_bf16 *X, const float *hidden,
                                     const w4a16_bf16 *A, const w4a16_bf16 *B, const void *adapters_dev,
                                     int id_bytes, const float *lora_scales, const w4a16_bf16 *dX_base,
                                     w4a16_bf16 *dX, w4a16_bf16 *dA, w4a16_bf16 *dB, int tokens,
                                     int num_adapters, int rank, int N, int K, void *workspace,
                                     size_t workspace_bytes, void *stream) {
    w4a16_status st = check_lora(tokens, num_adapters, rank, N, K);
    if (st != W4A16_OK) return st;
    if (id_bytes != 4 && id_bytes != 8) return W4A16_ERR_UNSUPPORTED;
    if (!dA || !dB || !aligned(dA, 16) || !aligned(dB, 16)) return W4A16_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (tokens == 0) {
        const size_t a = size_t(num_adapters) * rank * K * 2, b = size_t(num_adapters) * rank * N * 2;
        if (cudaMemsetAsync(dA, 0, a, s) != cudaSuccess) return W4A16_ERR_CUDA;
        return from_cuda(cudaMemsetAsync(dB, 0, b, s));
    }
    if (!dY || !X || !hidden || !A || !B || !adapters_dev || !lora_scales || !dX) return W4A16_ERR_INVALID_ARG;
    if (!aligned(dY, 2) || !aligned(X, 16) || !aligned(hidden, 16) || !aligned(A, 16) || !aligned(B, 16) ||
        !aligned(adapters_dev, id_bytes) || !aligned(lora_scales, 4) || !aligned(dX_base, 2) || !aligned(dX, 2))
        return W4A16_ERR_INVALID_ARG;
    const LoraWorkspace w = lora_workspace(tokens, num_adapters, rank, true);
    st = check_workspace(w, workspace, workspace_bytes);
    if (st != W4A16_OK) return st;
    int sms = 0;
    if (device_sm_count(&sms) != 0 || sms < 1) return W4A16_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    int *order = reinterpret_cast<int *>(ws + w.order), *sizes = reinterpret_cast<int *>(ws + w.sizes);
    cudaError_t e = launch_sort(adapters_dev, id_bytes, tokens, num_adapters,
                                reinterpret_cast<int *>(ws + w.counts), sizes, order, s);
    if (e != cudaSuccess) return W4A16_ERR_CUDA;
    LoraArgs p = {};
    p.x = dY, p.w1 = B, p.w2 = A, p.ids = adapters_dev, p.id_bytes = id_bytes, p.scale = lora_scales;
    p.order = order, p.sizes = sizes, p.base = dX_base, p.y = dX, p.hidden = const_cast<float *>(hidden);
    p.pg = reinterpret_cast<uint16_t *>(ws + w.g), p.ph = reinterpret_cast<uint16_t *>(ws + w.h);
    p.err = device_error_word();
    p.tokens = tokens, p.adapters = num_adapters, p.rank = rank, p.in = N, p.out = K;
    p.vec_in = N % 8 == 0 && aligned(dY, 16);
    p.vec_out = aligned(dX_base, 16) && aligned(dX, 16);
    e = launch_lora_many<true>(p, sms, s);
    if (e != cudaSuccess) return W4A16_ERR_CUDA;
    WgradArgs q = {};
    q.x = X, q.dy = dY, q.pg = p.pg, q.ph = p.ph, q.order = order, q.sizes = sizes, q.da = dA, q.db = dB;
    q.err = p.err, q.rank = rank, q.K = K, q.N = N, q.vec_x = 1, q.vec_dy = p.vec_in;
    return from_cuda(launch_wgrad(q, num_adapters, sms, s));
}

}  // extern "C"
