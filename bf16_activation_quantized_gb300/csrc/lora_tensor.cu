// lora_tensor.cu -- adapters for many tokens, on the tensor cores.
//
// lora_tensor_kernel: y = base + s B (A x) and, with the weights read along the
// other axis, dx = dx_base + A^T (s B^T dy), for tiles of 128 sorted tokens of one
// adapter (the formulas and the precision: lora.cu).  A cluster of CTAs owns a
// tile and splits first the input columns, then the output columns.  Four
// producer warps gather the rows of X (then of base) and the weights with
// 16-byte asynchronous copies into a ring of 128-column stages, in the 128-byte
// swizzle that tcgen05.mma reads; one warp issues the MMAs.  D1 = X W1^T (128
// tokens x rank, in TMEM) is read once, its partial sums are added over the
// cluster in CTA order, each CTA a share of the rows, and the result returns to
// every CTA as two bf16 planes, the A operand of D2 = H W2^T.  Eight epilogue
// warps add base in shared memory and store whole 128-byte pieces of rows.
//
// What bounds it: HBM.  At rank 64 the legacy MMA pipe would need two thirds of
// the memory's time and left a 64-token mma.sync version of this kernel waiting
// on MMA latency (78 us for 4096 tokens, 8192 x 8192); tcgen05 needs a tenth.
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
constexpr int kTmemD1 = 256;           // D2's two buffers take columns 0..255

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory"); }

// Byte of piece p (16 bytes) of row `row` in a block of 128-byte rows.
__device__ __forceinline__ uint32_t sw128(int row, int p) { return uint32_t(row * 128 + ((p ^ (row & 7)) << 4)); }

template <int RP>
struct TensorShape {
    static constexpr int kW = 2 * RP * 128 > kBlock ? 2 * RP * 128 : kBlock;   // weights of a stage
    static constexpr int kStage = 2 * kBlock + kW;
    static constexpr int PS = RP + 4;                       // floats of a row of partial sums
    static constexpr int kH = 2 * kBlock;                   // the planes of h
    static constexpr int kFixed = kH + kTile * PS * 4;
    static constexpr int kStages = (kSmemMax - 1024 - kFixed) / kStage;
    static constexpr int kSmem = kStages * kStage + kFixed + 1024;
    static_assert(RP <= 64 && kStages >= 2, "the ring does not fit");
};

template <int RP, bool TRANS>
__global__ void __launch_bounds__(kThreads, 1) lora_tensor_kernel(const LoraArgs p) {
    using S = TensorShape<RP>;
    constexpr int NS = S::kStages, PS = S::PS, KS = RP / 16;
    extern __shared__ unsigned char s_raw[];
    __shared__ uint64_t s_bar[3 * NS + 8];
    __shared__ int s_rows[kTile];
    __shared__ int s_tile[3];
    __shared__ int s_abort;
    __shared__ uint32_t s_tmem;
    unsigned char *s_mem = s_raw + (-smem_u32(s_raw) & 1023);
    unsigned char *s_hi = s_mem + NS * S::kStage, *s_lo = s_hi + kBlock;
    float *s_part = reinterpret_cast<float *>(s_lo + kBlock);            // [kTile][PS]

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int C = cluster_size(), c = cluster_rank();
    const uint32_t full = smem_u32(s_bar), empty1 = full + 8 * NS, empty2 = empty1 + 8 * NS;
    const uint32_t d1full = empty2 + 8 * NS, ready = d1full + 8, hready = ready + 8;
    const uint32_t dfull = hready + 8, dempty = dfull + 16, done = dempty + 16;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + 8 * i, kProducers);
            mbar_init(empty1 + 8 * i, 1);            // first product: the MMAs have read it
            mbar_init(empty2 + 8 * i, kEpiWarps);    // second: the epilogue has
        }
        mbar_init(d1full, 1);
        mbar_init(ready, C);
        mbar_init(hready, C);
        for (int i = 0; i < 2; ++i) mbar_init(dfull + 8 * i, 1), mbar_init(dempty + 8 * i, kEpiWarps);
        mbar_init(done, 1);
        s_abort = 0;
        fence_barrier_init();
    }
    pdl_wait();
    if (warp == 0) find_tile_sorted<kTile>(p, blockIdx.x / C, s_rows, s_tile);
    __syncthreads();
    const int adapter = s_tile[0], count = s_tile[1];
    if (count == 0) return;                          // the same in every CTA of the cluster
    if (adapter < 0) {
        // no adapter: y = base, h = 0
        if (p.y != p.base) {
            const int items = (p.out + 7) / 8;
            const int i0 = int((long long)items * c / C), i1 = int((long long)items * (c + 1) / C);
            for (int r = warp; r < count; r += kThreads / 32) {
                const long long at = (long long)s_rows[r] * p.out;
                #pragma unroll 8
                for (int i = i0 + lane; i < i1; i += 32) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (p.base) v = load_cols8(p.base + at + 8 * i, p.out - 8 * i, p.vec_out);
                    store_cols8(p.y + at + 8 * i, p.out - 8 * i, p.vec_out, v);
                }
            }
        }
        if (!TRANS && p.hidden && c == 0)
            for (int i = threadIdx.x; i < count * p.rank; i += kThreads)
                p.hidden[(long long)s_rows[i / p.rank] * p.rank + i % p.rank] = 0.f;
        return;
    }
    // Dependents may start only when every CTA holds its TMEM, so that an
    // allocation never waits for a kernel that waits for this one.
    if (warp == kMmaWarp) {
        tc_alloc(smem_u32(&s_tmem), kTmemCols);
        tc_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    if (C > 1) cluster_arrive();                     // barriers initialised
    const uint32_t tmem = s_tmem;

    const int r = p.rank;
    const int kin = (p.in + kCols - 1) / kCols, kout = (p.out + kCols - 1) / kCols;
    const int in0 = int((long long)kin * c / C), out0 = int((long long)kout * c / C);
    const int nin = int((long long)kin * (c + 1) / C) - in0;
    const int nall = nin + int((long long)kout * (c + 1) / C) - out0;
    volatile int *abort_flag = &s_abort;

    if (warp >= kEpiWarps && warp < kMmaWarp) {
        // ---- producers: the stages of both products in order
        const uint16_t *w1 = p.w1 + (long long)adapter * r * p.in, *w2 = p.w2 + (long long)adapter * r * p.out;
        const int pt = threadIdx.x - kEpiThreads, piece = pt % 16, row0 = pt / 16;
        constexpr int kRows = kProducers / 16;       // rows in one go
        for (int i = 0; i < nall; ++i) {
            const int s = i % NS;
            bool ok = true;
            if (i >= NS) {
                const int before = i - NS, use = before / NS;
                if (before < nin) {
                    ok = mbar_wait(empty1 + 8 * s, use & 1, abort_flag, p.err);
                } else {
                    const int uses1 = (nin - s + NS - 1) / NS;   // of this stage, in the first product
                    ok = mbar_wait(empty2 + 8 * s, (use - uses1) & 1, abort_flag, p.err);
                }
            }
            if (!__all_sync(0xffffffffu, ok)) break;
            const bool first = i < nin;
            const int cols = first ? p.in : p.out, col = (first ? in0 + i : out0 + i - nin) * kCols;
            const int n = min(kCols, cols - col), vec = first ? p.vec_in : p.vec_out;
            const uint16_t *rows = first ? p.x : p.base, *w = first ? w1 : w2;
            const uint32_t xs = smem_u32(s_mem) + s * S::kStage, ws = xs + 2 * kBlock;
            const bool in = 8 * piece < n;
            if (rows) {
                // columns past the end are zeros: they are summed over in the first product
                const uint32_t dst = xs + (piece / 8) * kBlock;
                if (vec) {
                    #pragma unroll 4
                    for (int k = row0; k < count; k += kRows) {
                        const uint16_t *src = rows + (long long)s_rows[k] * cols + (in ? col + 8 * piece : 0);
                        cp_async16z(dst + sw128(k, piece % 8), src, in);
                    }
                } else {
                    for (int k = row0; k < count; k += kRows) {
                        const uint4 v = load_cols8(rows + (long long)s_rows[k] * cols + col + 8 * piece,
                                                   n - 8 * piece, 0);
                        *reinterpret_cast<uint4 *>(s_mem + s * S::kStage + (piece / 8) * kBlock +
                                                   sw128(k, piece % 8)) = v;
                    }
                }
            }
            if (first != TRANS) {
                // [r][cols]: rows of ranks.  Ranks past r are summed over in the second product.
                const int rows_w = first ? r : RP;
                const uint32_t dst = ws + (piece / 8) * (RP * 128);
                #pragma unroll 4
                for (int k = row0; k < rows_w; k += kRows) {
                    const bool ok_w = in && k < r;
                    cp_async16z(dst + sw128(k, piece % 8), ok_w ? w + (long long)k * cols + col + 8 * piece : w, ok_w);
                }
            } else {
                // [cols][r]: rows of columns, zeros past the end and past r
                #pragma unroll 4
                for (int k = pt; k < kCols * (RP / 8); k += kProducers) {
                    const int row = k / (RP / 8), q = k % (RP / 8);
                    const bool ok_w = row < n && 8 * q < r;
                    cp_async16z(ws + sw128(row, q), ok_w ? w + (long long)(col + row) * r + 8 * q : w, ok_w);
                }
            }
            stage_done(full + 8 * s, vec);
        }
        cp_async_wait_all();
    } else if (warp == kMmaWarp) {
        // ---- MMA issuer
        constexpr uint32_t idesc1 = tc_idesc_bf16(kTile, RP) | (TRANS ? kTcBMajorN : 0);
        constexpr uint32_t idesc2 = tc_idesc_bf16(kTile, kCols) | (TRANS ? kTcBMajorN : 0);
        bool ok = true;
        for (int i = 0; i < nin && ok; ++i) {
            const int s = i % NS;
            ok = __all_sync(0xffffffffu, mbar_wait(full + 8 * s, (i / NS) & 1, abort_flag, p.err));
            if (!ok) break;
            fence_proxy_async();
            tc_fence_after();
            const uint32_t xs = smem_u32(s_mem) + s * S::kStage, ws = xs + 2 * kBlock;
            if (elect_one()) {
                #pragma unroll
                for (int k = 0; k < kCols / 16; ++k) {
                    const uint64_t a = tc_sdesc_sw128(xs + (k / 4) * kBlock + (k % 4) * 32);
                    const uint64_t b = TRANS ? tc_sdesc_sw128_mn(ws + k * 2048, kBlock)
                                             : tc_sdesc_sw128(ws + (k / 4) * (RP * 128) + (k % 4) * 32);
                    tc_mma_ss(tmem + kTmemD1, a, b, idesc1, i > 0 || k > 0);
                }
                tc_commit(empty1 + 8 * s);
            }
            __syncwarp();
        }
        if (ok && nin > 0 && elect_one()) tc_commit(d1full);
        __syncwarp();
        ok = ok && __all_sync(0xffffffffu, mbar_wait_cluster(hready, 0, abort_flag, p.err));
        for (int i = nin; i < nall && ok; ++i) {
            const int s = i % NS, j = i - nin, buf = j & 1;
            ok = j < 2 || mbar_wait(dempty + 8 * buf, ((j >> 1) - 1) & 1, abort_flag, p.err);
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
                    for (int k = 0; k < KS; ++k) {
                        const uint64_t a = tc_sdesc_sw128(smem_u32(part ? s_hi : s_lo) + k * 32);
                        const uint64_t b = TRANS ? tc_sdesc_sw128_mn(ws + k * 2048, RP * 128)
                                                 : tc_sdesc_sw128(ws + k * 32);
                        tc_mma_ss(tmem + buf * kCols, a, b, idesc2, part > 0 || k > 0);
                    }
                tc_commit(dfull + 8 * buf);
            }
            __syncwarp();
        }
        // every MMA issued has completed before TMEM is freed
        if (elect_one()) tc_commit(done);
        __syncwarp();
        drain_wait(done, 0);
        if (!ok) drain_wait(hready, 0);              // the others may still read this CTA's sums
    } else {
        // ---- h: D1's rows to shared memory, summed over the cluster
        const int sub = warp % 4, half = warp / 4;
        const int my_row = 32 * sub + lane;
        const uint32_t lanes = tmem + (uint32_t(32 * sub) << 16);
        const float scale = p.scale[adapter];
        bool bad = false;
        if (nin > 0) {
            bad = !__all_sync(0xffffffffu, mbar_wait(d1full, 0, abort_flag, p.err));
            tc_fence_after();
        }
        #pragma unroll
        for (int k = 0; k < RP / 16; ++k) {
            const int rank = half * (RP / 2) + 8 * k;
            uint32_t v[8];
            if (nin > 0 && !bad) {
                tc_ld_32x32b_x8(lanes + kTmemD1 + rank, v);
                tc_wait_ld();
            } else {
                #pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = bad ? 0x7fffffffu : 0u;
            }
            float *d = s_part + my_row * PS + rank;
            *reinterpret_cast<uint4 *>(d) = make_uint4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<uint4 *>(d + 4) = make_uint4(v[4], v[5], v[6], v[7]);
        }
        epi_sync();
        if (C > 1) {
            cluster_wait();
            if (threadIdx.x < C) mbar_arrive_cluster(ready, threadIdx.x);
            bad |= !mbar_wait_cluster(ready, 0, abort_flag, p.err);
        }
        // this CTA's share of the rows; the planes go to every CTA
        constexpr int kPieces = RP / 8;
        const int r0 = kTile / C * c;
        for (int i = threadIdx.x; i < kTile / C * kPieces; i += kEpiThreads) {
            const int row = r0 + i / kPieces, rank = 8 * (i % kPieces);
            const float *d = s_part + row * PS + rank;
            float v[8];
            #pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.f;
            for (int k = 0; k < C; ++k) {
                const float4 a = C > 1 ? ld_cluster4(d, k) : *reinterpret_cast<const float4 *>(d);
                const float4 b = C > 1 ? ld_cluster4(d + 4, k) : *reinterpret_cast<const float4 *>(d + 4);
                v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
                v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
            }
            const bool token = row < count, in = rank < r;
            if (bad) {
                #pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __int_as_float(0x7fffffff);
            }
            if (!TRANS && p.hidden && token && in) {
                float4 *h = reinterpret_cast<float4 *>(p.hidden + (long long)s_rows[row] * r + rank);
                h[0] = make_float4(v[0], v[1], v[2], v[3]);
                h[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
            // ranks past r are zeros: what was staged for them is not
            uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
            if (in) {
                split2(scale * v[0], scale * v[1], hi.x, lo.x), split2(scale * v[2], scale * v[3], hi.y, lo.y);
                split2(scale * v[4], scale * v[5], hi.z, lo.z), split2(scale * v[6], scale * v[7], hi.w, lo.w);
            }
            for (int k = 0; k < C; ++k) {
                const int to = (c + k) % C;
                st_cluster16(smem_u32(s_hi) + sw128(row, i % kPieces), to, hi);
                st_cluster16(smem_u32(s_lo) + sw128(row, i % kPieces), to, lo);
            }
            if (TRANS && token) {
                // g and s h of the sorted token, for the weight gradients
                const long long at = (long long)(s_tile[2] + row) * (plane_pitch(RP) / 2) + rank;
                *reinterpret_cast<uint4 *>(p.pg + at) = hi, *reinterpret_cast<uint4 *>(p.pg + at + RP) = lo;
                hi = lo = make_uint4(0, 0, 0, 0);
                if (in) {
                    const float4 *h = reinterpret_cast<const float4 *>(p.hidden + (long long)s_rows[row] * r + rank);
                    const float4 a = h[0], b = h[1];
                    split2(scale * a.x, scale * a.y, hi.x, lo.x), split2(scale * a.z, scale * a.w, hi.y, lo.y);
                    split2(scale * b.x, scale * b.y, hi.z, lo.z), split2(scale * b.z, scale * b.w, hi.w, lo.w);
                }
                *reinterpret_cast<uint4 *>(p.ph + at) = hi, *reinterpret_cast<uint4 *>(p.ph + at + RP) = lo;
            }
        }
        fence_proxy_async();
        epi_sync();
        if (threadIdx.x < C) mbar_arrive_cluster(hready, threadIdx.x);

        // ---- y: this warp's 32 rows x 64 columns of every stage
        for (int i = nin; i < nall; ++i) {
            const int s = i % NS, j = i - nin, buf = j & 1;
            const int col = (out0 + j) * kCols + 64 * half;
            unsigned char *bs = s_mem + s * S::kStage + half * kBlock;
            bool ok = mbar_wait(full + 8 * s, (i / NS) & 1, abort_flag, p.err);
            ok = ok && mbar_wait(dfull + 8 * buf, (j >> 1) & 1, abort_flag, p.err);
            bad |= !__all_sync(0xffffffffu, ok);
            tc_fence_after();
            if (col < p.out && 32 * sub < count) {
                uint32_t acc[2][32];
                tc_ld_32x32b_x32(lanes + buf * kCols + 64 * half, acc[0]);
                tc_ld_32x32b_x32(lanes + buf * kCols + 64 * half + 32, acc[1]);
                tc_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(dempty + 8 * buf);
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
                    if (bad) v = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
                    *at = v;
                }
                __syncwarp();
                #pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int row = 32 * sub + 4 * k + lane / 8, q = lane % 8;
                    if (row < count) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(bs + sw128(row, q));
                        store_cols8(p.y + (long long)s_rows[row] * p.out + col + 8 * q, p.out - col - 8 * q, p.vec_out, v);
                    }
                }
            } else {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(dempty + 8 * buf);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty2 + 8 * s);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tc_dealloc(tmem, kTmemCols);
    // every thread that arrived waits (the epilogue's did); no CTA is read or
    // written after its own hready, which it has passed
    if (C > 1 && warp >= kEpiWarps) cluster_wait();
}

// ---------------------------------------------------------- weight gradients
constexpr int kStageTokens = 32;

template <int RP>
struct WgradShape {
    static constexpr int kCols = RP <= 64 ? 512 : 256;      // columns of a CTA
    static constexpr int kQBlock = kStageTokens * 128;      // bytes of 32 tokens x 64 columns
    static constexpr int kQ = kCols / 64 * kQBlock;
    static constexpr int kP = (RP + 63) / 64 * kQBlock;     // of one plane
    static constexpr int kStage = kQ + 2 * kP;
    static constexpr int kSumsA = RP * (kCols + 4) * 4, kSumsB = kCols * (RP + 4) * 4;
    static constexpr int kSums = kSumsA > kSumsB ? kSumsA : kSumsB;
    static constexpr int kStages = (kSmemMax - 1024) / kStage;
    static constexpr int kSmem = kStages * kStage + 1024;
    static_assert(kStages >= 2 && kSums <= kStages * kStage, "the ring does not fit");
};

// Grid (slices * cluster, adapters): a cluster owns kCols columns of one
// adapter's dA (or rows of dB), D[column][rank] in TMEM in blocks of 128
// columns; its CTAs split the adapter's tokens, 32 to a stage, and add their
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

    if (warp >= kEpiWarps && warp < kMmaWarp) {
        constexpr int kRows = kStageTokens / kProducerWarps;     // rows of a producer warp
        const int first = (warp - kEpiWarps) * kRows;
        for (int i = 0; i < stages; ++i) {
            const int s = i % NS, tok = t0 + i * kStageTokens, n = min(kStageTokens, t1 - tok);
            const int row = lane < kRows && first + lane < n ? rows[tok + first + lane] : 0;
            const bool ok = i < NS || mbar_wait(empty + 8 * s, (i / NS - 1) & 1, abort_flag, p.err);
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint32_t qs = ring + s * S::kStage, ps = qs + S::kQ;
            // tokens past the end are zeros on both sides: they are summed over
            #pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const bool in = first + k < n;
                const uint16_t *src = q + (long long)__shfl_sync(0xffffffffu, row, k) * cols + col0;
                #pragma unroll
                for (int b = lane; b < S::kCols / 8; b += 32) {
                    const uint32_t dst = (b / 8) * S::kQBlock + sw128(first + k, b % 8);
                    const bool ok_q = in && 8 * b < width;
                    if (vec) {
                        if (8 * b < width) cp_async16z(qs + dst, ok_q ? src + 8 * b : q, ok_q);
                    } else if (8 * b < width) {
                        *reinterpret_cast<uint4 *>(s_mem + s * S::kStage + dst) =
                            load_cols8(src + 8 * b, in ? width - 8 * b : 0, 0);
                    }
                }
            }
            const uint16_t *src = planes + (long long)(start + tok) * (plane_pitch(RP) / 2);
            constexpr int kPieces = RP / 4;                      // 16-byte pieces of both planes
            #pragma unroll 4
            for (int k = threadIdx.x - kEpiThreads; k < kStageTokens * kPieces; k += kProducers) {
                const int t = k / kPieces, b = k % kPieces, plane = b / (RP / 8), e = b % (RP / 8);
                cp_async16z(ps + plane * S::kP + (e / 8) * S::kQBlock + sw128(t, e % 8),
                            t < n ? src + (long long)t * (plane_pitch(RP) / 2) + 8 * b : planes, t < n);
            }
            stage_done(full + 8 * s, vec);
        }
        cp_async_wait_all();
    } else if (warp == kMmaWarp) {
        constexpr uint32_t idesc = tc_idesc_bf16(128, RP) | kTcAMajorM | kTcBMajorN;
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
                    for (int part = 0; part < 2; ++part)         // the low plane first
                        #pragma unroll
                        for (int k = 0; k < kStageTokens / 16; ++k) {
                            const uint64_t a = tc_sdesc_sw128_mn(qs + m * 2 * S::kQBlock + k * 2048, S::kQBlock);
                            const uint64_t b = tc_sdesc_sw128_mn(ps + (part ? 0 : S::kP) + k * 2048, S::kQBlock);
                            tc_mma_ss(tmem + m * RP, a, b, idesc, i > 0 || part > 0 || k > 0);
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
    if (warp < kEpiWarps) {
        const int sub = warp % 4;
        for (int m = warp / 4; m < S::kCols / 128; m += 2) {
            const int col = 128 * m + 32 * sub + lane;
            #pragma unroll
            for (int k = 0; k < RP / 8; ++k) {
                uint32_t v[8];
                if (stages > 0 && !bad) {
                    tc_ld_32x32b_x8(tmem + (uint32_t(32 * sub) << 16) + m * RP + 8 * k, v);
                    tc_wait_ld();
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
    for (int i = i0 + threadIdx.x; i < i1; i += kThreads) {
        const int row = i / per, col = 8 * (i % per);
        const float *at = s_sum + row * kPitch + col;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        for (int k = 0; k < C; ++k) {
            const float4 u = C > 1 ? ld_cluster4(at, k) : *reinterpret_cast<const float4 *>(at);
            const float4 v = C > 1 ? ld_cluster4(at + 4, k) : *reinterpret_cast<const float4 *>(at + 4);
            a.x += u.x, a.y += u.y, a.z += u.z, a.w += u.w;
            b.x += v.x, b.y += v.y, b.z += v.z, b.w += v.w;
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
__global__ void __launch_bounds__(kThreads, 1) lora_wgrad_kernel(const WgradArgs p) {
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
        for (int i = 0; i < NS; ++i) mbar_init(bar + 8 * i, kProducers), mbar_init(bar + 8 * (NS + i), 1);
        mbar_init(bar + 16 * NS, 1);
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
    pdl_launch_dependents();
    pdl_wait();
    const int slice = blockIdx.x / cluster_size();
    if (slice < p.slices_x) wgrad_tile<RP, false>(p, slice, blockIdx.y, s_mem, s_bar, &s_abort, tmem);
    else wgrad_tile<RP, true>(p, slice - p.slices_x, blockIdx.y, s_mem, s_bar, &s_abort, tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tc_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------- host side
int ceil_div(long long a, long long b) { return int((a + b - 1) / b); }

template <int RP, bool TRANS>
cudaError_t launch_tensor_rank(const LoraArgs &p, int sms, cudaStream_t s) {
    using S = TensorShape<RP>;
    const cudaError_t e = allow_smem<lora_tensor_kernel<RP, TRANS>>(S::kSmem);
    if (e != cudaSuccess) return e;
    // CTAs per tile: as many as leave one CTA per SM (the adapters' last tiles
    // counted as half there), so that few tiles use every SM and many split nothing
    const int whole = ceil_div(p.tokens, kTile);
    const int tiles = whole + (p.adapters < whole ? p.adapters : whole) / 2;
    int cluster = kMaxCluster;
    while (cluster > 1 && tiles * cluster > sms) cluster /= 2;
    const int extra = p.adapters + 1 < p.tokens ? p.adapters + 1 : p.tokens;
    return launch_chained(lora_tensor_kernel<RP, TRANS>, dim3(unsigned(whole + extra) * cluster), kThreads, S::kSmem,
                          cluster, s, p);
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
    return launch_chained(lora_wgrad_kernel<RP>, dim3(slices * cluster, adapters), kThreads, S::kSmem, cluster, s, p);
}

}  // namespace

cudaError_t launch_lora_tensor(const LoraArgs &p, bool trans, int sms, cudaStream_t s) {
    switch (padded_rank(p.rank)) {
        case 16: return trans ? launch_tensor_rank<16, true>(p, sms, s) : launch_tensor_rank<16, false>(p, sms, s);
        case 32: return trans ? launch_tensor_rank<32, true>(p, sms, s) : launch_tensor_rank<32, false>(p, sms, s);
        case 64: return trans ? launch_tensor_rank<64, true>(p, sms, s) : launch_tensor_rank<64, false>(p, sms, s);
        default: return cudaErrorInvalidValue;
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
