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
// memory in CTA order, and split the output columns.  X, base and the weights
// go from global memory straight into MMA fragments: the order of k inside an
// MMA is free as long as both operands agree, so a lane takes 16 bytes of a
// row, and 32 columns of a row feed two MMAs.  Where a weight lies along the
// wrong axis its 8 x 8 blocks are transposed in registers.
//
// Precision: products of bf16 are exact in the MMA and summed in fp32; h (and g)
// stay in fp32 and enter the second product as a sum of two bf16 terms, which
// holds them to 2^-17.  The outputs are rounded once.
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "w4a16.h"
#include "async.cuh"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace w4a16 {
namespace {

constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraCols = 32;          // columns of a step: 16 bytes per lane of a quad
constexpr int kManyTile = 64;          // tokens of a cluster's tile
constexpr int kFewTile = 16;
constexpr int kFewTokens = 128;        // up to this many tokens clusters find their tiles in the ids
constexpr int kMaxRank = 128;
constexpr int kWgradCols = 256;        // columns of a weight-gradient CTA: 32 per warp
constexpr int kWgradStage = 64;        // tokens per staged block
constexpr int kMaxCluster = 8;

struct LoraArgs {
    const uint16_t *x;       // [tokens][in]
    const uint16_t *w1;      // forward A [L][r][in]; gradient B [L][in][r]
    const uint16_t *w2;      // forward B [L][out][r]; gradient A [L][r][out]
    const void *ids;
    const int *order, *sizes;   // sorted tokens (the many-token form)
    const float *scale;      // [L]
    const uint16_t *base;    // [tokens][out] or nullptr
    uint16_t *y;             // [tokens][out]
    float *hidden;           // [tokens][r] or nullptr: forward h, gradient g
    int id_bytes, tokens, adapters, rank, in, out;
    int vec_in, vec_out;     // rows of x / of base and y start on 16 bytes
};

__device__ __forceinline__ uint32_t movm(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_u32(p)) : "memory");
}

__device__ __forceinline__ void mma_acc(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    mma_16816_c(c, a, b0, b1, c);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ int cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return int(r);
}
__device__ __forceinline__ int cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return int(r);
}
// The same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_cluster4(const void *p, int rank) {
    uint32_t a;
    float4 v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}

// Eight bf16 from column p, `left` of them inside the row.  vec: the row
// starts on 16 bytes and its width is a multiple of 8.
__device__ __forceinline__ uint4 load_cols8(const uint16_t *p, int left, int vec) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (vec) {
        if (left > 0)
            asm("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
        return v;
    }
    uint32_t w[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = 2 * i < left ? p[2 * i] : 0, hi = 2 * i + 1 < left ? p[2 * i + 1] : 0;
        w[i] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store_cols8(uint16_t *p, int left, int vec, uint4 v) {
    if (vec) {
        if (left > 0) *reinterpret_cast<uint4 *>(p) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (2 * i < left) p[2 * i] = uint16_t(w[i]);
        if (2 * i + 1 < left) p[2 * i + 1] = uint16_t(w[i] >> 16);
    }
}

// hi + lo = v to 2^-17 of it; an infinity stays in hi alone.
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16x2_rn(a, b);
    const float ha = bf16_lo_to_f32(hi), hb = bf16_hi_to_f32(hi);
    lo = pack_bf16x2_rn(isinf(ha) ? 0.f : a - ha, isinf(hb) ? 0.f : b - hb);
}

__device__ __forceinline__ int adapter_of(const LoraArgs &p, int t) {
    const long long v = p.id_bytes == 8 ? static_cast<const long long *>(p.ids)[t]
                                        : static_cast<const int *>(p.ids)[t];
    return v >= 0 && v < p.adapters ? int(v) : -1;
}

// One warp: the tokens of tile `tile` into rows[], its adapter (-1: none) and
// their number into out[0], out[1] (number 0: no such tile).
// Few tokens: tile i belongs to token i and exists where the tokens of its
// adapter before it fill whole tiles; it holds that token and the next ones.
template <int TM>
__device__ void find_tile_few(const LoraArgs &p, int tile, int *rows, int *out) {
    const int lane = threadIdx.x & 31;
    const int key = adapter_of(p, tile);
    int before = 0, count = 0;
    for (int t0 = 0; t0 < p.tokens; t0 += 32) {
        const int t = t0 + lane;
        const bool same = t < p.tokens && adapter_of(p, t) == key;
        before += __popc(__ballot_sync(0xffffffffu, same && t < tile));
        const unsigned after = __ballot_sync(0xffffffffu, same && t >= tile);
        const int pos = count + __popc(after & ((1u << lane) - 1));
        if (same && t >= tile && pos < TM) rows[pos] = t;
        count += __popc(after);
    }
    if (lane == 0) {
        out[0] = key;
        out[1] = before % TM == 0 ? min(count, TM) : 0;
    }
}

// Sorted tokens: adapters' tiles in order, those without an adapter last.
template <int TM>
__device__ void find_tile_sorted(const LoraArgs &p, int tile, int *rows, int *out) {
    const int lane = threadIdx.x & 31;
    int tiles = 0, row = 0, adapter = -1, start = 0, count = 0;
    bool found = false;
    for (int a0 = 0; a0 < p.adapters && !found; a0 += 32) {
        const int size = a0 + lane < p.adapters ? p.sizes[a0 + lane] : 0;
        const int mine = (size + TM - 1) / TM;
        int tile_end = mine, row_end = size;
        #pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int u = __shfl_up_sync(0xffffffffu, tile_end, d);
            const int v = __shfl_up_sync(0xffffffffu, row_end, d);
            if (lane >= d) tile_end += u, row_end += v;
        }
        const int first = tiles + tile_end - mine;
        const unsigned hit = __ballot_sync(0xffffffffu, tile >= first && tile < tiles + tile_end);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const int skip = (tile - first) * TM;
            adapter = a0 + src;
            start = __shfl_sync(0xffffffffu, row + row_end - size + skip, src);
            count = __shfl_sync(0xffffffffu, min(TM, size - skip), src);
            found = true;
        }
        tiles += __shfl_sync(0xffffffffu, tile_end, 31);
        row += __shfl_sync(0xffffffffu, row_end, 31);
    }
    if (!found) {
        start = row + (tile - tiles) * TM;
        count = max(0, min(TM, p.tokens - start));
    }
    for (int i = lane; i < count; i += 32) rows[i] = p.order[start + i];
    if (lane == 0) out[0] = adapter, out[1] = count;
}

constexpr int lora_warp_rows(int TM) { return TM >= 32 ? 32 : 16; }   // rows of a warp, first product
constexpr int lora_k_warps(int TM) { return kLoraWarps / (TM / lora_warp_rows(TM)); }
constexpr size_t lora_smem(int RP, int TM) { return size_t(lora_k_warps(TM) + 1) * TM * (RP + 4) * 4; }

// TRANS: weights along the other axis (the gradient).  RP: the rank rounded up
// to 16, 32, 64 or 128; ranks past p.rank are zeros in registers.
template <int RP, int TM, bool TRANS, bool FEW>
__global__ void __launch_bounds__(kLoraThreads, RP <= 32 ? 2 : 1) lora_kernel(const LoraArgs p) {
    constexpr int MT = lora_warp_rows(TM) / 16;          // 16-row blocks of a warp, first product
    constexpr int RG = TM / (16 * MT), KW = kLoraWarps / RG;
    constexpr int NT = RP / 8;                           // 8-rank blocks
    constexpr int QN = RP >= 32 ? RP / 32 : 1;           // 32-rank blocks (one of 16)
    constexpr int JN = RP >= 32 ? 4 : 2;                 // 8-rank blocks of one
    constexpr int PS = RP + 4;                           // floats of a row of h
    constexpr int U = RP == 16 && TM == 16 ? 4 : RP <= 64 ? 2 : 1;   // steps loaded together
    extern __shared__ float s_mem[];
    float *s_part = s_mem;                               // [KW][TM][PS]
    float *s_h = s_mem + KW * TM * PS;                   // [TM][PS]
    __shared__ int s_rows[TM];
    __shared__ int s_tile[2];

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int C = cluster_size(), c = cluster_rank();
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
            for (int r = warp; r < count; r += kLoraWarps) {
                const long long at = (long long)s_rows[r] * p.out;
                for (int i = i0 + lane; i < i1; i += 32) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (p.base) v = load_cols8(p.base + at + 8 * i, p.out - 8 * i, p.vec_out);
                    store_cols8(p.y + at + 8 * i, p.out - 8 * i, p.vec_out, v);
                }
            }
        }
        if (p.hidden && c == 0)
            for (int i = threadIdx.x; i < count * p.rank; i += kLoraThreads)
                p.hidden[(long long)s_rows[i / p.rank] * p.rank + i % p.rank] = 0.f;
        return;
    }

    // ---- h: each warp takes rows [16 MT rg, +16 MT) over its share of the columns
    const int r = p.rank;
    {
        const int rg = warp % RG, kw = warp / RG;
        const int steps = (p.in + kLoraCols - 1) / kLoraCols;
        const int b0 = int((long long)steps * (c * KW + kw) / (C * KW));
        const int b1 = int((long long)steps * (c * KW + kw + 1) / (C * KW));
        const uint16_t *xrow[MT][2];
        #pragma unroll
        for (int m = 0; m < MT; ++m)
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = 16 * (rg * MT + m) + 8 * h + g;
                xrow[m][h] = i < count ? p.x + (long long)s_rows[i] * p.in + 8 * t : nullptr;
            }
        const uint16_t *w1 = p.w1 + (long long)adapter * r * p.in;
        float acc[MT][NT][4];
        #pragma unroll
        for (int m = 0; m < MT; ++m)
            #pragma unroll
            for (int n = 0; n < NT; ++n)
                #pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
        if (16 * MT * rg < count) {
            for (int bb = b0; bb < b1; bb += U) {
                uint4 xv[U][MT][2];
                uint32_t w[U][RP / 2];
                #pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int col = (bb + u) * kLoraCols;
                    const bool in = bb + u < b1;
                    #pragma unroll
                    for (int m = 0; m < MT; ++m)
                        #pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            xv[u][m][h] = make_uint4(0, 0, 0, 0);
                            if (in && xrow[m][h])
                                xv[u][m][h] = load_cols8(xrow[m][h] + col, p.in - col - 8 * t, p.vec_in);
                        }
                    if (!TRANS) {
                        // A's row of rank 8n + g, columns 8t..8t+7
                        #pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            uint4 v = make_uint4(0, 0, 0, 0);
                            if (in && 8 * n + g < r)
                                v = ldg_nc16(w1 + (long long)(8 * n + g) * p.in + col + 8 * t);
                            w[u][4 * n] = v.x, w[u][4 * n + 1] = v.y, w[u][4 * n + 2] = v.z, w[u][4 * n + 3] = v.w;
                        }
                    } else {
                        // B's rows of columns {8 (i/2) + 4 s + 2 hh + i%2}, i = 0..7: the
                        // k slots of MMA s that X's 16-byte loads fill
                        #pragma unroll
                        for (int sh = 0; sh < 4; ++sh) {
                            const int row = col + 8 * (g >> 1) + 2 * sh + (g & 1);
                            #pragma unroll
                            for (int q = 0; q < QN; ++q) {
                                if (RP >= 32) {
                                    uint4 v = make_uint4(0, 0, 0, 0);
                                    if (in && row < p.in && 32 * q + 8 * t < r)
                                        v = ldg_nc16(w1 + (long long)row * r + 32 * q + 8 * t);
                                    uint32_t *d = &w[u][(sh * QN + q) * JN];
                                    d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
                                } else {
                                    uint2 v = make_uint2(0, 0);
                                    if (in && row < p.in && 4 * t < r)
                                        v = __ldg(reinterpret_cast<const uint2 *>(w1 + (long long)row * r + 4 * t));
                                    w[u][sh * 2] = v.x, w[u][sh * 2 + 1] = v.y;
                                }
                            }
                        }
                    }
                }
                #pragma unroll
                for (int u = 0; u < U; ++u)
                    #pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        uint32_t a[MT][4];
                        #pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            a[m][0] = s ? xv[u][m][0].z : xv[u][m][0].x;
                            a[m][1] = s ? xv[u][m][1].z : xv[u][m][1].x;
                            a[m][2] = s ? xv[u][m][0].w : xv[u][m][0].y;
                            a[m][3] = s ? xv[u][m][1].w : xv[u][m][1].y;
                        }
                        #pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            uint32_t f0, f1;
                            if (!TRANS) {
                                f0 = w[u][4 * n + 2 * s], f1 = w[u][4 * n + 2 * s + 1];
                            } else {
                                const int q = n / JN, j = n % JN;
                                f0 = movm(w[u][(2 * s * QN + q) * JN + j]);
                                f1 = movm(w[u][((2 * s + 1) * QN + q) * JN + j]);
                            }
                            #pragma unroll
                            for (int m = 0; m < MT; ++m) mma_acc(acc[m][n], a[m], f0, f1);
                        }
                    }
            }
        }
        // columns 2t, 2t+1 of block n hold these two neighbouring ranks
        #pragma unroll
        for (int m = 0; m < MT; ++m)
            #pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int rank = !TRANS ? 8 * n + 2 * t
                                        : RP >= 32 ? 32 * (n / JN) + 8 * t + 2 * (n % JN) : 4 * t + 2 * n;
                float *d = s_part + (kw * TM + 16 * (rg * MT + m) + g) * PS + rank;
                *reinterpret_cast<float2 *>(d) = make_float2(acc[m][n][0], acc[m][n][1]);
                *reinterpret_cast<float2 *>(d + 8 * PS) = make_float2(acc[m][n][2], acc[m][n][3]);
            }
    }
    __syncthreads();
    const float scale = p.scale[adapter];
    constexpr int kQuads = RP / 4;
    for (int i = threadIdx.x; i < TM * kQuads; i += kLoraThreads) {
        float *d = s_part + (i / kQuads) * PS + 4 * (i % kQuads);
        float4 v = *reinterpret_cast<const float4 *>(d);
        #pragma unroll
        for (int k = 1; k < KW; ++k) {
            const float4 u = *reinterpret_cast<const float4 *>(d + k * TM * PS);
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
        *reinterpret_cast<float4 *>(d) = v;
    }
    if (C > 1) {
        cluster_arrive();
        cluster_wait();
    }
    for (int i = threadIdx.x; i < TM * kQuads; i += kLoraThreads) {
        const int row = i / kQuads, rank = 4 * (i % kQuads);
        const float *d = s_part + row * PS + rank;
        float4 v;
        if (C > 1) {
            v = ld_cluster4(d, 0);
            for (int k = 1; k < C; ++k) {
                const float4 u = ld_cluster4(d, k);
                v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
            }
        } else {
            v = *reinterpret_cast<const float4 *>(d);
        }
        // a rank past r is 0 also where x holds infinities (0 * inf)
        if (rank >= r) v = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 s = make_float4(scale * v.x, scale * v.y, scale * v.z, scale * v.w);
        *reinterpret_cast<float4 *>(s_h + row * PS + rank) = s;
        if (p.hidden && c == 0 && row < count && rank < r)
            *reinterpret_cast<float4 *>(p.hidden + (long long)s_rows[row] * r + rank) = TRANS ? s : v;
    }
    __syncthreads();
    if (C > 1) cluster_arrive();                         // this CTA has read the others' sums

    // ---- y: each warp takes 16 rows over its share of the output columns
    {
        constexpr int RG2 = TM / 16, CW = kLoraWarps / RG2, KS = RP / 16;
        const int rg = warp % RG2, cw = warp / RG2;
        const int steps = (p.out + kLoraCols - 1) / kLoraCols;
        const int n0 = int((long long)steps * (c * CW + cw) / (C * CW));
        const int n1 = int((long long)steps * (c * CW + cw + 1) / (C * CW));
        if (16 * rg < count) {
            uint32_t hi[KS][4], lo[KS][4];
            #pragma unroll
            for (int k = 0; k < KS; ++k)
                #pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // slots (2t, 2t+1) for i < 2, (2t+8, 2t+9) for i >= 2
                    const int rank = TRANS ? 16 * k + 2 * t + 8 * (i / 2)
                                           : RP >= 32 ? 32 * (k / 2) + 8 * t + 4 * (k % 2) + 2 * (i / 2)
                                                      : 4 * t + 2 * (i / 2);
                    const float2 v = *reinterpret_cast<const float2 *>(
                        s_h + (16 * rg + g + 8 * (i % 2)) * PS + rank);
                    split2(v.x, v.y, hi[k][i], lo[k][i]);
                }
            const uint16_t *w2 = p.w2 + (long long)adapter * r * p.out;
            const int i0 = 16 * rg + g, i1 = i0 + 8;
            const long long row0 = i0 < count ? (long long)s_rows[i0] * p.out : -1;
            const long long row1 = i1 < count ? (long long)s_rows[i1] * p.out : -1;
            #pragma unroll 2
            for (int nb = n0; nb < n1; ++nb) {
                const int col = nb * kLoraCols, mine = col + 8 * t;
                uint4 base0 = make_uint4(0, 0, 0, 0), base1 = base0;
                if (p.base && row0 >= 0) base0 = load_cols8(p.base + row0 + mine, p.out - mine, p.vec_out);
                if (p.base && row1 >= 0) base1 = load_cols8(p.base + row1 + mine, p.out - mine, p.vec_out);
                uint32_t w[RP / 2];
                if (!TRANS) {
                    // B's rows of columns {8 (i/2) + 2 j + i%2}: a lane's results are 8 neighbours
                    #pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int row = col + 8 * (g >> 1) + 2 * j + (g & 1);
                        #pragma unroll
                        for (int q = 0; q < QN; ++q) {
                            if (RP >= 32) {
                                uint4 v = make_uint4(0, 0, 0, 0);
                                if (row < p.out && 32 * q + 8 * t < r)
                                    v = ldg_nc16(w2 + (long long)row * r + 32 * q + 8 * t);
                                uint32_t *d = &w[(j * QN + q) * 4];
                                d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
                            } else {
                                uint2 v = make_uint2(0, 0);
                                if (row < p.out && 4 * t < r)
                                    v = __ldg(reinterpret_cast<const uint2 *>(w2 + (long long)row * r + 4 * t));
                                w[2 * j] = v.x, w[2 * j + 1] = v.y;
                            }
                        }
                    }
                } else {
                    #pragma unroll
                    for (int k = 0; k < 2 * KS; ++k) {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (8 * k + g < r && mine < p.out)
                            v = ldg_nc16(w2 + (long long)(8 * k + g) * p.out + mine);
                        w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
                    }
                }
                float acc[4][4];
                #pragma unroll
                for (int j = 0; j < 4; ++j) {
                    #pragma unroll
                    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
                    #pragma unroll
                    for (int k = 0; k < KS; ++k) {
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
                    store_cols8(p.y + row + mine, p.out - mine, p.vec_out, v);
                }
            }
        }
    }
    __syncwarp();
    if (C > 1) cluster_wait();                           // no CTA leaves while its sums are read
}

// ---------------------------------------------------------- weight gradients
struct WgradArgs {
    const uint16_t *x, *dy;        // [tokens][K], [tokens][N]
    const float *g, *h;            // [tokens][r]
    const float *scale;
    const int *order, *sizes;
    uint16_t *da, *db;             // [L][r][K], [L][N][r]
    int rank, K, N, slices_x;      // 256-column slices of x, then of dy
    int vec_x, vec_dy;
};

constexpr int kStageRow = kWgradStage + 8;     // bf16 of a staged rank's row
constexpr size_t wgrad_smem(int RP) {
    return size_t(RP) * kStageRow * 2 * 2 > size_t(kLoraThreads) * RP * 4 ? size_t(RP) * kStageRow * 2 * 2
                                                                         : size_t(kLoraThreads) * RP * 4;
}

// Grid (slices * cluster, adapters): a cluster owns 256 columns of one
// adapter's dA (or rows of dB); its CTAs split the adapter's tokens and add
// their sums through distributed shared memory, in CTA order.  The tokens are
// the MMA's k: rows of Q (x or dy) are read 16 bytes per lane and their 8 x 8
// blocks transposed in registers; P (g or s h) is staged as [rank][token], in
// two bf16 terms.  dA has the ranks as MMA rows, dB the columns of dy, so that
// either gradient's rows leave as 16-byte stores.
template <int RP, bool DB>
__device__ __forceinline__ void wgrad_tile(const WgradArgs &p, int slice, int adapter, uint16_t *s_p) {
    constexpr int JN = RP >= 32 ? 4 : 2;
    constexpr int TILES = RP / 4;                     // 16 x 8 accumulators of a warp
    const uint16_t *q = DB ? p.dy : p.x;
    const float *pr = DB ? p.h : p.g;
    const int cols = DB ? p.N : p.K, vec = DB ? p.vec_dy : p.vec_x, r = p.rank;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int C = cluster_size(), c = cluster_rank();
    int start = 0;
    for (int a = lane; a < adapter; a += 32) start += p.sizes[a];
    start = __reduce_add_sync(0xffffffffu, start);
    const int size = p.sizes[adapter];
    const int blocks = (size + 15) / 16;
    const int t0 = 16 * int((long long)blocks * c / C), t1 = min(size, 16 * int((long long)blocks * (c + 1) / C));
    const int *rows = p.order + start;
    const float mult = DB ? p.scale[adapter] : 1.f;
    const int mine = slice * kWgradCols + 32 * warp + 8 * t;

    float acc[TILES][4];
    #pragma unroll
    for (int i = 0; i < TILES; ++i)
        #pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    uint16_t *s_hi = s_p, *s_lo = s_p + RP * kStageRow;
    for (int tb = t0; tb < t1; tb += kWgradStage) {
        uint4 qv[kWgradStage / 16][2];
        #pragma unroll
        for (int k = 0; k < kWgradStage / 16; ++k)
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = tb + 16 * k + 8 * h + g;
                qv[k][h] = make_uint4(0, 0, 0, 0);
                if (i < t1) qv[k][h] = load_cols8(q + (long long)rows[i] * cols + mine, cols - mine, vec);
            }
        __syncthreads();
        for (int i = threadIdx.x; i < kWgradStage * RP / 4; i += kLoraThreads) {
            const int tok = i % kWgradStage, rank = 4 * (i / kWgradStage);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (tb + tok < t1 && rank < r)
                v = *reinterpret_cast<const float4 *>(pr + (long long)rows[tb + tok] * r + rank);
            uint32_t hi[2], lo[2];
            split2(mult * v.x, mult * v.y, hi[0], lo[0]);
            split2(mult * v.z, mult * v.w, hi[1], lo[1]);
            #pragma unroll
            for (int e = 0; e < 4; ++e) {
                s_hi[(rank + e) * kStageRow + tok] = uint16_t(hi[e / 2] >> (16 * (e % 2)));
                s_lo[(rank + e) * kStageRow + tok] = uint16_t(lo[e / 2] >> (16 * (e % 2)));
            }
        }
        __syncthreads();
        #pragma unroll
        for (int k = 0; k < kWgradStage / 16; ++k) {
            if (tb + 16 * k >= t1) break;
            uint32_t qt[2][4];                        // [tokens 0-7, 8-15][8-column block j]
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
                qt[h][0] = movm(qv[k][h].x), qt[h][1] = movm(qv[k][h].y);
                qt[h][2] = movm(qv[k][h].z), qt[h][3] = movm(qv[k][h].w);
            }
            #pragma unroll
            for (int part = 0; part < 2; ++part) {
                const uint16_t *s = (part ? s_hi : s_lo) + 16 * k;
                if (!DB) {
                    #pragma unroll
                    for (int m = 0; m < RP / 16; ++m) {
                        uint32_t a[4];
                        ldmatrix4(a, s + (16 * m + (lane & 15)) * kStageRow + 8 * (lane >> 4));
                        #pragma unroll
                        for (int j = 0; j < 4; ++j) mma_acc(acc[4 * m + j], a, qt[0][j], qt[1][j]);
                    }
                } else {
                    // two 8-rank blocks per load; block j of a 32-rank block holds the
                    // ranks {8 (i/2) + 2 j + i%2} (of a 16-rank block {4 (i/2) + 2 j + i%2})
                    #pragma unroll
                    for (int n = 0; n < RP / 8; n += 2) {
                        const int i = lane & 7, j = n % JN + (lane >> 4);
                        const int rank = RP >= 32 ? 32 * (n / JN) + 8 * (i >> 1) + 2 * j + (i & 1)
                                                  : 4 * (i >> 1) + 2 * j + (i & 1);
                        uint32_t b[4];
                        ldmatrix4(b, s + rank * kStageRow + 8 * ((lane >> 3) & 1));
                        #pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint32_t a[4] = {qt[0][2 * m], qt[0][2 * m + 1], qt[1][2 * m], qt[1][2 * m + 1]};
                            mma_acc(acc[m * (RP / 8) + n], a, b[0], b[1]);
                            mma_acc(acc[m * (RP / 8) + n + 1], a, b[2], b[3]);
                        }
                    }
                }
            }
        }
    }
    // Groups of W neighbouring results, [group][thread][W]; the cluster's CTAs
    // then share out the threads and add the CTAs' sums.
    constexpr int W = DB && RP < 32 ? 4 : 8, GROUPS = RP / W;
    float *s_sum = reinterpret_cast<float *>(s_p);
    __syncthreads();
    #pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
        float v[W];
        #pragma unroll
        for (int e = 0; e < W; ++e) {
            if (!DB) {       // group: 16-rank block i / 2, row half i % 2; 8 columns
                v[e] = acc[4 * (i / 2) + e / 2][2 * (i % 2) + e % 2];
            } else {         // group: row (m, half) = i % 4, rank block i / 4
                v[e] = acc[((i % 4) / 2) * (RP / 8) + (i / 4) * JN + e / 2][2 * (i % 2) + e % 2];
            }
        }
        #pragma unroll
        for (int e = 0; e < W; e += 4)
            *reinterpret_cast<float4 *>(s_sum + ((i * (W / 4) + e / 4) * kLoraThreads + threadIdx.x) * 4) =
                make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    }
    if (C > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    const int share = kLoraThreads / C;
    for (int idx = threadIdx.x; idx < share * GROUPS; idx += kLoraThreads) {
        const int src = c * share + idx % share, i = idx / share;
        float v[W];
        #pragma unroll
        for (int e = 0; e < W; e += 4) {
            const float *at = s_sum + ((i * (W / 4) + e / 4) * kLoraThreads + src) * 4;
            float4 s = C > 1 ? ld_cluster4(at, 0) : *reinterpret_cast<const float4 *>(at);
            for (int k = 1; k < C; ++k) {
                const float4 u = ld_cluster4(at, k);
                s.x += u.x, s.y += u.y, s.z += u.z, s.w += u.w;
            }
            v[e] = s.x, v[e + 1] = s.y, v[e + 2] = s.z, v[e + 3] = s.w;
        }
        const int sw = src / 32, sg = (src % 32) / 4, st = src % 4;
        const int col0 = slice * kWgradCols + 32 * sw;
        if (!DB) {
            const int rank = 16 * (i / 2) + 8 * (i % 2) + sg, col = col0 + 8 * st;
            if (rank >= r || col >= cols) continue;
            uint4 o;
            o.x = pack_bf16x2_rn(v[0], v[1]), o.y = pack_bf16x2_rn(v[2], v[3]);
            o.z = pack_bf16x2_rn(v[W - 4], v[W - 3]), o.w = pack_bf16x2_rn(v[W - 2], v[W - 1]);
            *reinterpret_cast<uint4 *>(p.da + ((long long)adapter * r + rank) * cols + col) = o;
        } else {
            // rows of the 16 x 8 block m: 8-column block 2m (first half), 2m + 1 (second)
            const int row = col0 + 8 * (sg >> 1) + 2 * (i % 4) + (sg & 1);
            const int rank = RP >= 32 ? 32 * (i / 4) + 8 * st : 4 * st;
            if (row >= cols || rank >= r) continue;
            uint16_t *d = p.db + ((long long)adapter * cols + row) * r + rank;
            uint4 o;
            o.x = pack_bf16x2_rn(v[0], v[1]), o.y = pack_bf16x2_rn(v[2], v[3]);
            o.z = pack_bf16x2_rn(v[W - 4], v[W - 3]), o.w = pack_bf16x2_rn(v[W - 2], v[W - 1]);
            if (W == 8) *reinterpret_cast<uint4 *>(d) = o;
            else *reinterpret_cast<uint2 *>(d) = make_uint2(o.x, o.y);
        }
    }
    if (C > 1) {
        cluster_arrive();
        cluster_wait();
    }
}

template <int RP>
__global__ void __launch_bounds__(kLoraThreads, RP <= 64 ? 2 : 1) lora_wgrad_kernel(const WgradArgs p) {
    extern __shared__ float s_mem[];
    pdl_wait();
    pdl_launch_dependents();
    const int slice = blockIdx.x / cluster_size();
    if (slice < p.slices_x) wgrad_tile<RP, false>(p, slice, blockIdx.y, reinterpret_cast<uint16_t *>(s_mem));
    else wgrad_tile<RP, true>(p, slice - p.slices_x, blockIdx.y, reinterpret_cast<uint16_t *>(s_mem));
}

// ---------------------------------------------------------------- host side
bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int ceil_div(long long a, long long b) { return int((a + b - 1) / b); }

int padded_rank(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }

// A kernel with more dynamic shared memory than the default limit has to be
// allowed it once per device.
template <auto Kernel>
cudaError_t allow_smem(size_t bytes) {
    static std::atomic<uint64_t> allowed{0};
    if (bytes <= 48 * 1024) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (allowed.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(reinterpret_cast<const void *>(Kernel),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
    if (e == cudaSuccess) allowed.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// One lora_kernel launch over `tiles` tiles of TM tokens.
template <int RP, int TM, bool TRANS, bool FEW>
cudaError_t launch_lora_tiles(const LoraArgs &p, int tiles, int cluster, cudaStream_t s) {
    const cudaError_t e = allow_smem<lora_kernel<RP, TM, TRANS, FEW>>(lora_smem(RP, TM));
    if (e != cudaSuccess) return e;
    return launch_chained(lora_kernel<RP, TM, TRANS, FEW>, dim3(unsigned(tiles) * cluster), kLoraThreads,
                          lora_smem(RP, TM), cluster, s, p);
}

template <int RP, bool TRANS>
cudaError_t launch_lora_rank(const LoraArgs &p, bool few, int cluster, cudaStream_t s) {
    if constexpr (!TRANS)
        if (few) return launch_lora_tiles<RP, kFewTile, TRANS, true>(p, p.tokens, cluster, s);
    // the adapters' and the adapterless tokens' last tiles may be part empty
    const int extra = p.adapters + 1 < p.tokens ? p.adapters + 1 : p.tokens;
    return launch_lora_tiles<RP, kManyTile, TRANS, false>(p, ceil_div(p.tokens, kManyTile) + extra, cluster, s);
}

template <bool TRANS>
cudaError_t launch_lora(const LoraArgs &p, bool few, int cluster, cudaStream_t s) {
    switch (padded_rank(p.rank)) {
        case 16: return launch_lora_rank<16, TRANS>(p, few, cluster, s);
        case 32: return launch_lora_rank<32, TRANS>(p, few, cluster, s);
        case 64: return launch_lora_rank<64, TRANS>(p, few, cluster, s);
        default: return launch_lora_rank<128, TRANS>(p, few, cluster, s);
    }
}

// CTAs per tile: as many as still let all tiles of a full batch be resident
// at once, so that a small batch uses every SM.
int tile_cluster(int tokens, int rank, int sms) {
    const int slots = (padded_rank(rank) <= 32 ? 2 : 1) * sms, tiles = ceil_div(tokens, kManyTile);
    int c = kMaxCluster;
    while (c > 1 && tiles * c > slots) c /= 2;
    return c;
}

template <int RP>
cudaError_t launch_wgrad_rank(const WgradArgs &p, int adapters, int slices, int cluster, cudaStream_t s) {
    const cudaError_t e = allow_smem<lora_wgrad_kernel<RP>>(wgrad_smem(RP));
    if (e != cudaSuccess) return e;
    return launch_chained(lora_wgrad_kernel<RP>, dim3(slices * cluster, adapters), kLoraThreads, wgrad_smem(RP),
                          cluster, s, p);
}

cudaError_t launch_wgrad(const WgradArgs &p, int adapters, int slices, int cluster, cudaStream_t s) {
    switch (padded_rank(p.rank)) {
        case 16: return launch_wgrad_rank<16>(p, adapters, slices, cluster, s);
        case 32: return launch_wgrad_rank<32>(p, adapters, slices, cluster, s);
        case 64: return launch_wgrad_rank<64>(p, adapters, slices, cluster, s);
        default: return launch_wgrad_rank<128>(p, adapters, slices, cluster, s);
    }
}

size_t round16(size_t b) { return (b + 15) / 16 * 16; }

// Workspace: order [tokens], sizes [adapters], the sort's counts, and for the
// gradient g [tokens][rank].
struct LoraWorkspace {
    size_t order, sizes, counts, g, total;
};
LoraWorkspace lora_workspace(int tokens, int adapters, int rank, bool backward) {
    LoraWorkspace w;
    w.order = 0;
    w.sizes = round16(size_t(tokens) * 4);
    w.counts = w.sizes + round16(size_t(adapters) * 4);
    w.g = w.counts + round16(sort_bytes(tokens, adapters));
    w.total = backward ? w.g + size_t(tokens) * rank * 4 : w.g;
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
    p.base = base, p.y = Y, p.hidden = hidden;
    p.tokens = tokens, p.adapters = num_adapters, p.rank = rank, p.in = K, p.out = N;
    p.vec_in = 1;
    p.vec_out = N % 8 == 0 && aligned(base, 16) && aligned(Y, 16);
    if (tokens <= kFewTokens) return from_cuda(launch_lora<false>(p, true, kMaxCluster, s));
    char *ws = static_cast<char *>(workspace);
    int *order = reinterpret_cast<int *>(ws + w.order), *sizes = reinterpret_cast<int *>(ws + w.sizes);
    cudaError_t e = launch_sort(adapters_dev, id_bytes, tokens, num_adapters,
                                reinterpret_cast<int *>(ws + w.counts), sizes, order, s);
    if (e != cudaSuccess) return W4A16_ERR_CUDA;
    p.order = order, p.sizes = sizes;
    return from_cuda(launch_lora<false>(p, false, tile_cluster(tokens, rank, sms), s));
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
    float *g = reinterpret_cast<float *>(ws + w.g);
    cudaError_t e = launch_sort(adapters_dev, id_bytes, tokens, num_adapters,
                                reinterpret_cast<int *>(ws + w.counts), sizes, order, s);
    if (e != cudaSuccess) return W4A16_ERR_CUDA;
    LoraArgs p = {};
    p.x = dY, p.w1 = B, p.w2 = A, p.ids = adapters_dev, p.id_bytes = id_bytes, p.scale = lora_scales;
    p.order = order, p.sizes = sizes, p.base = dX_base, p.y = dX, p.hidden = g;
    p.tokens = tokens, p.adapters = num_adapters, p.rank = rank, p.in = N, p.out = K;
    p.vec_in = N % 8 == 0 && aligned(dY, 16);
    p.vec_out = aligned(dX_base, 16) && aligned(dX, 16);
    e = launch_lora<true>(p, false, tile_cluster(tokens, rank, sms), s);
    if (e != cudaSuccess) return W4A16_ERR_CUDA;
    WgradArgs q = {};
    q.x = X, q.dy = dY, q.g = g, q.h = hidden, q.scale = lora_scales, q.order = order, q.sizes = sizes;
    q.da = dA, q.db = dB, q.rank = rank, q.K = K, q.N = N, q.slices_x = ceil_div(K, kWgradCols);
    q.vec_x = 1, q.vec_dy = p.vec_in;
    const int slices = q.slices_x + ceil_div(N, kWgradCols);
    int cluster = 1;
    while (cluster < kMaxCluster && (long long)slices * num_adapters * cluster < 2LL * sms) cluster *= 2;
    return from_cuda(launch_wgrad(q, num_adapters, slices, cluster, s));
}

}  // extern "C"
