// lora.cu -- low-rank adapters of many requests beside a shared projection: the
// C ABI and the kernel for few tokens (lora_tensor.cu has those for many).
//
// Token t with adapter a = ids[t] (outside [0, L): none):
//   h[t] = A_a x[t],  y[t] = base[t] + s_a B_a h[t]          A [r][K], B [N][r]
// and the gradients, with g[t] = s_a B_a^T dy[t],
//   dx[t] = dx_base[t] + A_a^T g[t],  dA_a = sum_t g[t] x[t]^T,
//   dB_a = s_a sum_t dy[t] h[t]^T     (sums over the adapter's tokens).
// y and dx are one computation: a product down to the rank, then one up to the
// output, with the weights read along the other axis.
//
// Precision: products of bf16 are exact in the MMA and summed in fp32; h (and g)
// stay in fp32 and enter the second product as a sum of three bf16 terms, which is
// their value itself.  The outputs are rounded once.
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "w4a16.h"
#include "internal.h"
#include "launch.cuh"
#include "lora.cuh"

namespace w4a16 {
namespace {

constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kStepCols = 32;          // columns of a step: 16 bytes per lane of a quad
constexpr int kFewTile = 16;
// Up to `tokens` tokens take this kernel, and up to `most` while the adapters have at
// most `each` on average (many adapters leave the tensor core kernels' tiles of 128
// tokens mostly empty).  Measured at 8192 x 8192, this kernel / the tensor core kernels,
// in us.  Rank 16: 384 tokens of 1 adapter 24.7 / 30.3, 512 35.8 / 29.9; 512 of 16 24.5 /
// 27.6, 768 40.3 / 28.5; 768 of 64 31.3 / 61.2.  Rank 32: 192 tokens of 1 adapter 15.4 /
// 26.6, 384 of 4 26.7 / 28.4, 768 of 64 37.1 / 63.6.  Rank 64: 128 tokens of 1 adapter
// 17.5 / 22.6, 192 27.3 / 25.5; 256 of 16 25.1 / 31.8, 384 36.7 / 32.3; 512 of 64 62.0 /
// 73.8, 768 78.2 / 74.3.  Rank 128: 128 of 4 20.5 / 23.2, 512 of 64 80.5 / 96.8.
// The border is 8192 x 8192's; other shapes have another, at rank 16: 1024 x 1024, 256 of
// 1 13.0 / 16.1, 384 20.3 / 15.9; 2560 to 19456 columns, 192 of 1 17.3 / 19.0, 384 32.6 /
// 21.7.  And the adapters counted are the table's, not those in use, which only the
// device knows: 768 tokens that all use one of 64 take 37.2 / 29.3 (2560 to 19456: 56.1 /
// 26.9), against 31.3 / 61.2 (48.5 / 78.8) where they are spread.
struct FewLimits {
    int tokens, most, each;
};
constexpr FewLimits few_limits(int rank) { return rank <= 32 ? FewLimits{384, 768, 32} : FewLimits{128, 512, 16}; }
constexpr int kMaxRank = 128;

__device__ __forceinline__ void mma_acc(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    mma_16816_c(c, a, b0, b1, c);
}

// Few tokens: one launch.  A cluster of eight CTAs (fewer where not all clusters
// would be resident, few_cluster) owns up to 16 tokens of one adapter (cluster i
// starts at token i, or leaves if an earlier one has it), found in the ids without a
// sort.  Its warps split the columns of the first product, add their sums of h in
// shared and then distributed shared memory in a fixed order, and split the columns
// of the second.  Everything goes from
// global memory straight into MMA fragments: the order of k inside an MMA is
// free as long as both operands agree, so a lane takes 16 bytes of a row and 32
// columns feed two MMAs; and the columns of the second product are dealt to the
// MMAs so that a lane's results are 8 neighbours.
//
// What bounds it: latency.  One token at rank 16 and 8192 x 8192 needs 0.5 MB;
// the chain is ids -> rows and A -> sums over warps and CTAs -> y, so the first
// B and base of each warp are on their way before the sums are.  Measured at 8192 x
// 8192 and rank 16: one token 5.5 us, 32 tokens of 64 adapters 6.8 (2.7 TB/s, of which
// much from L2); 61 tokens of 64 adapters at rank 32, 2560 to 19456 columns: 20.2
// us (57 MB, 2.8 TB/s), bound by how many loads the 8 warps of a CTA hold in registers.
// h's third term costs 0.4 us of one token's and 0.6 of 61 tokens' (two terms in an MMA
// that has no tokens in half its rows; three MMAs instead: 23.1).
template <int RP>
__global__ void __launch_bounds__(kFewThreads, RP <= 32 ? 2 : 1) lora_few_kernel(const LoraArgs p) {
    constexpr int TM = kFewTile, NT = RP / 8, QN = RP >= 32 ? RP / 32 : 1, KS = RP / 16;
    constexpr int PS = RP + 4;                           // floats of a row of h
    // Steps of the first and of the second product whose operands a lane loads together,
    // as many as its registers hold (128 up to rank 32, else 255): three of the first at
    // rank 64 or two at 128 gained nothing, one more of the second spilled.
    constexpr int U = RP <= 32 ? 2 : 1, PF = RP == 16 || RP == 64 ? 4 : RP == 32 ? 3 : 2;
    constexpr int kQuads = RP / 4;
    extern __shared__ float s_mem[];
    float *s_part = s_mem;                               // [kFewWarps][TM][PS]
    // s h: fragments of the second product, [plane][KS][lane]
    uint4 *s_h = reinterpret_cast<uint4 *>(s_mem + kFewWarps * TM * PS);
    __shared__ int s_rows[TM];
    __shared__ int s_tile[3];

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int C = cluster_size(), c = cluster_rank();
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) find_tile_few<TM>(p, blockIdx.x / C, s_rows, s_tile);
    __syncthreads();
    const int adapter = s_tile[0], count = s_tile[1], r = p.rank;
    if (count == 0) return;                              // the same in every CTA of the cluster
    if (adapter < 0) {
        // no adapter: y = base, h = 0
        if (p.y != p.base) {
            const int items = (p.out + 7) / 8;
            const int i0 = int((long long)items * c / C), i1 = int((long long)items * (c + 1) / C);
            for (int k = warp; k < count; k += kFewWarps) {
                const long long at = (long long)s_rows[k] * p.out;
                #pragma unroll 4
                for (int i = i0 + lane; i < i1; i += 32) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (p.base) v = load_cols8(p.base + at + 8 * i, p.out - 8 * i, p.vec_out);
                    store_cols8(p.y + at + 8 * i, p.out - 8 * i, p.vec_out, v);
                }
            }
        }
        if (p.hidden && c == 0)
            for (int i = threadIdx.x; i < count * r; i += kFewThreads)
                p.hidden[(long long)s_rows[i / r] * r + i % r] = 0.f;
        return;
    }

    // ---- the second product's operands, PF steps at a time
    const uint16_t *w2 = p.w2 + (long long)adapter * r * p.out;
    const int out_steps = (p.out + kStepCols - 1) / kStepCols;
    const int n0 = int((long long)out_steps * (c * kFewWarps + warp) / (C * kFewWarps));
    const int n1 = int((long long)out_steps * (c * kFewWarps + warp + 1) / (C * kFewWarps));
    const long long row0 = g < count ? (long long)s_rows[g] * p.out : -1;
    const long long row1 = g + 8 < count ? (long long)s_rows[g + 8] * p.out : -1;
    uint32_t w[PF][RP / 2];
    uint4 base[PF];                                      // of rows g; rows g + 8 come when they are needed
    const auto load_up = [&](int nb) {
        #pragma unroll
        for (int f = 0; f < PF; ++f) {
            if (nb + f >= n1) break;
            const int col = (nb + f) * kStepCols, mine = col + 8 * t;
            base[f] = make_uint4(0, 0, 0, 0);
            if (p.base && row0 >= 0) base[f] = load_cols8(p.base + row0 + mine, p.out - mine, p.vec_out);
            // B's rows of columns {8 (i/2) + 2 j + i%2}
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = col + 8 * (g >> 1) + 2 * j + (g & 1);
                #pragma unroll
                for (int q = 0; q < QN; ++q) {
                    if (RP >= 32) {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (row < p.out && 32 * q + 8 * t < r) v = ldg_nc16(w2 + (long long)row * r + 32 * q + 8 * t);
                        uint32_t *d = &w[f][(j * QN + q) * 4];
                        d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
                    } else {
                        uint2 v = make_uint2(0, 0);
                        if (row < p.out && 4 * t < r)
                            v = __ldg(reinterpret_cast<const uint2 *>(w2 + (long long)row * r + 4 * t));
                        w[f][2 * j] = v.x, w[f][2 * j + 1] = v.y;
                    }
                }
            }
        }
    };

    // ---- h
    {
        const int steps = p.in / kStepCols;
        const int b0 = int((long long)steps * (c * kFewWarps + warp) / (C * kFewWarps));
        const int b1 = int((long long)steps * (c * kFewWarps + warp + 1) / (C * kFewWarps));
        const uint16_t *x0 = g < count ? p.x + (long long)s_rows[g] * p.in + 8 * t : nullptr;
        const uint16_t *x1 = g + 8 < count ? p.x + (long long)s_rows[g + 8] * p.in + 8 * t : nullptr;
        const uint16_t *w1 = p.w1 + (long long)adapter * r * p.in + 8 * t;
        float acc[NT][4];
        #pragma unroll
        for (int n = 0; n < NT; ++n)
            #pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
        for (int bb = b0; bb < b1; bb += U) {
            uint4 xv[U][2], wv[U][NT];
            #pragma unroll
            for (int u = 0; u < U; ++u) {
                const int col = (bb + u) * kStepCols;
                const bool in = bb + u < b1;
                xv[u][0] = xv[u][1] = make_uint4(0, 0, 0, 0);
                if (in && x0) xv[u][0] = load_cols8(x0 + col, 8, 1);
                if (in && x1) xv[u][1] = load_cols8(x1 + col, 8, 1);
                #pragma unroll
                for (int n = 0; n < NT; ++n) {           // A's row of rank 8n + g
                    wv[u][n] = make_uint4(0, 0, 0, 0);
                    if (in && 8 * n < r) wv[u][n] = ldg_nc16(w1 + (long long)(8 * n + g) * p.in + col);
                }
            }
            #pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t a0[4] = {xv[u][0].x, xv[u][1].x, xv[u][0].y, xv[u][1].y};
                const uint32_t a1[4] = {xv[u][0].z, xv[u][1].z, xv[u][0].w, xv[u][1].w};
                #pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_acc(acc[n], a0, wv[u][n].x, wv[u][n].y);
                    mma_acc(acc[n], a1, wv[u][n].z, wv[u][n].w);
                }
            }
        }
        load_up(n0);
        #pragma unroll
        for (int n = 0; n < NT; ++n) {
            float *d = s_part + (warp * TM + g) * PS + 8 * n + 2 * t;
            *reinterpret_cast<float2 *>(d) = make_float2(acc[n][0], acc[n][1]);
            *reinterpret_cast<float2 *>(d + 8 * PS) = make_float2(acc[n][2], acc[n][3]);
        }
    }
    __syncthreads();
    const float scale = p.scale[adapter];
    const bool packed = count <= 8;                      // see s_h below
    for (int i = threadIdx.x; i < count * kQuads; i += kFewThreads) {
        float *d = s_part + (i / kQuads) * PS + 4 * (i % kQuads);
        float4 v = *reinterpret_cast<const float4 *>(d);
        #pragma unroll
        for (int k = 1; k < kFewWarps; ++k) {
            const float4 u = *reinterpret_cast<const float4 *>(d + k * TM * PS);
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
        *reinterpret_cast<float4 *>(d) = v;
    }
    cluster_arrive();
    cluster_wait();
    #pragma unroll 1
    for (int i = threadIdx.x; i < count * kQuads; i += kFewThreads) {
        const int row = i / kQuads, rank = 4 * (i % kQuads);
        float4 part[kMaxCluster], v = make_float4(0.f, 0.f, 0.f, 0.f);
        #pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
            if (k < C) part[k] = ld_cluster4(s_part + row * PS + rank, k);
        #pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
            if (k < C) v.x += part[k].x, v.y += part[k].y, v.z += part[k].z, v.w += part[k].w;
        if (p.hidden && c == 0 && rank < r)
            *reinterpret_cast<float4 *>(p.hidden + (long long)s_rows[row] * r + rank) = v;
        // the MMA's slots (2t, 2t + 1) and (2t + 8, 2t + 9) of row g (or g + 8) hold ranks
        // 4 t + 0..3 of a rank block of 16, 8 t + 4 (k % 2) + 0..3 of two
        uint32_t lo2[kPlanes], hi2[kPlanes];
        // a rank past r is 0 also where x or the scale is infinite (0 * inf)
        v = rank < r ? make_float4(scale * v.x, scale * v.y, scale * v.z, scale * v.w) : make_float4(0.f, 0.f, 0.f, 0.f);
        split3(v.x, v.y, lo2), split3(v.z, v.w, hi2);
        const int k = RP >= 32 ? 2 * (rank / 32) + (rank / 4) % 2 : 0;
        const int slot = RP >= 32 ? rank % 32 / 8 : rank / 4;
        uint32_t *d = reinterpret_cast<uint32_t *>(s_h + k * 32 + 4 * (row % 8) + slot) + row / 8;
        if (packed) {
            // rows g + 8 have no tokens: the high plane in rows g, the middle one there,
            // then the low one, so that two MMAs take the three
            d[0] = lo2[0], d[1] = lo2[1], d[2] = hi2[0], d[3] = hi2[1];
            d += KS * 32 * 4;
            d[0] = 0, d[1] = lo2[2], d[2] = 0, d[3] = hi2[2];
        } else {
            #pragma unroll
            for (int e = 0; e < kPlanes; ++e, d += KS * 32 * 4) d[0] = lo2[e], d[2] = hi2[e];
        }
    }
    __syncthreads();
    cluster_arrive();                                    // this CTA has read the others' sums

    // ---- y
    {
        // s h's upper fragments stay in registers (read anew for every step they cost 1 of
        // 20 us at 61 tokens)
        uint4 held[2][KS];
        #pragma unroll
        for (int e = 0; e < 2; ++e)
            #pragma unroll
            for (int k = 0; k < KS; ++k) held[e][k] = s_h[(e * KS + k) * 32 + lane];
        for (int nb = n0; nb < n1; nb += PF) {
            if (nb > n0) load_up(nb);
            #pragma unroll
            for (int f = 0; f < PF; ++f) {
                if (nb + f >= n1) break;
                const int mine = (nb + f) * kStepCols + 8 * t;
                float acc[4][4];
                #pragma unroll
                for (int j = 0; j < 4; ++j)
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
                // the low plane first; rows past the tokens hold anything and are not stored
                #pragma unroll
                for (int e = kPlanes - 1; e >= 0; --e)
                    #pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        if (e == 2 && packed) break;
                        const uint4 v = e == 2 ? s_h[(e * KS + k) * 32 + lane] : held[e][k];
                        const uint32_t h[4] = {v.x, v.y, v.z, v.w};
                        #pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t f0 = RP >= 32 ? w[f][(j * QN + k / 2) * 4 + 2 * (k % 2)] : w[f][2 * j];
                            const uint32_t f1 = RP >= 32 ? w[f][(j * QN + k / 2) * 4 + 2 * (k % 2) + 1] : w[f][2 * j + 1];
                            mma_acc(acc[j], h, f0, f1);
                        }
                    }
                if (packed) {
                    #pragma unroll
                    for (int j = 0; j < 4; ++j) acc[j][0] += acc[j][2], acc[j][1] += acc[j][3];
                }
                #pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const long long row = h ? row1 : row0;
                    if (row < 0) continue;
                    uint4 b = base[f];
                    if (h) {
                        b = make_uint4(0, 0, 0, 0);
                        if (p.base) b = load_cols8(p.base + row1 + mine, p.out - mine, p.vec_out);
                    }
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
    cluster_wait();                                      // no CTA leaves while its sums are read
}

// ---------------------------------------------------------------- host side
bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool takes_few(int tokens, int adapters, int rank) {
    const FewLimits m = few_limits(rank);
    return tokens <= m.tokens || (tokens <= m.most && tokens <= m.each * adapters);
}

// Clusters of c CTAs of the kernel that can be resident at once on the current device.
template <int RP>
int resident_clusters(int c, size_t smem) {
    static std::atomic<int> known[64][kMaxCluster + 1];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < 64 && (n = known[dev][c].load(std::memory_order_relaxed)) > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = c;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, lora_few_kernel<RP>, &cfg) != cudaSuccess) return 0;
    if (dev < 64) known[dev][c].store(n, std::memory_order_relaxed);
    return n;
}

// CTAs of a cluster: eight where all clusters can be resident at once, counting one
// per adapter in use and one per 16 tokens.  Measured at 8192 x 8192 with 64
// adapters, 8 / 4 / 2 CTAs: rank 16, 32 tokens 6.8 / 8.0 / 11.9 us, 64 tokens 13.4 /
// 9.8 / 12.3; rank 64, 16 tokens (one cluster of eight too many) 15.6 / 12.4 / 20.0,
// 64 tokens 51.2 / 37.0 / 32.8.
template <int RP>
int few_cluster(int tokens, int adapters, size_t smem) {
    const int used = adapters + tokens / kFewTile, clusters = tokens < used ? tokens : used;
    int c = kMaxCluster;
    while (c > 2 && clusters > resident_clusters<RP>(c, smem)) c /= 2;
    return c;
}

template <int RP>
cudaError_t launch_few(const LoraArgs &p, cudaStream_t s) {
    constexpr size_t smem = size_t(kFewWarps) * kFewTile * (RP + 4) * 4 + kPlanes * (RP / 16) * 32 * sizeof(uint4);
    const cudaError_t e = allow_smem<lora_few_kernel<RP>>(smem);
    if (e != cudaSuccess) return e;
    const int cluster = few_cluster<RP>(p.tokens, p.adapters, smem);
    return launch_chained(lora_few_kernel<RP>, dim3(unsigned(p.tokens) * cluster), kFewThreads, smem, cluster, s, p);
}

cudaError_t launch_lora_few(const LoraArgs &p, cudaStream_t s) {
    switch (padded_rank(p.rank)) {
        case 16: return launch_few<16>(p, s);
        case 32: return launch_few<32>(p, s);
        case 64: return launch_few<64>(p, s);
        default: return launch_few<128>(p, s);
    }
}

size_t round16(size_t b) { return (b + 15) / 16 * 16; }

// Workspace: order [tokens], sizes [adapters], the sort's counts, the partial
// sums (of h, then of the weight gradients), the planes of h or g, and in the
// gradient the planes of g and s h by tile.
struct LoraWorkspace {
    size_t order, sizes, counts, partial, planes, tg, th, total;
};
LoraWorkspace lora_workspace(int tokens, int adapters, int rank, bool backward) {
    LoraWorkspace w;
    w.order = 0;
    w.sizes = round16(size_t(tokens) * 4);
    w.counts = w.sizes + round16(size_t(adapters) * 4);
    w.partial = w.counts + round16(sort_bytes(tokens, adapters));
    w.planes = w.partial + lora_partial_bytes(tokens, adapters, rank, backward);
    w.tg = w.planes + size_t(tokens) * plane_pitch(padded_rank(rank));
    const size_t by_tile = backward ? size_t(lora_max_tiles(tokens, adapters)) * tile_planes(padded_rank(rank)) * 2 : 0;
    w.th = w.tg + by_tile;
    w.total = w.th + by_tile;
    if (!backward && takes_few(tokens, adapters, rank)) w.total = 0;
    return w;
}

w4a16_status check_lora(int tokens, int adapters, int rank, int N, int K) {
    if (tokens < 0 || tokens > (1 << 24) || adapters < 1 || adapters > kMaxGroups) return W4A16_ERR_INVALID_ARG;
    if (rank < 8 || rank > kMaxRank || rank % 8) return W4A16_ERR_UNSUPPORTED;
    if (N < 1 || N > (1 << 24) || K < kGroup || K % kGroup || K > (1 << 20)) return W4A16_ERR_INVALID_ARG;
    return W4A16_OK;
}

w4a16_status from_cuda(cudaError_t e) { return e == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA; }

void place_workspace(LoraArgs *p, char *ws, const LoraWorkspace &w) {
    p->partial = reinterpret_cast<float *>(ws + w.partial);
    p->planes = reinterpret_cast<uint16_t *>(ws + w.planes);
    p->tg = reinterpret_cast<uint16_t *>(ws + w.tg);
    p->th = reinterpret_cast<uint16_t *>(ws + w.th);
}

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
    if (takes_few(tokens, num_adapters, rank)) return from_cuda(launch_lora_few(p, s));
    char *ws = static_cast<char *>(workspace);
    int *order = reinterpret_cast<int *>(ws + w.order), *sizes = reinterpret_cast<int *>(ws + w.sizes);
    cudaError_t e = launch_sort(adapters_dev, id_bytes, tokens, num_adapters,
                                reinterpret_cast<int *>(ws + w.counts), sizes, order, s);
    if (e != cudaSuccess) return W4A16_ERR_CUDA;
    p.order = order, p.sizes = sizes;
    place_workspace(&p, ws, w);
    e = launch_lora_tensor(p, false, kLoraDown, sms, s);
    if (e != cudaSuccess) return W4A16_ERR_CUDA;
    return from_cuda(launch_lora_tensor(p, false, kLoraUp, sms, s));
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
    p.err = device_error_word();
    p.tokens = tokens, p.adapters = num_adapters, p.rank = rank, p.in = N, p.out = K;
    p.vec_in = N % 8 == 0 && aligned(dY, 16);
    p.vec_out = aligned(dX_base, 16) && aligned(dX, 16);
    place_workspace(&p, ws, w);
    e = launch_lora_tensor(p, true, kLoraDown, sms, s);
    if (e != cudaSuccess) return W4A16_ERR_CUDA;
    WgradArgs q = {};
    q.x = X, q.dy = dY, q.tg = p.tg, q.th = p.th, q.order = order, q.sizes = sizes, q.partial = p.partial;
    q.da = dA, q.db = dB, q.err = p.err, q.adapters = num_adapters, q.rank = rank, q.K = K, q.N = N;
    q.vec_dy = p.vec_in;
    // The weight gradients' runs come right after g, while dY is still in L2; dX
    // fills the SMs that they leave, and their sums, which wait for all of them, end.
    e = launch_wgrad(q, kWgradRuns, sms, s);
    if (e == cudaSuccess) e = launch_lora_tensor(p, true, kLoraUp, sms, s);
    if (e != cudaSuccess) return W4A16_ERR_CUDA;
    return from_cuda(launch_wgrad(q, kWgradSums, sms, s));
}

}  // extern "C"
