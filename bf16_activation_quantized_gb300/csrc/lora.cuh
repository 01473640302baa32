// lora.cuh -- what the adapter kernels share: arguments, tiles, cluster and
// copy helpers.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "async.cuh"
#include "common.cuh"

namespace w4a16 {

// h and g enter their second product as a sum of bf16 terms, one plane each (split3).
constexpr int kPlanes = 3;
// Bytes of a sorted token's row of h or g: the planes, high to low, of RP ranks.
__host__ __device__ constexpr int plane_pitch(int RP) { return 2 * kPlanes * RP; }
// The same by tile of 128 tokens of an adapter, for the weight gradients: rows of
// 128 tokens, RP of each plane, zeros past the last token.  In elements.
__host__ __device__ constexpr int tile_planes(int RP) { return kPlanes * RP * 128; }

struct LoraArgs {
    const uint16_t *x;       // [tokens][in]
    const uint16_t *w1;      // forward A [L][r][in]; gradient B [L][in][r]
    const uint16_t *w2;      // forward B [L][out][r]; gradient A [L][r][out]
    const void *ids;
    const int *order, *sizes;   // sorted tokens (the many-token form)
    const float *scale;      // [L]
    const uint16_t *base;    // [tokens][out] or nullptr
    uint16_t *y;             // [tokens][out]
    float *hidden;           // [tokens][r]: forward h, written (or nullptr); gradient: read
    uint16_t *planes;        // of the sorted tokens: s h (gradient: g), see plane_pitch
    uint16_t *tg, *th;       // gradient: planes of g and of s h by tile, see tile_planes
    float *partial;          // partial sums of h (many tokens)
    int *err;
    int id_bytes, tokens, adapters, rank, in, out;
    int vec_in, vec_out;     // rows of x / of base and y start on 16 bytes
};

// Both are instructions of a whole warp (.aligned): its lanes, which may come out of
// loops and branches of their own, meet first.
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
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
__device__ __forceinline__ int ld_cluster1(const int *p, int rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_address(smem_u32(p), rank)) : "memory");
    return v;
}

// Makes ordinary writes of shared memory visible to the tensor core and back.
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or zeros where !in (src is not read then).
__device__ __forceinline__ void cp_async16z(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
// Counts as this thread's arrival once its copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Eight bf16 from column p, `left` of them inside the row.  vec: the row
// starts on 16 bytes and its width is a multiple of 8.  volatile: the load stays
// behind pdl_wait.
__device__ __forceinline__ uint4 load_cols8(const uint16_t *p, int left, int vec) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (vec) {
        if (left > 0)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
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

// Producer: its pieces of a stage are under way.
__device__ __forceinline__ void stage_done(uint32_t bar, bool async) {
    if (async) {
        cp_async_arrive(bar);
    } else {
        cp_async_wait_all();
        mbar_arrive(bar);
    }
}

// The values a, b as sums of three bf16 terms: the upper 8 bits of the 24, the next 8
// and the rest, cut off, so that the sum is the value itself; an infinity stays in the
// first term alone.  Two terms hold 17 bits: a sum that cancels shows the rest.
__device__ __forceinline__ float upper8(float a) { return __uint_as_float(__float_as_uint(a) & 0xffff0000u); }
__device__ __forceinline__ uint32_t upper8x2(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ void split3(float a, float b, uint32_t (&v)[kPlanes]) {
    v[0] = upper8x2(a, b);
    a = isinf(a) ? 0.f : a - upper8(a), b = isinf(b) ? 0.f : b - upper8(b);
    v[1] = upper8x2(a, b);
    v[2] = upper8x2(a - upper8(a), b - upper8(b));
}

__device__ __forceinline__ int adapter_of(const LoraArgs &p, int t) {
    const long long v = p.id_bytes == 8 ? static_cast<const long long *>(p.ids)[t]
                                        : static_cast<const int *>(p.ids)[t];
    return v >= 0 && v < p.adapters ? int(v) : -1;
}

// One warp: the tokens of tile `tile` into rows[], its adapter (-1: none),
// their number and their first place in the sort into out[0..2] (number 0: no
// such tile).
// Few tokens: tile i belongs to token i and exists where the tokens of its
// adapter before it fill whole tiles; it holds that token and the next ones.
template <int TM>
__device__ void find_tile_few(const LoraArgs &p, int tile, int *rows, int *out) {
    const int lane = threadIdx.x & 31;
    const int key = adapter_of(p, tile);
    int before = 0, count = 0;
    #pragma unroll 4
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

// Sorted tokens: adapters' tiles in order, those without an adapter last.  All lanes
// get the tile's adapter, its tokens and their first place in the sort.
struct Tile {
    int adapter, count, start;
};
template <int TM>
__device__ Tile locate_tile(const LoraArgs &p, int tile) {
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
    return {adapter, count, start};
}
template <int TM>
__device__ void find_tile_sorted(const LoraArgs &p, int tile, int *rows, int *out) {
    const int lane = threadIdx.x & 31;
    const Tile t = locate_tile<TM>(p, tile);
    for (int i = lane; i < t.count; i += 32) rows[i] = p.order[t.start + i];
    if (lane == 0) out[0] = t.adapter, out[1] = t.count, out[2] = t.start;
}

struct WgradArgs {
    const uint16_t *x, *dy;        // [tokens][K], [tokens][N]
    const uint16_t *tg, *th;       // g and s h by tile (tile_planes)
    const int *order, *sizes;
    float *partial;                // two tiles of sums per CTA
    uint16_t *da, *db;             // [L][r][K], [L][N][r]
    int *err;
    int adapters, rank, K, N;
    int slices_x, slices;          // column slices of x, of x and dy
    int vec_dy;                    // rows of dy start on 16 bytes, as x's do
};

constexpr int kMaxCluster = 8;

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

// lora_tensor.cu.  lora_partial_bytes: the workspace of the partial sums.
size_t lora_partial_bytes(int tokens, int adapters, int rank, bool backward);
int lora_max_tiles(int tokens, int adapters);
enum LoraStep { kLoraDown, kLoraUp };   // h, published in the planes; y
cudaError_t launch_lora_tensor(const LoraArgs &p, bool trans, LoraStep step, int sms, cudaStream_t s);
enum WgradStep { kWgradRuns, kWgradSums };
cudaError_t launch_wgrad(const WgradArgs &p, WgradStep step, int sms, cudaStream_t s);

inline int padded_rank(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }

}  // namespace w4a16
