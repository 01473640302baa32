// routing.cu -- rows in expert order for the grouped product, and back.
//
// dispatch: token t's k ids f = t*k + j name the groups its row goes to.  With
// key(f) = ids[f], or num_groups where ids[f] lies outside [0, num_groups),
//   row(f) = #{f' : key(f') < key(f)} + #{f' < f : key(f') = key(f)},
// a stable counting sort: group by group, inside a group by token.  Dropped
// slots come last; they own the rows no group covers, which are written as
// zeros, and are recorded as ~row(f).  Every output row thus has exactly one
// slot, and the copies, like the gradients, go token by token: a row of X is
// read once and written k times.
#include <cstdint>
#include <cuda_runtime.h>

#include "w4a16.h"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace w4a16 {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
// Ids one CTA of the sort ranks; 8 warps of 256.
constexpr int kSortChunk = 2048;
// Up to this many ids the ranking CTAs count all ids themselves (one launch).
constexpr int kSortDirect = 8 * kSortChunk;
// Up to this many ids every CTA ranks its own token's by counting over all of
// them (one launch); beyond, the counting sort runs first.
constexpr int kCountIds = 4096;
constexpr int kMaxSlots = 1 << 24;     // tokens * top_k

template <bool I64>
__device__ __forceinline__ int load_key(const void *ids, int f, int groups) {
    if (I64) {
        const long long v = static_cast<const long long *>(ids)[f];
        return v >= 0 && v < groups ? int(v) : groups;
    }
    const int v = static_cast<const int *>(ids)[f];
    return v >= 0 && v < groups ? v : groups;
}

// VEC consecutive bf16: 8 (one 16-byte access) or 1.
template <int VEC>
struct Cols;
template <>
struct Cols<8> {
    uint4 v;
    __device__ __forceinline__ void load(const uint16_t *p) { v = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(uint16_t *p) const { *reinterpret_cast<uint4 *>(p) = v; }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void unpack(float (&f)[8]) const {
        f[0] = bf16_lo_to_f32(v.x); f[1] = bf16_hi_to_f32(v.x);
        f[2] = bf16_lo_to_f32(v.y); f[3] = bf16_hi_to_f32(v.y);
        f[4] = bf16_lo_to_f32(v.z); f[5] = bf16_hi_to_f32(v.z);
        f[6] = bf16_lo_to_f32(v.w); f[7] = bf16_hi_to_f32(v.w);
    }
    __device__ __forceinline__ void pack(const float (&f)[8]) {
        v.x = pack_bf16x2_rn(f[0], f[1]);
        v.y = pack_bf16x2_rn(f[2], f[3]);
        v.z = pack_bf16x2_rn(f[4], f[5]);
        v.w = pack_bf16x2_rn(f[6], f[7]);
    }
};
template <>
struct Cols<1> {
    uint16_t v;
    __device__ __forceinline__ void load(const uint16_t *p) { v = *p; }
    __device__ __forceinline__ void store(uint16_t *p) const { *p = v; }
    __device__ __forceinline__ void zero() { v = 0; }
    __device__ __forceinline__ void unpack(float (&f)[1]) const { f[0] = bf16_bits_to_f32(v); }
    __device__ __forceinline__ void pack(const float (&f)[1]) { v = f32_to_bf16_rn(f[0]); }
};

// Few ids: one launch.  CTA (t, c) copies its columns of token t to the rows
// of the token's slots, which it finds by counting: with c(f) = key(f) * 2^13
// + f, row(f) is the number of ids with a smaller c.  CTA (tokens, 0) counts
// the group sizes.
template <bool I64, int VEC>
__global__ void __launch_bounds__(kRouteThreads)
    dispatch_few_kernel(const uint16_t *__restrict__ X, const void *__restrict__ ids,
                        uint16_t *__restrict__ Xs, int *__restrict__ sizes, int *__restrict__ slots,
                        int tokens, int top_k, int width, int groups) {
    __shared__ int s_place[8];
    __shared__ int s_sizes[kMaxGroups];
    pdl_wait();
    pdl_launch_dependents();
    const int n = tokens * top_k;
    const int t = blockIdx.x;
    if (t == tokens) {
        if (blockIdx.y != 0) return;
        for (int e = threadIdx.x; e < groups; e += blockDim.x) s_sizes[e] = 0;
        __syncthreads();
        for (int f = threadIdx.x; f < n; f += blockDim.x) {
            const int key = load_key<I64>(ids, f, groups);
            if (key < groups) atomicAdd(&s_sizes[key], 1);
        }
        __syncthreads();
        for (int e = threadIdx.x; e < groups; e += blockDim.x) sizes[e] = s_sizes[e];
        return;
    }
    const int col = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
    Cols<VEC> x;
    x.zero();
    if (col < width) x.load(X + (long long)t * width + col);
    for (int j0 = 0; j0 < top_k; j0 += 8) {
        const int jn = min(8, top_k - j0);
        int mine[8], below[8];
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int f = t * top_k + j0 + j;
            mine[j] = j < jn ? (load_key<I64>(ids, f, groups) << 13) + f : 0;
            below[j] = 0;
        }
        if (threadIdx.x < 8) s_place[threadIdx.x] = 0;
        __syncthreads();
        for (int f = threadIdx.x; f < n; f += blockDim.x) {
            const int c = (load_key<I64>(ids, f, groups) << 13) + f;
            #pragma unroll
            for (int j = 0; j < 8; ++j) below[j] += c < mine[j] ? 1 : 0;
        }
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int sum = __reduce_add_sync(0xffffffffu, below[j]);
            if ((threadIdx.x & 31) == j && j < jn && sum) atomicAdd(&s_place[j], sum);
        }
        __syncthreads();
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= jn) break;
            const int row = s_place[j];
            const bool kept = (mine[j] >> 13) < groups;
            if (blockIdx.y == 0 && threadIdx.x == 0) slots[t * top_k + j0 + j] = kept ? row : ~row;
            if (col < width) {
                Cols<VEC> v = x;
                if (!kept) v.zero();
                v.store(Xs + (long long)row * width + col);
            }
        }
        __syncthreads();
    }
}

// counter[key] += 1 for every lane with a key (-1: none), one shared-memory
// atomic per distinct key of the warp: ids are often all alike (one adapter).
__device__ __forceinline__ void count_key(int *counter, int key) {
    const unsigned same = __match_any_sync(0xffffffffu, key);
    if (key >= 0 && (threadIdx.x & 31) == __ffs(same) - 1) atomicAdd(&counter[key], __popc(same));
}

// The sort's first pass: counts[c][key] over the ids of chunk c.
template <bool I64>
__global__ void __launch_bounds__(kRouteThreads)
    sort_count_kernel(const void *__restrict__ ids, int *__restrict__ counts, int n, int groups) {
    __shared__ int s_count[kMaxGroups + 1];
    pdl_wait();
    pdl_launch_dependents();
    for (int e = threadIdx.x; e <= groups; e += kRouteThreads) s_count[e] = 0;
    __syncthreads();
    const int f0 = blockIdx.x * kSortChunk + threadIdx.x;
    #pragma unroll
    for (int i = 0; i < kSortChunk; i += kRouteThreads)
        count_key(s_count, f0 + i < n ? load_key<I64>(ids, f0 + i, groups) : -1);
    __syncthreads();
    for (int e = threadIdx.x; e <= groups; e += kRouteThreads)
        counts[(long long)blockIdx.x * (groups + 1) + e] = s_count[e];
}

// The second pass: a chunk's ids in order.  Its CTA sums the chunks' counts
// (all of them for the groups' starts, the earlier ones for its own place in
// each group; with counts == nullptr it counts all ids itself), each warp
// counts its 256 ids, and the warps then rank their ids 32 at a time: equal
// ids of a step find each other by match, the lowest lane moves the group's
// counter.  slots[f] receives the place, order[place] the id's index; either
// may be nullptr.
template <bool I64>
__global__ void __launch_bounds__(kRouteThreads)
    sort_rank_kernel(const void *__restrict__ ids, const int *__restrict__ counts,
                     int *__restrict__ sizes, int *__restrict__ slots, int *__restrict__ order, int n,
                     int groups, int chunks) {
    __shared__ int s_total[kMaxGroups + 1];
    __shared__ int s_next[kRouteWarps][kMaxGroups + 1];
    __shared__ int s_scan[kRouteWarps];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int keys = groups + 1;
    pdl_wait();
    pdl_launch_dependents();
    for (int e = threadIdx.x; e < keys; e += kRouteThreads) s_total[e] = 0;
    for (int i = threadIdx.x; i < kRouteWarps * keys; i += kRouteThreads) s_next[i / keys][i % keys] = 0;
    __syncthreads();
    // s_next[0][e]: ids of key e in earlier chunks
    if (counts) {
        const int all = chunks * keys, before = blockIdx.x * keys;
        for (int i = threadIdx.x; i < all; i += kRouteThreads) {
            const int v = counts[i];
            if (v) {
                atomicAdd(&s_total[i % keys], v);
                if (i < before) atomicAdd(&s_next[0][i % keys], v);
            }
        }
    } else {
        for (int f0 = 0; f0 < n; f0 += kSortChunk) {
            #pragma unroll
            for (int i = 0; i < kSortChunk; i += kRouteThreads) {
                const int f = f0 + i + threadIdx.x;
                const int key = f < n ? load_key<I64>(ids, f, groups) : -1;
                count_key(s_total, key);
                if (f0 < int(blockIdx.x) * kSortChunk) count_key(s_next[0], key);
            }
        }
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e < groups; e += kRouteThreads) sizes[e] = s_total[e];
    // the groups' starts: exclusive scan over the keys, a run of them per thread
    const int per = (keys + kRouteThreads - 1) / kRouteThreads;
    const int e0 = min(keys, int(threadIdx.x) * per), e1 = min(keys, e0 + per);
    int mine = 0;
    for (int e = e0; e < e1; ++e) mine += s_total[e];
    int scan = mine;
    #pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += v;
    }
    if (lane == 31) s_scan[warp] = scan;
    __syncthreads();
    int start = scan - mine;
    for (int w = 0; w < warp; ++w) start += s_scan[w];
    for (int e = e0; e < e1; ++e) {
        s_next[0][e] += start;
        start += s_total[e];
    }
    __syncthreads();
    // each warp's own counts, in the row after its own; then their prefix
    const int f0 = blockIdx.x * kSortChunk + warp * (kSortChunk / kRouteWarps);
    constexpr int kSteps = kSortChunk / kRouteWarps / 32;
    int key[kSteps];
    #pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int f = f0 + 32 * i + lane;
        key[i] = f < n ? load_key<I64>(ids, f, groups) : -1;
        if (warp + 1 < kRouteWarps) count_key(s_next[warp + 1], key[i]);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < keys; e += kRouteThreads) {
        int run = s_next[0][e];
        #pragma unroll
        for (int w = 1; w < kRouteWarps; ++w) {
            run += s_next[w][e];
            s_next[w][e] = run;
        }
    }
    __syncthreads();
    #pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const unsigned same = __match_any_sync(0xffffffffu, key[i]);
        const int lead = __ffs(same) - 1;
        int base = 0;
        if (key[i] >= 0 && lane == lead) {
            base = s_next[warp][key[i]];
            s_next[warp][key[i]] = base + __popc(same);
        }
        base = __shfl_sync(0xffffffffu, base, lead);
        __syncwarp();
        if (key[i] >= 0) {
            const int row = base + __popc(same & ((1u << lane) - 1));
            if (slots) slots[f0 + 32 * i + lane] = key[i] < groups ? row : ~row;
            if (order) order[row] = f0 + 32 * i + lane;
        }
    }
}

// Token t's columns to the rows of its slots.
template <int VEC>
__global__ void __launch_bounds__(kRouteThreads)
    dispatch_copy_kernel(const uint16_t *__restrict__ X, const int *__restrict__ slots,
                         uint16_t *__restrict__ Xs, int top_k, int width) {
    pdl_wait();
    pdl_launch_dependents();
    const int t = blockIdx.x;
    const int col = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
    if (col >= width) return;
    Cols<VEC> x;
    x.load(X + (long long)t * width + col);
    const int *mine = slots + (long long)t * top_k;
    #pragma unroll 8
    for (int j = 0; j < top_k; ++j) {
        const int slot = mine[j];
        Cols<VEC> v = x;
        if (slot < 0) v.zero();
        v.store(Xs + (long long)(slot < 0 ? ~slot : slot) * width + col);
    }
}

__device__ __forceinline__ float load_weight(const void *w, int bytes, long long i) {
    return bytes == 4 ? static_cast<const float *>(w)[i]
                      : bf16_bits_to_f32(static_cast<const uint16_t *>(w)[i]);
}

// y[t] = sum over the kept slots of w * ys[row], in fp32, j ascending, rounded
// once.  w == nullptr: weights of one (the gradient of dispatch).  A slot at
// or past `rows` is skipped.
template <int VEC>
__global__ void __launch_bounds__(kRouteThreads)
    combine_kernel(const uint16_t *__restrict__ Ys, const int *__restrict__ slots,
                   const void *__restrict__ weights, int weight_bytes, uint16_t *__restrict__ Y,
                   int top_k, int rows, int width) {
    pdl_wait();
    pdl_launch_dependents();
    const int t = blockIdx.x;
    const int col = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
    if (col >= width) return;
    const long long f0 = (long long)t * top_k;
    float sum[VEC];
    #pragma unroll
    for (int i = 0; i < VEC; ++i) sum[i] = 0.f;
    for (int j0 = 0; j0 < top_k; j0 += 8) {
        Cols<VEC> v[8];
        bool kept[8];
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int slot = j0 + j < top_k ? slots[f0 + j0 + j] : -1;
            kept[j] = slot >= 0 && slot < rows;
            v[j].zero();
            if (kept[j]) v[j].load(Ys + (long long)slot * width + col);
        }
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (!kept[j]) continue;
            const float w = weights ? load_weight(weights, weight_bytes, f0 + j0 + j) : 1.f;
            float f[VEC];
            v[j].unpack(f);
            #pragma unroll
            for (int i = 0; i < VEC; ++i) sum[i] = fmaf(w, f[i], sum[i]);
        }
    }
    Cols<VEC> y;
    y.pack(sum);
    y.store(Y + (long long)t * width + col);
}

// One CTA per token: dys[row] = w * dy (zeros for a dropped slot's own row),
// dw[t][j] = <dy[t], ys[row]> in fp32.  Eight slots a pass.
template <int VEC>
__global__ void __launch_bounds__(kRouteThreads)
    combine_backward_kernel(const uint16_t *__restrict__ dY, const uint16_t *__restrict__ Ys,
                            const int *__restrict__ slots, const void *__restrict__ weights,
                            int weight_bytes, uint16_t *__restrict__ dYs, void *__restrict__ dW,
                            int top_k, int rows, int width) {
    __shared__ float s_dot[8][kRouteWarps];
    pdl_wait();
    pdl_launch_dependents();
    const int t = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int warps = blockDim.x / 32;
    for (int j0 = 0; j0 < top_k; j0 += 8) {
        const int jn = min(8, top_k - j0);
        const long long f0 = (long long)t * top_k + j0;
        int slot[8];
        float w[8], dot[8];
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
            slot[j] = j < jn ? slots[f0 + j] : 0;
            w[j] = j < jn ? load_weight(weights, weight_bytes, f0 + j) : 0.f;
            dot[j] = 0.f;
        }
        for (int col = threadIdx.x * VEC; col < width; col += blockDim.x * VEC) {
            Cols<VEC> g, v[8];
            g.load(dY + (long long)t * width + col);
            #pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j].zero();
                if (j < jn && slot[j] >= 0 && slot[j] < rows)
                    v[j].load(Ys + (long long)slot[j] * width + col);
            }
            float gf[VEC];
            g.unpack(gf);
            #pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j >= jn) break;
                const bool kept = slot[j] >= 0 && slot[j] < rows;
                const int row = slot[j] >= 0 ? slot[j] : ~slot[j];
                float f[VEC], out[VEC];
                v[j].unpack(f);
                #pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    if (kept) dot[j] = fmaf(gf[i], f[i], dot[j]);
                    out[i] = kept ? w[j] * gf[i] : 0.f;
                }
                Cols<VEC> o;
                o.pack(out);
                if (row < rows) o.store(dYs + (long long)row * width + col);
            }
        }
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
            #pragma unroll
            for (int d = 16; d > 0; d /= 2) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
            if (lane == 0) s_dot[j][warp] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < jn) {
            float sum = 0.f;
            for (int i = 0; i < warps; ++i) sum += s_dot[threadIdx.x][i];
            if (weight_bytes == 4)
                static_cast<float *>(dW)[f0 + threadIdx.x] = sum;
            else
                static_cast<uint16_t *>(dW)[f0 + threadIdx.x] = f32_to_bf16_rn(sum);
        }
        __syncthreads();
    }
}

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int ceil_div(long long a, long long b) { return int((a + b - 1) / b); }

// Column blocks of up to 256 threads with one VEC each, evened out.
struct ColSplit {
    int blocks, threads;
};
ColSplit col_split(int width, int vec) {
    const int items = ceil_div(width, vec);
    ColSplit c;
    c.blocks = ceil_div(items, kRouteThreads);
    c.threads = ceil_div(ceil_div(items, c.blocks), 32) * 32;
    return c;
}

w4a16_status check_routing(int tokens, int top_k, int width) {
    if (tokens < 0 || top_k < 1 || width < 1 || width > (1 << 20)) return W4A16_ERR_INVALID_ARG;
    if ((long long)tokens * top_k > kMaxSlots) return W4A16_ERR_INVALID_ARG;
    if (ceil_div(width, kRouteThreads) > 65535) return W4A16_ERR_INVALID_ARG;
    return W4A16_OK;
}

w4a16_status from_cuda(cudaError_t e) { return e == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA; }

size_t dispatch_sort_bytes(int n, int groups) { return n <= kCountIds ? 0 : sort_bytes(n, groups); }

}  // namespace

size_t sort_bytes(int n, int groups) {
    return n <= kSortDirect ? 0 : size_t(ceil_div(n, kSortChunk)) * size_t(groups + 1) * sizeof(int);
}

cudaError_t launch_sort(const void *ids, int id_bytes, int n, int groups, int *counts, int *sizes,
                        int *slots, int *order, cudaStream_t s) {
    const int chunks = ceil_div(n, kSortChunk);
    if (n <= kSortDirect) {
        counts = nullptr;
    } else {
        const cudaError_t e = launch_chained(id_bytes == 8 ? sort_count_kernel<true> : sort_count_kernel<false>,
                                             dim3(chunks), kRouteThreads, 0, 1, s, ids, counts, n, groups);
        if (e != cudaSuccess) return e;
    }
    return launch_chained(id_bytes == 8 ? sort_rank_kernel<true> : sort_rank_kernel<false>, dim3(chunks),
                          kRouteThreads, 0, 1, s, ids, counts, sizes, slots, order, n, groups, chunks);
}

namespace {

template <bool I64>
cudaError_t launch_dispatch(const uint16_t *X, const void *ids, uint16_t *Xs, int *sizes, int *slots,
                            int tokens, int top_k, int width, int groups, int *counts, cudaStream_t s) {
    const bool vec = width % 8 == 0;
    const ColSplit c = col_split(width, vec ? 8 : 1);
    const int n = tokens * top_k;
    if (n <= kCountIds) {
        const dim3 grid(tokens + 1, c.blocks);
        return launch_chained(vec ? dispatch_few_kernel<I64, 8> : dispatch_few_kernel<I64, 1>, grid,
                              c.threads, 0, 1, s, X, ids, Xs, sizes, slots, tokens, top_k, width, groups);
    }
    cudaError_t e = launch_sort(ids, I64 ? 8 : 4, n, groups, counts, sizes, slots, nullptr, s);
    if (e != cudaSuccess) return e;
    return launch_chained(vec ? dispatch_copy_kernel<8> : dispatch_copy_kernel<1>,
                          dim3(tokens, c.blocks), c.threads, 0, 1, s, X, slots, Xs, top_k, width);
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

w4a16_status w4a16_dispatch_workspace_bytes(int tokens, int top_k, int num_groups, size_t *bytes) {
    if (!bytes || num_groups < 1 || num_groups > kMaxGroups) return W4A16_ERR_INVALID_ARG;
    const w4a16_status st = check_routing(tokens, top_k, 1);
    if (st != W4A16_OK) return st;
    *bytes = dispatch_sort_bytes(tokens * top_k, num_groups);
    return W4A16_OK;
}

w4a16_status w4a16_dispatch(const w4a16_bf16 *X, const void *ids_dev, int id_bytes, w4a16_bf16 *Xs,
                            int32_t *M_sizes_dev, int32_t *slots_dev, int tokens, int top_k, int width,
                            int num_groups, void *workspace, size_t workspace_bytes, void *stream) {
    const w4a16_status st = check_routing(tokens, top_k, width);
    if (st != W4A16_OK) return st;
    if (id_bytes != 4 && id_bytes != 8) return W4A16_ERR_UNSUPPORTED;
    if (num_groups < 1 || num_groups > kMaxGroups) return W4A16_ERR_INVALID_ARG;
    if (!M_sizes_dev || !aligned(M_sizes_dev, 4)) return W4A16_ERR_INVALID_ARG;
    if (tokens > 0) {
        if (!X || !ids_dev || !Xs || !slots_dev) return W4A16_ERR_INVALID_ARG;
        if (!aligned(X, 16) || !aligned(Xs, 16) || !aligned(ids_dev, id_bytes) || !aligned(slots_dev, 4))
            return W4A16_ERR_INVALID_ARG;
    }
    const size_t need = dispatch_sort_bytes(tokens * top_k, num_groups);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return W4A16_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned(workspace, 16)) return W4A16_ERR_INVALID_ARG;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int *counts = static_cast<int *>(workspace);
    return from_cuda(id_bytes == 8 ? launch_dispatch<true>(X, ids_dev, Xs, M_sizes_dev, slots_dev, tokens,
                                                           top_k, width, num_groups, counts, s)
                                   : launch_dispatch<false>(X, ids_dev, Xs, M_sizes_dev, slots_dev, tokens,
                                                            top_k, width, num_groups, counts, s));
}

w4a16_status w4a16_combine(const w4a16_bf16 *Ys, const int32_t *slots_dev, const void *weights_dev,
                           int weight_bytes, w4a16_bf16 *Y, int tokens, int top_k, int width,
                           void *stream) {
    const w4a16_status st = check_routing(tokens, top_k, width);
    if (st != W4A16_OK) return st;
    if (weights_dev && weight_bytes != 4 && weight_bytes != 2) return W4A16_ERR_UNSUPPORTED;
    if (tokens == 0) return W4A16_OK;
    if (!Ys || !slots_dev || !Y) return W4A16_ERR_INVALID_ARG;
    if (!aligned(Ys, 2) || !aligned(Y, 2) || !aligned(slots_dev, 4) ||
        (weights_dev && !aligned(weights_dev, weight_bytes)))
        return W4A16_ERR_INVALID_ARG;
    const bool vec = width % 8 == 0 && aligned(Ys, 16) && aligned(Y, 16);
    const ColSplit c = col_split(width, vec ? 8 : 1);
    return from_cuda(launch_chained(vec ? combine_kernel<8> : combine_kernel<1>, dim3(tokens, c.blocks),
                                    c.threads, 0, 1, static_cast<cudaStream_t>(stream), Ys, slots_dev,
                                    weights_dev, weight_bytes, Y, top_k, tokens * top_k, width));
}

w4a16_status w4a16_combine_backward(const w4a16_bf16 *dY, const w4a16_bf16 *Ys, const int32_t *slots_dev,
                                    const void *weights_dev, int weight_bytes, w4a16_bf16 *dYs,
                                    void *dweights_dev, int tokens, int top_k, int width, void *stream) {
    const w4a16_status st = check_routing(tokens, top_k, width);
    if (st != W4A16_OK) return st;
    if (weight_bytes != 4 && weight_bytes != 2) return W4A16_ERR_UNSUPPORTED;
    if (tokens == 0) return W4A16_OK;
    if (!dY || !Ys || !slots_dev || !weights_dev || !dYs || !dweights_dev) return W4A16_ERR_INVALID_ARG;
    if (!aligned(dY, 2) || !aligned(Ys, 2) || !aligned(dYs, 2) || !aligned(slots_dev, 4) ||
        !aligned(weights_dev, weight_bytes) || !aligned(dweights_dev, weight_bytes))
        return W4A16_ERR_INVALID_ARG;
    const bool vec = width % 8 == 0 && aligned(dY, 16) && aligned(Ys, 16) && aligned(dYs, 16);
    const ColSplit c = col_split(width, vec ? 8 : 1);
    return from_cuda(launch_chained(vec ? combine_backward_kernel<8> : combine_backward_kernel<1>,
                                    dim3(tokens), c.threads, 0, 1, static_cast<cudaStream_t>(stream), dY, Ys,
                                    slots_dev, weights_dev, weight_bytes, dYs, dweights_dev, top_k,
                                    tokens * top_k, width));
}

}  // extern "C"
