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
// Ids one CTA ranks at most.
constexpr int kRankIds = 256;
// Up to this many ids every ranking CTA counts all ids itself (one launch).
// Beyond, a counting kernel cuts them into at most kMaxChunks chunks first.
// One launch / three, us, 8 ids a token and 128 groups (8 groups take 0.5 less),
// 2560 and 4096 columns: 4096 ids 7.5 / 9.6 and 9.0 / 11.2, 8192 11.9 / 11.9 and
// 17.6 / 15.7, 16384 24.2 / 19.5 and 38.8 / 30.4, 32768 54.2 / 37.0 and 74.8 / 53.2.
constexpr int kDirectIds = 16384;
constexpr int kMinChunk = 2048;
constexpr int kMaxChunks = 64;
constexpr int kSortThreads = 1024;     // of a CTA of the sort alone: they count, the first kRankIds rank
constexpr int kMaxTopK = 256;
// Rows a thread of the combine kernels holds at once.  Four rather than eight
// lets twice the warps reside: 8192 tokens of 8 rows of 4096 columns took 91.5
// against 101.5 us, the gradients of 4096 of 4 rows of 5120 59.7 against 86.4.
constexpr int kSlotsAtOnce = 4;
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

// VEC consecutive bf16 in one access: 8, 4, 2 or 1, as the rows' starts allow.
template <int VEC>
struct Cols {                                        // of 4 or 2
    static constexpr int W = VEC / 2;
    uint32_t v[W];
    __device__ __forceinline__ void load(const uint16_t *p) {
        if constexpr (W == 2) {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            v[0] = u.x, v[1] = u.y;
        } else {
            v[0] = *reinterpret_cast<const uint32_t *>(p);
        }
    }
    __device__ __forceinline__ void store(uint16_t *p) const {
        if constexpr (W == 2) *reinterpret_cast<uint2 *>(p) = make_uint2(v[0], v[1]);
        else *reinterpret_cast<uint32_t *>(p) = v[0];
    }
    __device__ __forceinline__ void zero() {
        #pragma unroll
        for (int i = 0; i < W; ++i) v[i] = 0;
    }
    __device__ __forceinline__ void unpack(float (&f)[VEC]) const {
        #pragma unroll
        for (int i = 0; i < W; ++i) f[2 * i] = bf16_lo_to_f32(v[i]), f[2 * i + 1] = bf16_hi_to_f32(v[i]);
    }
    __device__ __forceinline__ void pack(const float (&f)[VEC]) {
        #pragma unroll
        for (int i = 0; i < W; ++i) v[i] = pack_bf16x2_rn(f[2 * i], f[2 * i + 1]);
    }
};
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

// The ids' chunks of the counting kernel (n > kDirectIds).
__host__ __device__ __forceinline__ int chunk_ids(int n) {
    const int even = (n + kMaxChunks - 1) / kMaxChunks;
    return even > kMinChunk ? even : kMinChunk;
}

// counts[c][key] over the ids of chunk c: a histogram in shared memory.  Bound by
// latency (one chunk's ids in a few loads a thread): 65536 ids of 128 keys 3.6 us.
template <bool I64>
__global__ void __launch_bounds__(4 * kRouteThreads)
    sort_count_kernel(const void *__restrict__ ids, int *__restrict__ counts, int n, int groups) {
    __shared__ int s_count[kMaxGroups + 1];
    pdl_wait();
    pdl_launch_dependents();
    for (int e = threadIdx.x; e <= groups; e += blockDim.x) s_count[e] = 0;
    __syncthreads();
    const int chunk = chunk_ids(n);
    const int f0 = blockIdx.x * chunk, f1 = min(n, f0 + chunk);
    #pragma unroll 4
    for (int f = f0 + threadIdx.x; f < f1; f += blockDim.x)
        atomicAdd(&s_count[load_key<I64>(ids, f, groups)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= groups; e += blockDim.x)
        counts[(long long)blockIdx.x * (groups + 1) + e] = s_count[e];
}

struct RankSmem {
    int total[kMaxGroups + 1];   // ids of each key
    int next[kMaxGroups + 1];    // place of the key's next id
    int scan[kSortThreads / 32];
    int place[kRankIds];         // ~place for a dropped id
};

// The CTA (THREADS threads) gets the places of ids f0, f0 + 1, ... ready:
// next[key] = ids with a smaller key + ids of this key before f0.  counts (of
// the counting kernel, or nullptr: all ids are counted here) makes a CTA read
// only its own chunk's ids.  Block 0 writes the sizes.
template <bool I64, int THREADS>
__device__ void rank_prepare(RankSmem &sm, const void *ids, const int *counts, int *sizes, int n, int groups,
                             int f0) {
    const int keys = groups + 1, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int e = threadIdx.x; e < keys; e += THREADS) sm.total[e] = sm.next[e] = 0;
    __syncthreads();
    if (counts) {
        const int chunk = chunk_ids(n), chunks = (n + chunk - 1) / chunk, mine = f0 / chunk;
        #pragma unroll 4
        for (int i = threadIdx.x; i < chunks * keys; i += THREADS) {
            const int v = counts[i], c = i / keys, e = i - c * keys;
            if (v == 0) continue;
            atomicAdd(&sm.total[e], v);
            if (c < mine) atomicAdd(&sm.next[e], v);
        }
        #pragma unroll 4
        for (int f = mine * chunk + threadIdx.x; f < f0; f += THREADS)
            atomicAdd(&sm.next[load_key<I64>(ids, f, groups)], 1);
    } else {
        #pragma unroll 4
        for (int f = threadIdx.x; f < n; f += THREADS) {
            const int key = load_key<I64>(ids, f, groups);
            atomicAdd(&sm.total[key], 1);
            if (f < f0) atomicAdd(&sm.next[key], 1);
        }
    }
    __syncthreads();
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int e = threadIdx.x; e < groups; e += THREADS) sizes[e] = sm.total[e];
    // exclusive scan over the keys, a run of them per thread
    const int per = (keys + THREADS - 1) / THREADS;
    const int e0 = min(keys, int(threadIdx.x) * per), e1 = min(keys, e0 + per);
    int sum = 0;
    for (int e = e0; e < e1; ++e) sum += sm.total[e];
    int scan = sum;
    #pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += v;
    }
    if (lane == 31) sm.scan[warp] = scan;
    __syncthreads();
    int start = scan - sum;
    if (e0 < e1)
        for (int w = 0; w < warp; ++w) start += sm.scan[w];
    for (int e = e0; e < e1; ++e) {
        sm.next[e] += start;
        start += sm.total[e];
    }
    __syncthreads();
}

// Places of the next m <= kRankIds ids from f0, into place[].  A warp takes 32
// of them; equal keys find each other through one ballot per key bit (a
// match.any over mostly different keys took several times as long), and the
// warps move the keys' counters one after the other.
template <bool I64>
__device__ void rank_ids(RankSmem &sm, const void *ids, int groups, int f0, int m) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int i = threadIdx.x;
    const int key = i < m ? load_key<I64>(ids, f0 + i, groups) : -1;
    unsigned same = __ballot_sync(0xffffffffu, key >= 0);
    if (key < 0) same = ~same;
    for (int bit = 0; groups >> bit; ++bit) {
        const bool set = (key >> bit) & 1;
        const unsigned with = __ballot_sync(0xffffffffu, set);
        same &= set ? with : ~with;
    }
    const int lead = __ffs(same) - 1;
    for (int w = 0; w < (m + 31) / 32; ++w) {
        if (w == warp) {
            int base = 0;
            if (key >= 0 && lane == lead) {
                base = sm.next[key];
                sm.next[key] = base + __popc(same);
            }
            base = __shfl_sync(0xffffffffu, base, lead);
            const int row = base + __popc(same & ((1u << lane) - 1));
            if (key >= 0) sm.place[i] = key < groups ? row : ~row;
        }
        __syncthreads();
    }
}

// The sort alone: slots[f] = place (~place for a dropped id), order[place] = f;
// either may be nullptr.  Bound by latency (ids, counts, scan, ranks, one after the
// other), so a CTA of 1024 threads counts and its first 256 rank: 65536 ids of 128
// keys 10 us after the counts, 4096 ids of one key 5 us by itself.
template <bool I64>
__global__ void __launch_bounds__(kSortThreads)
    sort_rank_kernel(const void *__restrict__ ids, const int *__restrict__ counts,
                     int *__restrict__ sizes, int *__restrict__ slots, int *__restrict__ order, int n,
                     int groups) {
    __shared__ RankSmem sm;
    pdl_wait();
    pdl_launch_dependents();
    const int f0 = blockIdx.x * kRankIds, m = min(kRankIds, n - f0);
    rank_prepare<I64, kSortThreads>(sm, ids, counts, sizes, n, groups, f0);
    rank_ids<I64>(sm, ids, groups, f0, m);
    if (int(threadIdx.x) < m) {
        const int place = sm.place[threadIdx.x];
        if (slots) slots[f0 + threadIdx.x] = place;
        if (order) order[place < 0 ? ~place : place] = f0 + threadIdx.x;
    }
}

// Token t's columns to the rows of its slots: xs[row(f)] = x[t], read once and
// written top_k times; no arithmetic.  Bound by HBM's writes.  A thread holds one
// access of a token: blocks in token order keep each group's writes together, and
// thousands of small CTAs leave enough stores in flight.  8192 tokens of 8 rows of
// 4096 columns: 89 us, 6.8 TB/s (99.8 with the sort before it).
template <int VEC>
__global__ void __launch_bounds__(kRouteThreads)
    dispatch_copy_kernel(const uint16_t *__restrict__ X, const int *__restrict__ slots,
                         uint16_t *__restrict__ Xs, int top_k, int width) {
    const int t = blockIdx.x;
    const int col = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
    // The sort's CTAs had waited for what came before them when they let this
    // kernel start: X may be read before the sort has ended.
    Cols<VEC> x;
    if (col < width) x.load(X + (long long)t * width + col);
    pdl_wait();
    pdl_launch_dependents();
    if (col >= width) return;
    const int *mine = slots + (long long)t * top_k;
    #pragma unroll 8
    for (int j = 0; j < top_k; ++j) {
        const int slot = mine[j];
        Cols<VEC> v = x;
        if (slot < 0) v.zero();
        v.store(Xs + (long long)(slot < 0 ? ~slot : slot) * width + col);
    }
}

// CTA (b, c) ranks the slots of tokens [b * per, ...) and copies their columns
// of part c: each row is read once and written top_k times.  Bound by latency: the
// ids, the counts and the scan come before the first store.  One launch instead of
// three: one token of 8 rows of 8192 columns 2.9 us, 1322 tokens of 2 rows of 2560
// columns 5.5 us (3.7 TB/s).  Loading X before the ranking, four pieces a thread,
// took 3.2 and 7.4 us.
template <bool I64, int VEC>
__global__ void __launch_bounds__(kRouteThreads)
    dispatch_few_kernel(const uint16_t *__restrict__ X, const void *__restrict__ ids,
                        uint16_t *__restrict__ Xs, int *__restrict__ sizes, int *__restrict__ slots,
                        int tokens, int top_k, int width, int groups, int per) {
    __shared__ RankSmem sm;
    pdl_wait();
    pdl_launch_dependents();
    const int t0 = blockIdx.x * per, t1 = min(tokens, t0 + per);
    const int items = (width + VEC - 1) / VEC;
    const int c0 = int((long long)items * blockIdx.y / gridDim.y);
    const int c1 = int((long long)items * (blockIdx.y + 1) / gridDim.y);
    const int f0 = t0 * top_k, m = (t1 - t0) * top_k;
    rank_prepare<I64, kRouteThreads>(sm, ids, nullptr, sizes, tokens * top_k, groups, f0);
    rank_ids<I64>(sm, ids, groups, f0, m);
    if (blockIdx.y == 0 && int(threadIdx.x) < m) slots[f0 + threadIdx.x] = sm.place[threadIdx.x];
    int t = t0, c = c0 + threadIdx.x;
    while (t < t1) {
        while (c >= c1 && t < t1) c -= c1 - c0, ++t;
        if (t >= t1) break;
        const long long col = (long long)c * VEC;
        Cols<VEC> x;
        x.load(X + (long long)t * width + col);
        const int *mine = sm.place + (t - t0) * top_k;
        #pragma unroll 8
        for (int j = 0; j < top_k; ++j) {
            const int place = mine[j];
            Cols<VEC> v = x;
            if (place < 0) v.zero();
            v.store(Xs + (long long)(place < 0 ? ~place : place) * width + col);
        }
        c += kRouteThreads;
    }
}

__device__ __forceinline__ float load_weight(const void *w, int bytes, long long i) {
    return bytes == 4 ? static_cast<const float *>(w)[i]
                      : bf16_bits_to_f32(static_cast<const uint16_t *>(w)[i]);
}

// y[t] = sum over the kept slots of w * ys[row], in fp32, j ascending, rounded
// once.  w == nullptr: weights of one (the gradient of dispatch).  A slot at
// or past `rows` is skipped.  Bound by HBM's reads, one VEC of a token's columns
// per thread with kSlotsAtOnce rows in flight; gathering by token leaves no atomics
// and a fixed order.  8192 tokens of 8 rows of 4096 columns: 91.4 us, 6.6 TB/s; as
// dispatch's gradient 4096 tokens of 4 rows of 5120 columns: 32.7 us, 6.4 TB/s.
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
    for (int j0 = 0; j0 < top_k; j0 += kSlotsAtOnce) {
        Cols<VEC> v[kSlotsAtOnce];
        bool kept[kSlotsAtOnce];
        #pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j) {
            const int slot = j0 + j < top_k ? slots[f0 + j0 + j] : -1;
            kept[j] = slot >= 0 && slot < rows;
            v[j].zero();
            if (kept[j]) v[j].load(Ys + (long long)slot * width + col);
        }
        #pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j) {
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
// dw[t][j] = <dy[t], ys[row]> in fp32.  kSlotsAtOnce slots a pass.  Bound by HBM:
// dy is read once per pass, ys once, dys written once, and the dot products need the
// token's whole row in one CTA.  4096 tokens of 4 rows of 5120 columns: 59.9 us,
// 6.3 TB/s.
template <int VEC>
__global__ void __launch_bounds__(kRouteThreads)
    combine_backward_kernel(const uint16_t *__restrict__ dY, const uint16_t *__restrict__ Ys,
                            const int *__restrict__ slots, const void *__restrict__ weights,
                            int weight_bytes, uint16_t *__restrict__ dYs, void *__restrict__ dW,
                            int top_k, int rows, int width) {
    __shared__ float s_dot[kSlotsAtOnce][kRouteWarps];
    pdl_wait();
    pdl_launch_dependents();
    const int t = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int warps = blockDim.x / 32;
    for (int j0 = 0; j0 < top_k; j0 += kSlotsAtOnce) {
        const int jn = min(kSlotsAtOnce, top_k - j0);
        const long long f0 = (long long)t * top_k + j0;
        int slot[kSlotsAtOnce];
        float w[kSlotsAtOnce], dot[kSlotsAtOnce];
        #pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j) {
            slot[j] = j < jn ? slots[f0 + j] : 0;
            w[j] = j < jn ? load_weight(weights, weight_bytes, f0 + j) : 0.f;
            dot[j] = 0.f;
        }
        for (int col = threadIdx.x * VEC; col < width; col += blockDim.x * VEC) {
            Cols<VEC> g, v[kSlotsAtOnce];
            g.load(dY + (long long)t * width + col);
            #pragma unroll
            for (int j = 0; j < kSlotsAtOnce; ++j) {
                v[j].zero();
                if (j < jn && slot[j] >= 0 && slot[j] < rows)
                    v[j].load(Ys + (long long)slot[j] * width + col);
            }
            float gf[VEC];
            g.unpack(gf);
            #pragma unroll
            for (int j = 0; j < kSlotsAtOnce; ++j) {
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
        for (int j = 0; j < kSlotsAtOnce; ++j) {
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

// Columns that one access of rows of `width` can take.
int row_vec(int width, const void *a, const void *b, const void *c) {
    for (int v = 8; v > 1; v /= 2)
        if (width % v == 0 && aligned(a, 2 * v) && aligned(b, 2 * v) && aligned(c, 2 * v)) return v;
    return 1;
}

w4a16_status check_routing(int tokens, int top_k, int width) {
    if (tokens < 0 || top_k < 1 || top_k > kMaxTopK || width < 1 || width > (1 << 20)) return W4A16_ERR_INVALID_ARG;
    if ((long long)tokens * top_k > kMaxSlots) return W4A16_ERR_INVALID_ARG;
    if (ceil_div(width, kRouteThreads) > 65535) return W4A16_ERR_INVALID_ARG;
    return W4A16_OK;
}

w4a16_status from_cuda(cudaError_t e) { return e == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA; }

}  // namespace

size_t sort_bytes(int n, int groups) {
    return n <= kDirectIds ? 0 : size_t(ceil_div(n, chunk_ids(n))) * size_t(groups + 1) * sizeof(int);
}

namespace {

template <bool I64>
cudaError_t launch_sort_ids(const void *ids, int n, int groups, int *counts, int *sizes, int *slots,
                            int *order, cudaStream_t s) {
    if (n <= kDirectIds) {
        counts = nullptr;
    } else {
        const cudaError_t e = launch_chained(sort_count_kernel<I64>, dim3(ceil_div(n, chunk_ids(n))),
                                             4 * kRouteThreads, 0, 1, s, ids, counts, n, groups);
        if (e != cudaSuccess) return e;
    }
    return launch_chained(sort_rank_kernel<I64>, dim3(ceil_div(n, kRankIds)), kSortThreads, 0, 1, s, ids,
                          counts, sizes, slots, order, n, groups);
}

// Few ids: one launch, whose CTAs each count all ids, so there are only about
// three per SM (1322 tokens of 2 ids and 2560 columns: 5.5 us, with six per SM
// 8.0), each with at most kRankIds ids; few tokens also split their columns.
// Many ids: the sort, then a copy in token order, whose writes advance through
// every group together (8192 tokens of 8 ids and 4096 columns: 99.8 us; 911
// CTAs that rank and copy nine tokens each took 111).
template <bool I64>
cudaError_t launch_dispatch(const uint16_t *X, const void *ids, uint16_t *Xs, int *sizes, int *slots,
                            int tokens, int top_k, int width, int groups, int *counts, int sms,
                            cudaStream_t s) {
    const int n = tokens * top_k;
    const int vec = row_vec(width, X, Xs, nullptr);
    if (n > kDirectIds) {
        const cudaError_t e = launch_sort_ids<I64>(ids, n, groups, counts, sizes, slots, nullptr, s);
        if (e != cudaSuccess) return e;
        const ColSplit c = col_split(width, vec);
        return launch_chained(vec == 8 ? dispatch_copy_kernel<8> : vec == 4 ? dispatch_copy_kernel<4>
                              : vec == 2 ? dispatch_copy_kernel<2> : dispatch_copy_kernel<1>,
                              dim3(tokens, c.blocks), c.threads, 0, 1, s, X, slots, Xs, top_k, width);
    }
    const int items = ceil_div(width, vec);
    int per = ceil_div(tokens, 3 * sms);
    if (per * top_k > kRankIds) per = kRankIds / top_k;
    if (per < 1) per = 1;
    const int blocks = tokens > 0 ? ceil_div(tokens, per) : 1;
    int parts = ceil_div(2 * sms, blocks);
    if (parts > ceil_div(items, kRouteThreads)) parts = ceil_div(items, kRouteThreads);
    return launch_chained(vec == 8 ? dispatch_few_kernel<I64, 8> : vec == 4 ? dispatch_few_kernel<I64, 4>
                          : vec == 2 ? dispatch_few_kernel<I64, 2> : dispatch_few_kernel<I64, 1>,
                          dim3(blocks, parts), kRouteThreads, 0, 1, s, X, ids, Xs, sizes, slots, tokens, top_k,
                          width, groups, per);
}

}  // namespace

cudaError_t launch_sort(const void *ids, int id_bytes, int n, int groups, int *counts, int *sizes, int *order,
                        cudaStream_t s) {
    return id_bytes == 8 ? launch_sort_ids<true>(ids, n, groups, counts, sizes, nullptr, order, s)
                         : launch_sort_ids<false>(ids, n, groups, counts, sizes, nullptr, order, s);
}

}  // namespace w4a16

using namespace w4a16;

extern "C" {

w4a16_status w4a16_dispatch_workspace_bytes(int tokens, int top_k, int num_groups, size_t *bytes) {
    if (!bytes || num_groups < 1 || num_groups > kMaxGroups) return W4A16_ERR_INVALID_ARG;
    const w4a16_status st = check_routing(tokens, top_k, 1);
    if (st != W4A16_OK) return st;
    *bytes = sort_bytes(tokens * top_k, num_groups);
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
        if (!aligned(X, 2) || !aligned(Xs, 2) || !aligned(ids_dev, id_bytes) || !aligned(slots_dev, 4))
            return W4A16_ERR_INVALID_ARG;
    }
    const size_t need = sort_bytes(tokens * top_k, num_groups);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return W4A16_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned(workspace, 16)) return W4A16_ERR_INVALID_ARG;
    }
    int sms = 0;
    if (device_sm_count(&sms) != 0 || sms < 1) return W4A16_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int *counts = static_cast<int *>(workspace);
    return from_cuda(id_bytes == 8 ? launch_dispatch<true>(X, ids_dev, Xs, M_sizes_dev, slots_dev, tokens,
                                                           top_k, width, num_groups, counts, sms, s)
                                   : launch_dispatch<false>(X, ids_dev, Xs, M_sizes_dev, slots_dev, tokens,
                                                            top_k, width, num_groups, counts, sms, s));
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
    const int vec = row_vec(width, Ys, Y, nullptr);
    const ColSplit c = col_split(width, vec);
    const auto kernel = vec == 8 ? combine_kernel<8> : vec == 4 ? combine_kernel<4>
                        : vec == 2 ? combine_kernel<2> : combine_kernel<1>;
    return from_cuda(launch_chained(kernel, dim3(tokens, c.blocks),
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
    const int vec = row_vec(width, dY, Ys, dYs);
    const ColSplit c = col_split(width, vec);
    const auto kernel = vec == 8 ? combine_backward_kernel<8> : vec == 4 ? combine_backward_kernel<4>
                        : vec == 2 ? combine_backward_kernel<2> : combine_backward_kernel<1>;
    return from_cuda(launch_chained(kernel, dim3(tokens), c.threads, 0, 1, static_cast<cudaStream_t>(stream), dY, Ys,
                                    slots_dev, weights_dev, weight_bytes, dYs, dweights_dev, top_k,
                                    tokens * top_k, width));
}

}  // extern "C"
