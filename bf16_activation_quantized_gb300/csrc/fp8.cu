// fp8.cu -- bf16 rows and weights in 8-bit floating point (e4m3), a scale for 128
// elements of a row or for a block of 128 x 128; the entry points of these products.
//
// A block's scale is max |x| / 448 and its codes are 448 x / max |x|, rounded to the
// nearest e4m3, ties to even: exactly, at the cost of one product.  448 x is
// 7 x 2^6 with 11 significant bits, max |x| has 8 and a border between two codes has
// 5: a quotient that is not a border is 2^-13 of it away at least.  The factor
// 448 / max is therefore taken one step up (2^-23), so that a quotient on a border
// comes out on it or just above, and the product's last 8 bits are dropped (2^-15),
// which puts the former back on the border and moves no other across one.
//
// Both kernels are bound by memory: one pass, 16 bytes a lane, half a warp for the 128
// elements of a row's block.
#include "async.cuh"
#include "common.cuh"
#include "fp8.cuh"
#include "groups.cuh"
#include "internal.h"
#include "launch.cuh"
#include "w4a16.h"

namespace w4a16 {

namespace {

// Eight bf16 as they lie in memory; element by element where rows start anywhere.
// volatile: the load stays behind pdl_wait (the rows are what the stream's previous kernel
// wrote, as a rule).
__device__ __forceinline__ uint4 load8(const uint16_t *p, int left, bool vec) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (left <= 0) return v;
    if (vec) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
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

// The largest magnitude of eight bf16, as a bf16's bits: magnitudes order like their
// bits, and a NaN above infinity.
__device__ __forceinline__ uint32_t most8(const uint4 &v) {
    const uint32_t m = 0x7fff7fffu;
    const uint32_t a = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
    return max(a & 0xffffu, a >> 16);
}

// What turns x into 448 x / most: x * up * by (up: a power of two that keeps the factor of
// the smallest blocks finite).
struct Factor {
    float up, by;
};
__device__ __forceinline__ Factor factor_of(float most) {
    Factor f;
    f.up = most < 0x1p-60f ? 0x1p64f : 1.f;
    const float q = 448.f / (most * f.up);
    // most = 0: all codes are 0; infinite: finite elements are 0, infinite ones NaN
    f.by = most > 0.f && q > 0.f ? __uint_as_float(__float_as_uint(q) + 1) : most > 0.f ? 0.f : most;
    return f;
}

__device__ __forceinline__ uint32_t code2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(r) : "f"(__uint_as_float(__float_as_uint(hi) & 0xffffff00u)),
                    "f"(__uint_as_float(__float_as_uint(lo) & 0xffffff00u)));
    return r;
}
__device__ __forceinline__ uint2 code8(const uint4 &v, Factor f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
        if (f.up != 1.f) lo *= f.up, hi *= f.up;
        c[i] = code2(lo * f.by, hi * f.by);
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

// The largest of 16 lanes' values, in all of them.
__device__ __forceinline__ uint32_t most16(uint32_t m) {
    #pragma unroll
    for (int d = 1; d < 16; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    return m;
}

constexpr int kQuantThreads = 128, kQuantRows = kQuantThreads / 16;

// A CTA takes 8 rows and J blocks of 128 columns, half a warp a row; the scales leave
// through shared memory, since those of neighbouring rows stand together.  65536 x 4096:
// 122 us, 0.98 of the measured copy bandwidth (16 rows, 4 blocks: 133 us; 2 blocks: 156).
// PAD: the last block of a row has columns past the width.
template <int J, bool VEC, bool PAD>
__global__ void __launch_bounds__(kQuantThreads) quantize_rows_kernel(const uint16_t *x, uint8_t *codes,
                                                                      float *scales, int rows, int width,
                                                                      int blocks) {
    __shared__ float s_scale[J][kQuantRows];
    pdl_wait();
    pdl_launch_dependents();
    const int half = threadIdx.x / 16, piece = threadIdx.x % 16;
    const long long row0 = (long long)blockIdx.x * kQuantRows, row = row0 + half;
    const int block0 = blockIdx.y * J;
    uint4 v[J];
    #pragma unroll
    for (int j = 0; j < J; ++j) {
        const int col = (block0 + j) * kFp8Block + 8 * piece;
        v[j] = load8(x + row * width + col, row < rows ? width - col : 0, VEC);
    }
    #pragma unroll
    for (int j = 0; j < J; ++j) {
        const float most = bf16_value(most16(most8(v[j])));
        if (piece == 0) s_scale[j][half] = most / 448.f;
        if (row < rows && block0 + j < blocks)
            *reinterpret_cast<uint2 *>(codes + (row * blocks + block0 + j) * kFp8Block + 8 * piece) =
                code8(v[j], factor_of(most));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < J * kQuantRows; i += kQuantThreads) {
        const int j = i / kQuantRows, r = i % kQuantRows;
        if (block0 + j < blocks && row0 + r < rows)
            scales[(long long)(block0 + j) * rows + row0 + r] = s_scale[j][r];
    }
    // In a block that holds a NaN the columns past the width, 0 times NaN, become zeros again.
    const int last = blocks - 1 - block0;
    if (PAD && last < J && row < rows && s_scale[last][half] != s_scale[last][half]) {
        const int left = width - (blocks - 1) * kFp8Block - 8 * piece;
        for (int e = max(left, 0); e < 8; ++e) codes[(row * blocks + blocks - 1) * kFp8Block + 8 * piece + e] = 0;
    }
}

// A CTA takes a block of 128 x 128, half a warp 16 of its rows.  8 x 2048 x 4096: 32.6 us,
// 0.91 of the measured copy bandwidth (256 threads: 34.0 us).
__global__ void __launch_bounds__(kQuantThreads) quantize_blocks_kernel(const uint16_t *w, uint8_t *codes,
                                                                        float *scales, int rows, int width,
                                                                        int row_blocks) {
    constexpr int kEach = kFp8Block / kQuantRows;
    __shared__ uint32_t s_most[kQuantThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int half = threadIdx.x / 16, piece = threadIdx.x % 16;
    const int col_blocks = width / kFp8Block;
    const int rb = blockIdx.x / col_blocks, cb = blockIdx.x % col_blocks;
    const long long base = (long long)blockIdx.y * rows * width + (long long)rb * kFp8Block * width + cb * kFp8Block;
    const int left = rows - rb * kFp8Block;
    uint4 v[kEach];
    uint32_t m = 0;
    #pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int r = half + kQuantRows * i;
        v[i] = load8(w + base + (long long)r * width + 8 * piece, r < left ? 8 : 0, true);
    }
    #pragma unroll
    for (int i = 0; i < kEach; ++i) m = max(m, most8(v[i]));
    m = __reduce_max_sync(0xffffffffu, m);
    if (threadIdx.x % 32 == 0) s_most[threadIdx.x / 32] = m;
    __syncthreads();
    #pragma unroll
    for (int i = 0; i < kQuantThreads / 32; ++i) m = max(m, s_most[i]);
    const float most = bf16_value(m);
    const Factor f = factor_of(most);
    #pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int r = half + kQuantRows * i;
        if (r < left) *reinterpret_cast<uint2 *>(codes + base + (long long)r * width + 8 * piece) = code8(v[i], f);
    }
    if (threadIdx.x == 0) scales[(long long)blockIdx.y * row_blocks * col_blocks + blockIdx.x] = most / 448.f;
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
w4a16_status from_cuda(cudaError_t e) { return e == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA; }

}  // namespace

cudaError_t launch_quantize_rows(const uint16_t *x, uint8_t *codes, float *scales, int rows, int width,
                                 cudaStream_t s) {
    const int blocks = (width + kFp8Block - 1) / kFp8Block;
    const bool vec = width % 8 == 0 && aligned(x, 16);
    const dim3 grid((rows + kQuantRows - 1) / kQuantRows);
    // Eight blocks a CTA once that leaves every SM several CTAs, else one for latency.
    constexpr int J = 8;
    const bool many = (long long)grid.x * blocks >= 8192;
    const dim3 g(grid.x, many ? (blocks + J - 1) / J : blocks);
    const auto launch = [&](auto kernel) {
        return launch_chained(kernel, g, kQuantThreads, 0, 1, s, x, codes, scales, rows, width, blocks);
    };
    if (width % kFp8Block == 0 && vec)
        return many ? launch(quantize_rows_kernel<J, true, false>) : launch(quantize_rows_kernel<1, true, false>);
    if (vec) return many ? launch(quantize_rows_kernel<J, true, true>) : launch(quantize_rows_kernel<1, true, true>);
    return many ? launch(quantize_rows_kernel<J, false, true>) : launch(quantize_rows_kernel<1, false, true>);
}

cudaError_t launch_quantize_blocks(const uint16_t *w, uint8_t *codes, float *scales, int groups, int rows,
                                   int width, cudaStream_t s) {
    const int row_blocks = (rows + kFp8Block - 1) / kFp8Block;
    return launch_chained(quantize_blocks_kernel, dim3(row_blocks * (width / kFp8Block), groups), kQuantThreads, 0, 1,
                          s, w, codes, scales, rows, width, row_blocks);
}

namespace {

constexpr int kMost = 1 << 24, kMostSummed = 1 << 20;

w4a16_status fp8_product(const uint8_t *X, const float *x_scales, const uint8_t *W, const float *w_scales,
                         const int32_t *m_sizes, w4a16_bf16 *Y, int groups, int M, int N, int K, int transposed,
                         int resident, int *status, cudaStream_t s) {
    if (M < 0 || M > kMost || N < 1 || N > kMost || K < kFp8Block || K % kFp8Block || K > kMostSummed)
        return W4A16_ERR_INVALID_ARG;
    if (transposed && N > kMostSummed) return W4A16_ERR_INVALID_ARG;
    const int out = transposed ? K : N;
    if ((long long)M * out > (1LL << 40)) return W4A16_ERR_INVALID_ARG;
    if (M == 0 && !m_sizes) return W4A16_OK;
    if (M > 0 && (!X || !x_scales || !W || !w_scales || !Y)) return W4A16_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(W, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) || !aligned(Y, 2))
        return W4A16_ERR_INVALID_ARG;
    if (M == 0) return from_cuda(launch_group_status(m_sizes, groups, status, s));
    int sms = 0;
    if (device_sm_count(&sms) != 0 || sms < 1) return W4A16_ERR_CUDA;
    const int n_blocks = (N + kFp8Block - 1) / kFp8Block, k_blocks = K / kFp8Block;
    Fp8Args a = {};
    a.xs = x_scales, a.ws = w_scales, a.y = Y, a.m_sizes = m_sizes, a.status = status;
    a.err = device_error_word();
    if (!a.err) return W4A16_ERR_CUDA;
    a.ws_group = (long long)n_blocks * k_blocks;
    a.ws_tile = transposed ? 1 : k_blocks, a.ws_block = transposed ? k_blocks : 1;
    a.M = M, a.out = out, a.blocks = transposed ? n_blocks : k_blocks;
    a.out_tiles = (out + kFp8Block - 1) / kFp8Block, a.groups = groups;
    a.vec = out % 8 == 0 && aligned(Y, 16);
    a.resident = resident;
    const Fp8Plan p = fp8_plan(M, out, a.blocks, groups, m_sizes != nullptr, sms);
    return from_cuda(launch_fp8_gemm(p, a, X, W, N, K, transposed != 0, s));
}

}  // namespace

}  // namespace w4a16

using namespace w4a16;

extern "C" {

w4a16_status w4a16_quantize_fp8(const w4a16_bf16 *X, uint8_t *codes, float *scales, int rows, int width,
                                void *stream) {
    if (rows < 0 || rows > kMost || width < 1 || width > kMostSummed) return W4A16_ERR_INVALID_ARG;
    if (rows == 0) return W4A16_OK;
    if (!X || !codes || !scales) return W4A16_ERR_INVALID_ARG;
    if (!aligned(X, 2) || !aligned(codes, 16) || !aligned(scales, 4)) return W4A16_ERR_INVALID_ARG;
    return from_cuda(launch_quantize_rows(X, codes, scales, rows, width, static_cast<cudaStream_t>(stream)));
}

w4a16_status w4a16_quantize_fp8_blocks(const w4a16_bf16 *W, uint8_t *codes, float *scales, int num_groups, int N,
                                       int K, void *stream) {
    if (num_groups < 1 || num_groups > kMaxGroups || N < 1 || N > kMost || K < kFp8Block || K % kFp8Block ||
        K > kMostSummed)
        return W4A16_ERR_INVALID_ARG;
    if (!W || !codes || !scales) return W4A16_ERR_INVALID_ARG;
    if (!aligned(W, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return W4A16_ERR_INVALID_ARG;
    return from_cuda(launch_quantize_blocks(W, codes, scales, num_groups, N, K, static_cast<cudaStream_t>(stream)));
}

w4a16_status w4a16_gemm_fp8(const uint8_t *X, const float *x_scales, const uint8_t *W, const float *w_scales,
                            w4a16_bf16 *Y, int M, int N, int K, int transposed, int flags, void *stream) {
    if (flags & ~W4A16_FLAG_RESIDENT_WEIGHTS) return W4A16_ERR_INVALID_ARG;
    return fp8_product(X, x_scales, W, w_scales, nullptr, Y, 1, M, N, K, transposed,
                       flags & W4A16_FLAG_RESIDENT_WEIGHTS, nullptr, static_cast<cudaStream_t>(stream));
}

w4a16_status w4a16_gemm_fp8_grouped(const uint8_t *X, const float *x_scales, const uint8_t *W,
                                    const float *w_scales, const int32_t *M_sizes_dev, w4a16_bf16 *Y,
                                    int num_groups, int M_total, int N, int K, int transposed, int32_t *status_dev,
                                    void *stream) {
    if (num_groups < 1 || num_groups > kMaxGroups) return W4A16_ERR_INVALID_ARG;
    if (!M_sizes_dev || !status_dev || !aligned(M_sizes_dev, 4) || !aligned(status_dev, 4))
        return W4A16_ERR_INVALID_ARG;
    return fp8_product(X, x_scales, W, w_scales, M_sizes_dev, Y, num_groups, M_total, N, K, transposed, 0,
                       status_dev, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
