// fp8.cuh -- what the products in 8-bit floating point share: arguments and launchers.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "split_plan.h"

namespace w4a16 {

// Both kernels multiply a row's scale by the weights' first, one product a row and block.
// Where fp32 does not hold it (below 2^-126, from 2^128 on) a term that it would hold is
// lost: the calls exclude such scales.  Sums multiplied by 2^64 or 2^-64 beforehand in that case
// cost every call 1 to 10 % even where no block took that path (4096 x 8192 x 8192: 187 to 192 us,
// 61 x 2560 x 9728: 11.6 to 12.7), two factors for every element more than the adding warps have.
struct Fp8Args {
    const float *xs;         // [blocks][M]
    const float *ws;         // [groups][ceil(N / 128)][K / 128]
    uint16_t *y;             // [M][out]
    const int32_t *m_sizes;  // nullptr: one group of M rows
    int *status, *err;
    long long ws_group;      // scales of a group's weights
    int ws_tile, ws_block;   // from one output tile's scale to the next one's, from one summed block's
    int M, out, blocks;      // rows, output columns, blocks of 128 that are summed over
    int out_tiles, groups;   // tiles of 128 output columns (many rows: of 256)
    int bt;                  // rows of x per tile at most (a multiple of 16)
    int stages;              // ring depth
    int vec;                 // rows of y start on 16 bytes and hold a multiple of 8 columns
    int resident;            // the weights may be read before the stream's previous kernel has ended
};

cudaError_t launch_fp8_gemm(const Fp8Plan &p, Fp8Args a, const uint8_t *x, const uint8_t *w, int N, int K,
                            bool trans, cudaStream_t s);
cudaError_t launch_fp8_many(const Fp8Plan &p, const Fp8Args &a, const CUtensorMap &tx, const CUtensorMap &tw,
                            bool trans, cudaStream_t s);
cudaError_t launch_quantize_rows(const uint16_t *x, uint8_t *codes, float *scales, int rows, int width,
                                 cudaStream_t s);
cudaError_t launch_quantize_blocks(const uint16_t *w, uint8_t *codes, float *scales, int groups, int rows,
                                   int width, cudaStream_t s);

}  // namespace w4a16
