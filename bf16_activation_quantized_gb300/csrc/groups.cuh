// groups.cuh -- groups of ragged sizes that stand on the device, as the products over
// 8-bit rows and the weights' gradients walk them.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace w4a16 {

// The status word alone, for calls without rows.
cudaError_t launch_group_status(const int32_t *m_sizes, int groups, int *status, cudaStream_t s);

__device__ __forceinline__ int row_tiles(int rows, int bt) { return (rows + bt - 1) / bt; }

// Tile r of a grid of `rows` by `cols`, in bands of kBand rows, down a band's columns: the
// tiles that run at the same time form a block and share both operands' tiles in L2.  (Row
// by row, the weight gradient of 4096 x 8192 x 8192 took 304 us instead of 284, the 8-bit
// product of these sizes 193 instead of 187; bands of 4, 8 and 32 lie between.)
constexpr int kBand = 16;
__device__ __forceinline__ void banded(int r, int rows, int cols, int &row, int &col) {
    const int band = r / (kBand * cols), in_band = r - band * (kBand * cols);
    const int height = min(kBand, rows - band * kBand);
    col = in_band / height;
    row = band * kBand + in_band - col * height;
}

// One warp: tab_rows[g] and tab_tiles[g], the first row and the first tile of each group
// (unless nullptr) and the ends in [groups], where a group of n rows has ceil(n / bt) * per tiles.  A
// negative size counts as 0 (status bit 0), rows at or past M belong to no group (bit 1).
__device__ __forceinline__ void scan_groups(const int32_t *m_sizes, int groups, int M, int bt, int per,
                                            int *tab_rows, int *tab_tiles, int *status_out) {
    constexpr int kEach = 4;                     // groups a lane takes at a time
    const int lane = threadIdx.x & 31;
    int status = 0, tiles = 0;
    long long rows = 0;
    for (int g0 = 0; g0 < groups; g0 += 32 * kEach) {
        const int first = g0 + kEach * lane;
        int size[kEach], mine[kEach];
        #pragma unroll
        for (int j = 0; j < kEach; ++j) size[j] = first + j < groups ? m_sizes[first + j] : 0;
        long long end = 0;
        #pragma unroll
        for (int j = 0; j < kEach; ++j) {
            if (size[j] < 0) status |= 1, size[j] = 0;
            end += size[j];
        }
        long long row = end;
        #pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const long long v = __shfl_up_sync(0xffffffffu, end, d);
            if (lane >= d) end += v;
        }
        row = rows + end - row;                  // the lane's first
        rows += __shfl_sync(0xffffffffu, end, 31);
        int t_end = 0;
        #pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int r0 = int(row < M ? row : M);
            row += size[j];
            const int r1 = int(row < M ? row : M);
            if (first + j < groups) tab_rows[first + j] = r0;
            if (first + j == groups - 1) tab_rows[groups] = r1;
            mine[j] = row_tiles(r1 - r0, bt) * per;
            t_end += mine[j];
        }
        if (row > M) status |= 2;
        int tile = t_end;
        #pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, t_end, d);
            if (lane >= d) t_end += v;
        }
        tile = tiles + t_end - tile;
        tiles += __shfl_sync(0xffffffffu, t_end, 31);
        #pragma unroll
        for (int j = 0; j < kEach; ++j) {
            if (tab_tiles && first + j < groups) tab_tiles[first + j] = tile;
            tile += mine[j];
            if (tab_tiles && first + j == groups - 1) tab_tiles[groups] = tile;
        }
    }
    status = __reduce_or_sync(0xffffffffu, status);
    if (lane == 0 && status_out) *status_out = status;
}

}  // namespace w4a16
