// groups.cuh -- groups of ragged sizes that stand on the device, as the products over
// 8-bit rows and the weights' gradients walk them.
#pragma once

#include <cstdint>

namespace w4a16 {

__device__ __forceinline__ int row_tiles(int rows, int bt) { return (rows + bt - 1) / bt; }

// One warp: tab_rows[g] and tab_tiles[g], the first row and the first tile of each group
// and the ends in [groups], where a group of n rows has ceil(n / bt) * per tiles.  A
// negative size counts as 0 (status bit 0), rows at or past M belong to no group (bit 1).
__device__ __forceinline__ void scan_groups(const int32_t *m_sizes, int groups, int M, int bt, int per,
                                            int *tab_rows, int *tab_tiles, int *status_out) {
    const int lane = threadIdx.x & 31;
    int status = 0, tiles = 0;
    long long rows = 0;
    // The sizes of 128 groups are fetched at once.
    int ahead[4];
    for (int g0 = 0; g0 < groups; g0 += 32) {
        const int g = g0 + lane;
        if (g0 % 128 == 0) {
            #pragma unroll
            for (int j = 0; j < 4; ++j) ahead[j] = g + 32 * j < groups ? m_sizes[g + 32 * j] : 0;
        }
        const int given = ahead[0], size = given < 0 ? 0 : given;
        ahead[0] = ahead[1], ahead[1] = ahead[2], ahead[2] = ahead[3];
        if (given < 0) status |= 1;
        long long end = size;
        #pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const long long v = __shfl_up_sync(0xffffffffu, end, d);
            if (lane >= d) end += v;
        }
        end += rows;
        rows = __shfl_sync(0xffffffffu, end, 31);
        if (end > M) status |= 2;
        const int r0 = int(end - size < M ? end - size : M), r1 = int(end < M ? end : M);
        const int mine = row_tiles(r1 - r0, bt) * per;
        int t_end = mine;
        #pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, t_end, d);
            if (lane >= d) t_end += v;
        }
        if (g < groups) tab_rows[g] = r0, tab_tiles[g] = tiles + t_end - mine;
        if (g == groups - 1) tab_rows[groups] = r1, tab_tiles[groups] = tiles + t_end;
        tiles += __shfl_sync(0xffffffffu, t_end, 31);
    }
    status = __reduce_or_sync(0xffffffffu, status);
    if (lane == 0 && status_out) *status_out = status;
}

}  // namespace w4a16
