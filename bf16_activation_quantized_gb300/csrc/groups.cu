// groups.cu -- the status word of group sizes where there are no rows to multiply.
#include "groups.cuh"

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace w4a16 {

namespace {

__global__ void __launch_bounds__(32) group_status_kernel(const int32_t *m_sizes, int groups, int *status) {
    __shared__ int s_rows[kMaxGroups + 1];
    pdl_wait();
    pdl_launch_dependents();
    scan_groups(m_sizes, groups, 0, 1, 0, s_rows, nullptr, status);
}

}  // namespace

cudaError_t launch_group_status(const int32_t *m_sizes, int groups, int *status, cudaStream_t s) {
    return launch_chained(group_status_kernel, dim3(1), 32, 0, 1, s, m_sizes, groups, status);
}

}  // namespace w4a16
