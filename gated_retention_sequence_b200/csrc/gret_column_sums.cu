// Sums over the groups of partial results, in a fixed order: the last step of
// the parameter gradients, so that they do not depend on the order in which
// blocks end.
#include "gret_block.cuh"

namespace gret {
namespace {

constexpr int kCols = 32, kLanes = 8;

// partial [groups][cols]; output j takes the columns offset[j] .. offset[j + 1] - 1
__global__ void __launch_bounds__(kCols* kLanes) column_sums_kernel(const float* partial, int groups, long long cols,
                                                                    ColumnOutputs out) {
    __shared__ float red[kLanes][kCols];
    const long long c = (long long)blockIdx.x * kCols + threadIdx.x;
    float s = 0.f;
    if (c < cols) {
#pragma unroll 4
        for (int g = threadIdx.y; g < groups; g += kLanes) s += partial[g * cols + c];
    }
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y != 0 || c >= cols) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kLanes; ++i) s += red[i][threadIdx.x];
    int j = 0;
    while (j + 1 < out.count && c >= out.offset[j + 1]) ++j;
    if (out.dst[j]) out.dst[j][(c - out.offset[j]) * out.stride[j]] = s;
}

}  // namespace

cudaError_t launch_column_sums(const float* partial, int groups, const ColumnOutputs& out, cudaStream_t s) {
    const long long cols = out.offset[out.count];
    column_sums_kernel<<<(unsigned)((cols + kCols - 1) / kCols), dim3(kCols, kLanes), 0, s>>>(partial, groups, cols, out);
    return cudaGetLastError();
}

}  // namespace gret
