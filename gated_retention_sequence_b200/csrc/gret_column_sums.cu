// Sums over the groups of partial results: the last step of the parameter
// gradients.
#include "gret_block.cuh"

namespace gret {
namespace {

__global__ void __launch_bounds__(kSumThreads) column_sums_kernel(const float* partial, int groups, ColumnOutputs out,
                                                                 int width) {
    column_sums(partial, groups, out, width, blockIdx.x);
}

}  // namespace

cudaError_t launch_column_sums(const float* partial, int groups, const ColumnOutputs& out, cudaStream_t s) {
    const int width = column_width(out, groups);
    column_sums_kernel<<<(unsigned)column_blocks(out, width), kSumThreads, 0, s>>>(partial, groups, out, width);
    return cudaGetLastError();
}

}  // namespace gret
