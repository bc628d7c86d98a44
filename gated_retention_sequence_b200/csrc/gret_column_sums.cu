// Sums over the groups of partial results: the last step of the parameter
// gradients.
#include "gret_block.cuh"

namespace gret {
namespace {

__global__ void __launch_bounds__(kSumThreads) column_sums_kernel(const float* partial, int groups, ColumnOutputs out) {
    column_sums(partial, groups, out, blockIdx.x);
}

}  // namespace

cudaError_t launch_column_sums(const float* partial, int groups, const ColumnOutputs& out, cudaStream_t s) {
    column_sums_kernel<<<(unsigned)column_blocks(out), kSumThreads, 0, s>>>(partial, groups, out);
    return cudaGetLastError();
}

}  // namespace gret
