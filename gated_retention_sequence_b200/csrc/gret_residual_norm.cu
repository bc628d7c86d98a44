// The norm after a block, its gate and residual scale, and the norm before the
// next block, in one pass over the rows:
//
//   p = rms(y) (.) w_post (.) swish(gate),  r = x + scale (.) p,  n = rms(r) (.) w_next
//   rms(v) = v / sqrt(mean(v^2) + eps)
//
// A block of threads holds one row in registers: every input is read once and
// every output written once, and both sums are taken from the registers in
// fp32.  n is formed from r before r is rounded to its storage type.
#include "gret_block.cuh"

namespace gret {
namespace {

__device__ __forceinline__ float block_sum(float v, float* red, int warps) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < warps; ++w) s += red[w];
    return s;
}

// TS: the residual stream's type; T: the block's.  Thread i holds the vectors
// i, i + blockDim.x, ... of the row.
template <typename TS, typename T, int V>
__global__ void residual_norm_kernel(const NormArgs a) {
    __shared__ float red[2][32];
    const int warps = blockDim.x >> 5;
    const long long t = blockIdx.x;
    const TS* x = static_cast<const TS*>(a.x) + t * a.ldx;
    const T* y = static_cast<const T*>(a.y) + (a.y ? t * a.ldy : 0);
    const T* g = static_cast<const T*>(a.gate) + (a.gate ? t * a.ldg : 0);
    float r[V][kVec], p[V][kVec];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = (threadIdx.x + j * blockDim.x) * kVec;
#pragma unroll
        for (int e = 0; e < kVec; ++e) r[j][e] = p[j][e] = 0.f;
        if (c < a.D) {
            load8(x + c, r[j]);
            if (a.y) load8(y + c, p[j]);
        }
    }
    if (a.y) {
        float k = 1.f;
        if (a.w_post) {
            float sq = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int e = 0; e < kVec; ++e) sq = fmaf(p[j][e], p[j][e], sq);
            k = rsqrtf(block_sum(sq, red[0], warps) / (float)a.D + a.eps);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (threadIdx.x + j * blockDim.x) * kVec;
            if (c >= a.D) continue;
            float w[kVec];
            if (a.w_post) {
                load8(a.w_post + c, w);
#pragma unroll
                for (int e = 0; e < kVec; ++e) p[j][e] *= k * w[e];
            }
            if (a.gate) {
                load8(g + c, w);
#pragma unroll
                for (int e = 0; e < kVec; ++e) p[j][e] *= w[e] * sigmoidf_(w[e]);
            }
            if (a.scale) {
                load8(a.scale + c, w);
#pragma unroll
                for (int e = 0; e < kVec; ++e) p[j][e] *= w[e];
            }
#pragma unroll
            for (int e = 0; e < kVec; ++e) r[j][e] += p[j][e];
            store8(static_cast<TS*>(a.r) + t * a.D + c, r[j]);
        }
    }
    if (!a.w_next) return;
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < kVec; ++e) sq = fmaf(r[j][e], r[j][e], sq);
    const float k = rsqrtf(block_sum(sq, red[1], warps) / (float)a.D + a.eps);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = (threadIdx.x + j * blockDim.x) * kVec;
        if (c >= a.D) continue;
        float w[kVec];
        load8(a.w_next + c, w);
#pragma unroll
        for (int e = 0; e < kVec; ++e) w[e] *= r[j][e] * k;
        store8(static_cast<T*>(a.n) + t * a.D + c, w);
    }
}

template <typename TS, typename T>
cudaError_t norm(const NormArgs& a, cudaStream_t s) {
    const int vecs = a.D / kVec;
    const int V = vecs <= 256 ? 1 : 2;
    const int threads = ((vecs + V - 1) / V + 31) & ~31;
    if (V == 1)
        residual_norm_kernel<TS, T, 1><<<(unsigned)a.T, threads, 0, s>>>(a);
    else
        residual_norm_kernel<TS, T, 2><<<(unsigned)a.T, threads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_residual_norm(const NormArgs& a, int num_sms, cudaStream_t s) {
    (void)num_sms;
    if (a.io == GRET_F32) return norm<float, float>(a, s);
    if (a.stream_type == GRET_F32) return norm<float, __nv_bfloat16>(a, s);
    return norm<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace gret
