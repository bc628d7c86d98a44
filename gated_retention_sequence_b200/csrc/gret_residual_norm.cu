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

// Gradients, with everything of the forward formed again from x, y and gate
// (kv = 1 / rms(v), vn = v kv, q = yn w_post, t = dn w_next):
//   dx = dr + kr (t - rn mean(t rn)),  dscale = sum dx q swish(gate),  dw_next = sum dn rn
//   dp = dx scale,  dgate = dp q swish'(gate),  dq = dp swish(gate),  dw_post = sum dq yn
//   dy = ky (dq w_post - yn mean(dq w_post yn))
// A block walks rows blockIdx.x, + gridDim.x, ... and keeps its share of the
// three parameter gradients in registers.
template <typename TS, typename T, int V>
__global__ void __launch_bounds__(512) residual_norm_backward_kernel(const NormBackwardArgs g, float* partial) {
    __shared__ float red[4][32];
    const NormArgs& a = g.f;
    const int warps = blockDim.x >> 5;
    float acc[3][V][kVec] = {};
    for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
        float x[V][kVec] = {}, y[V][kVec] = {}, gt[V][kVec] = {}, dn[V][kVec] = {}, dr[V][kVec] = {};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (threadIdx.x + j * blockDim.x) * kVec;
            if (c >= a.D) continue;
            load8(static_cast<const TS*>(a.x) + t * a.ldx + c, x[j]);
            if (a.y) load8(static_cast<const T*>(a.y) + t * a.ldy + c, y[j]);
            if (a.gate) load8(static_cast<const T*>(a.gate) + t * a.ldg + c, gt[j]);
            if (a.w_next) load8(static_cast<const T*>(g.dn) + t * a.D + c, dn[j]);
            if (g.dr) load8(static_cast<const TS*>(g.dr) + t * a.D + c, dr[j]);
        }
        float ky = 1.f;
        if (a.w_post) {
            float sq = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int e = 0; e < kVec; ++e) sq = fmaf(y[j][e], y[j][e], sq);
            ky = rsqrtf(block_sum(sq, red[0], warps) / (float)a.D + a.eps);
        }
        if (a.y) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (threadIdx.x + j * blockDim.x) * kVec;
                if (c >= a.D) continue;
                float wp[kVec], sc[kVec];
                if (a.w_post) load8(a.w_post + c, wp);
                if (a.scale) load8(a.scale + c, sc);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    float p = y[j][e] * ky;
                    if (a.w_post) p *= wp[e];
                    if (a.gate) p *= gt[j][e] * sigmoidf_(gt[j][e]);
                    if (a.scale) p *= sc[e];
                    x[j][e] += p;                               // r
                }
            }
        }
        if (a.w_next) {
            float s2 = 0.f, s3 = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (threadIdx.x + j * blockDim.x) * kVec;
                if (c >= a.D) continue;
                float wn[kVec];
                load8(a.w_next + c, wn);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    s2 = fmaf(x[j][e], x[j][e], s2);
                    s3 = fmaf(dn[j][e] * wn[e], x[j][e], s3);
                }
            }
            s2 = block_sum(s2, red[1], warps);
            s3 = block_sum(s3, red[2], warps);
            const float kr = rsqrtf(s2 / (float)a.D + a.eps), m = s3 * kr / (float)a.D;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (threadIdx.x + j * blockDim.x) * kVec;
                if (c >= a.D) continue;
                float wn[kVec];
                load8(a.w_next + c, wn);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const float rn = x[j][e] * kr;
                    acc[2][j][e] = fmaf(dn[j][e], rn, acc[2][j][e]);
                    dr[j][e] += kr * (dn[j][e] * wn[e] - rn * m);
                }
            }
        }
        float s4 = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (threadIdx.x + j * blockDim.x) * kVec;
            if (c >= a.D) continue;
            store8(static_cast<TS*>(g.dx) + t * a.D + c, dr[j]);
            if (!a.y) continue;
            float wp[kVec], sc[kVec], dg[kVec];
            if (a.w_post) load8(a.w_post + c, wp);
            if (a.scale) load8(a.scale + c, sc);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float yn = y[j][e] * ky, q = a.w_post ? yn * wp[e] : yn;
                const float sig = a.gate ? sigmoidf_(gt[j][e]) : 1.f, sw = a.gate ? gt[j][e] * sig : 1.f;
                const float dp = a.scale ? dr[j][e] * sc[e] : dr[j][e];
                const float dq = dp * sw;
                acc[0][j][e] = fmaf(dr[j][e], q * sw, acc[0][j][e]);
                acc[1][j][e] = fmaf(dq, yn, acc[1][j][e]);
                dg[e] = dp * q * swish_slope(gt[j][e], sig);
                const float up = a.w_post ? dq * wp[e] : dq;
                s4 = fmaf(up, yn, s4);
                y[j][e] = yn;
                dr[j][e] = up;
            }
            if (a.gate) store8(static_cast<T*>(g.dgate) + t * a.D + c, dg);
        }
        if (a.y) {
            const float m = a.w_post ? block_sum(s4, red[3], warps) / (float)a.D : 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (threadIdx.x + j * blockDim.x) * kVec;
                if (c >= a.D) continue;
#pragma unroll
                for (int e = 0; e < kVec; ++e) dr[j][e] = ky * (dr[j][e] - y[j][e] * m);
                store8(static_cast<T*>(g.dy) + t * a.D + c, dr[j]);
            }
        }
        __syncthreads();                                        // the sums' shared words are used again
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (threadIdx.x + j * blockDim.x) * kVec;
            if (c < a.D) store8(partial + ((size_t)blockIdx.x * 3 + i) * a.D + c, acc[i][j]);
        }
}

template <typename TS, typename T>
cudaError_t norm_backward(const NormBackwardArgs& g, int grid, cudaStream_t s) {
    const int vecs = g.f.D / kVec, V = vecs <= 512 ? 1 : 2;
    const int threads = ((vecs + V - 1) / V + 31) & ~31;
    float* partial = static_cast<float*>(g.workspace);
    if (V == 1)
        residual_norm_backward_kernel<TS, T, 1><<<grid, threads, 0, s>>>(g, partial);
    else
        residual_norm_backward_kernel<TS, T, 2><<<grid, threads, 0, s>>>(g, partial);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || (!g.dscale && !g.dw_post && !g.dw_next)) return err;
    const long long D = g.f.D;
    const ColumnOutputs out = {3, {0, D, 2 * D, 3 * D}, {g.dscale, g.dw_post, g.dw_next}, {1, 1, 1}};
    return launch_column_sums(partial, grid, out, s);
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

static int backward_grid(long long T, int num_sms) {
    const long long most = 2LL * num_sms;
    return (int)(T < most ? T : most);
}

size_t residual_norm_backward_ws_bytes(long long T, int D, int num_sms) {
    return align256((size_t)backward_grid(T, num_sms) * 3 * D * sizeof(float));
}

cudaError_t launch_residual_norm_backward(NormBackwardArgs g, int num_sms, cudaStream_t s) {
    const int grid = backward_grid(g.f.T, num_sms);
    if (g.f.io == GRET_F32) return norm_backward<float, float>(g, grid, s);
    if (g.f.stream_type == GRET_F32) return norm_backward<float, __nv_bfloat16>(g, grid, s);
    return norm_backward<__nv_bfloat16, __nv_bfloat16>(g, grid, s);
}

}  // namespace gret
