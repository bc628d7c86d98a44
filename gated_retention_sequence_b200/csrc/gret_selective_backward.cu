// Gradients of the selective scan.  With g[t,d,i] the gradient of the state,
//
//   y = C.h + skip u,  dz = do y swish'(z),  dy = do swish(z)
//   g[t] = C[t] dy[t] + a[t+1] g[t+1],  a[t] = exp(delta[t] A),  g past the end = dh_final
//   dC[t,i] = sum_d h dy,  dB[t,i] = sum_d g delta u,  s = sum_i g B
//   du = skip dy + delta s,  ddelta = sum_i A g a h[t-1] + u s,  ddt = ddelta sigmoid(dt + dt_bias)
//   dA = sum_t delta g a h[t-1],  dskip = sum_t dy u,  ddt_bias = sum_t ddt,  dh0 = a[0] g[0]
//
// One pass forward leaves the state before every segment of kSeg tokens; one
// pass backward forms a segment's states again and walks it in reverse.
#include "gret_block.cuh"

namespace gret {
namespace {

constexpr int kSeg = 16;
constexpr int kThreads = 32;

__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

template <typename T, int NS>
__global__ void __launch_bounds__(kThreads) states_kernel(const ScanArgs a, float* states) {
    const int d = blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y, N = a.rows.N, segs = (N + kSeg - 1) / kSeg;
    if (d >= a.D) return;
    float h[NS], A[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        A[i] = a.A[(size_t)d * NS + i];
        h[i] = a.h0 ? a.h0[((size_t)b * a.D + d) * NS + i] : 0.f;
    }
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    for (int t = 0; t < N; ++t) {
        if (t % kSeg == 0) {
            float* to = states + (((size_t)b * segs + t / kSeg) * a.D + d) * NS;
#pragma unroll
            for (int i = 0; i < NS; ++i) to[i] = h[i];
        }
        const long long row = (long long)b * N + t;
        const float delta = softplus(to_f32(static_cast<const T*>(a.dt)[row * a.lddt + d]) + bias);
        const float du = delta * to_f32(static_cast<const T*>(a.u)[row * a.ldu + d]);
        const T* B = static_cast<const T*>(a.Bm) + row * a.ldb;
#pragma unroll
        for (int i = 0; i < NS; ++i) h[i] = fmaf(expf(delta * A[i]), h[i], du * to_f32(B[i]));
    }
}

// One warp: 32 channels of one sequence, its segments from the last to the
// first.  bc [D / 32][rows][2 NS]: this warp's share of dB and dC.
template <typename T, int NS>
__global__ void __launch_bounds__(kThreads) selective_backward_kernel(const ScanBackwardArgs g, const float* states,
                                                                      float* bc, float* partial) {
    const ScanArgs& a = g.f;
    const int lane = threadIdx.x, D = a.D, b = blockIdx.y, N = a.rows.N, segs = (N + kSeg - 1) / kSeg;
    const bool on = blockIdx.x * kThreads + lane < (unsigned)D;
    const int d = on ? blockIdx.x * kThreads + lane : D - 1;
    const long long rows = (long long)a.rows.B * N;
    float A[NS], dA[NS], gh[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        A[i] = a.A[(size_t)d * NS + i];
        dA[i] = 0.f;
        gh[i] = g.dh_final ? g.dh_final[((size_t)b * D + d) * NS + i] : 0.f;
    }
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f, skip = a.skip ? a.skip[d] : 0.f;
    float dskip = 0.f, dbias = 0.f;
    for (int s = segs - 1; s >= 0; --s) {
        const int len = min(kSeg, N - s * kSeg);
        float hs[kSeg + 1][NS];
        const float* from = states + (((size_t)b * segs + s) * D + d) * NS;
#pragma unroll
        for (int i = 0; i < NS; ++i) hs[0][i] = from[i];
        for (int t = 0; t < len; ++t) {
            const long long row = (long long)b * N + s * kSeg + t;
            const float delta = softplus(to_f32(static_cast<const T*>(a.dt)[row * a.lddt + d]) + bias);
            const float du = delta * to_f32(static_cast<const T*>(a.u)[row * a.ldu + d]);
            const T* B = static_cast<const T*>(a.Bm) + row * a.ldb;
#pragma unroll
            for (int i = 0; i < NS; ++i) hs[t + 1][i] = fmaf(expf(delta * A[i]), hs[t][i], du * to_f32(B[i]));
        }
        for (int t = len - 1; t >= 0; --t) {
            const long long row = (long long)b * N + s * kSeg + t;
            const T* B = static_cast<const T*>(a.Bm) + row * a.ldb;
            const T* C = static_cast<const T*>(a.Cm) + row * a.ldc;
            const float raw = to_f32(static_cast<const T*>(a.dt)[row * a.lddt + d]) + bias;
            const float delta = softplus(raw), u = to_f32(static_cast<const T*>(a.u)[row * a.ldu + d]);
            const float up = on ? to_f32(static_cast<const T*>(g.dout)[row * D + d]) : 0.f;
            float dy = up;
            if (a.z) {
                const float z = to_f32(static_cast<const T*>(a.z)[row * a.ldz + d]), sig = sigmoidf_(z);
                float y = skip * u;
#pragma unroll
                for (int i = 0; i < NS; ++i) y = fmaf(to_f32(C[i]), hs[t + 1][i], y);
                dy = up * z * sig;
                if (on) static_cast<T*>(g.dz)[row * D + d] = from_f32<T>(up * y * swish_slope(z, sig));
            }
            float sB = 0.f, sA = 0.f;
            float* to = bc + ((size_t)blockIdx.x * rows + row) * 2 * NS;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const float Bi = to_f32(B[i]);
                gh[i] = fmaf(to_f32(C[i]), dy, gh[i]);
                const float dB = warp_sum(on ? gh[i] * delta * u : 0.f), dC = warp_sum(hs[t + 1][i] * dy);
                if (lane == 0) {
                    to[i] = dB;
                    to[NS + i] = dC;
                }
                sB = fmaf(gh[i], Bi, sB);
                gh[i] *= expf(delta * A[i]);
                const float through = gh[i] * hs[t][i];
                sA = fmaf(through, A[i], sA);
                dA[i] = fmaf(through, delta, dA[i]);
            }
            const float ddt = fmaf(u, sB, sA) * sigmoidf_(raw);
            dskip = fmaf(dy, u, dskip);
            dbias += ddt;
            if (on) {
                static_cast<T*>(g.du)[row * D + d] = from_f32<T>(fmaf(delta, sB, skip * dy));
                static_cast<T*>(g.ddt)[row * D + d] = from_f32<T>(ddt);
            }
        }
    }
    if (!on) return;
    float* to = partial + (size_t)b * D * (NS + 2);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        to[(size_t)d * NS + i] = dA[i];
        if (g.dh0) g.dh0[((size_t)b * D + d) * NS + i] = gh[i];
    }
    to[(size_t)D * NS + d] = dskip;
    to[(size_t)D * (NS + 1) + d] = dbias;
}

// dB, dC: the channel blocks' shares, added in order.
template <typename T>
__global__ void __launch_bounds__(256) join_kernel(const float* bc, int blocks, long long rows, int n, T* dB, T* dC) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= rows * 2 * n) return;
    float s = 0.f;
    for (int k = 0; k < blocks; ++k) s += bc[(size_t)k * rows * 2 * n + i];
    const long long row = i / (2 * n);
    const int j = (int)(i - row * 2 * n);
    (j < n ? dB[row * n + j] : dC[row * n + j - n]) = from_f32<T>(s);
}

struct Sizes {
    size_t states, bc, partial;
};
Sizes sizes(int B, int N, int D, int n) {
    const size_t segs = (N + kSeg - 1) / kSeg, blocks = (D + kThreads - 1) / kThreads;
    return {align256((size_t)B * segs * D * n * 4), align256(blocks * B * N * 2 * n * 4),
            align256((size_t)B * D * (n + 2) * 4)};
}

template <typename T, int NS>
cudaError_t backward(const ScanBackwardArgs& g, cudaStream_t s) {
    const ScanArgs& a = g.f;
    const Sizes z = sizes(a.rows.B, a.rows.N, a.D, NS);
    char* ws = static_cast<char*>(g.workspace);
    float* states = reinterpret_cast<float*>(ws);
    float* bc = reinterpret_cast<float*>(ws + z.states);
    float* partial = reinterpret_cast<float*>(ws + z.states + z.bc);
    const dim3 grid((a.D + kThreads - 1) / kThreads, a.rows.B);
    states_kernel<T, NS><<<grid, kThreads, 0, s>>>(a, states);
    selective_backward_kernel<T, NS><<<grid, kThreads, 0, s>>>(g, states, bc, partial);
    const long long rows = (long long)a.rows.B * a.rows.N;
    join_kernel<T><<<(unsigned)((rows * 2 * NS + 255) / 256), 256, 0, s>>>(bc, grid.x, rows, NS, static_cast<T*>(g.dBm),
                                                                          static_cast<T*>(g.dCm));
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const long long D = a.D;
    const ColumnOutputs out = {3, {0, D * NS, D * (NS + 1), D * (NS + 2)}, {g.dA, g.dskip, g.ddt_bias}, {1, 1, 1}};
    return launch_column_sums(partial, a.rows.B, out, s);
}

}  // namespace

size_t selective_backward_ws_bytes(int B, int N, int D, int n, gret_dtype) {
    const Sizes z = sizes(B, N, D, n);
    return z.states + z.bc + z.partial;
}

cudaError_t launch_selective_backward(ScanBackwardArgs g, int num_sms, cudaStream_t s) {
    (void)num_sms;
    const bool bf = g.f.io == GRET_BF16;
    switch (g.f.n) {
        case 8: return bf ? backward<__nv_bfloat16, 8>(g, s) : backward<float, 8>(g, s);
        case 16: return bf ? backward<__nv_bfloat16, 16>(g, s) : backward<float, 16>(g, s);
        case 32: return bf ? backward<__nv_bfloat16, 32>(g, s) : backward<float, 32>(g, s);
        default: return bf ? backward<__nv_bfloat16, 64>(g, s) : backward<float, 64>(g, s);
    }
}

}  // namespace gret
