// Selective state space scan: a state of n numbers per channel whose decay and
// input depend on the token.
//
//   delta[t,d] = softplus(dt[t,d] + dt_bias[d])
//   h[t,d,i]   = exp(delta[t,d] A[d,i]) h[t-1,d,i] + delta[t,d] u[t,d] B[t,i]
//   o[t,d]     = (sum_i C[t,i] h[t,d,i] + skip[d] u[t,d]) swish(z[t,d])
//
// B and C are shared by all channels of a token.
#include "gret_block.cuh"

namespace gret {
namespace {

constexpr int kStepThreads = 128;

__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

// A thread owns one channel of one sequence and walks its tokens.
template <typename T, int NS>
__global__ void __launch_bounds__(64) selective_scan_kernel(const ScanArgs a) {
    const Slot f = find_slot(a.rows, blockIdx.x);
    const int d = blockIdx.y * 64 + threadIdx.x;
    if (f.b < 0 || d >= a.D) return;
    float h[NS], A[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        A[i] = a.A[(size_t)d * NS + i];
        h[i] = a.h0 ? a.h0[((size_t)f.b * a.D + d) * NS + i] : 0.f;
    }
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f, skip = a.skip ? a.skip[d] : 0.f;
    for (int t = 0; t < f.len; ++t) {
        const long long row = f.row0 + t;
        const float u = to_f32(static_cast<const T*>(a.u)[row * a.ldu + d]);
        const float delta = softplus(to_f32(static_cast<const T*>(a.dt)[row * a.lddt + d]) + bias);
        const T* B = static_cast<const T*>(a.Bm) + row * a.ldb;
        const T* C = static_cast<const T*>(a.Cm) + row * a.ldc;
        const float du = delta * u;
        float y = skip * u;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            h[i] = fmaf(expf(delta * A[i]), h[i], du * to_f32(B[i]));
            y = fmaf(to_f32(C[i]), h[i], y);
        }
        if (a.z) {
            const float z = to_f32(static_cast<const T*>(a.z)[row * a.ldz + d]);
            y *= z * sigmoidf_(z);
        }
        static_cast<T*>(a.o)[row * a.D + d] = from_f32<T>(y);
    }
    if (a.h) {
#pragma unroll
        for (int i = 0; i < NS; ++i) a.h[((size_t)f.b * a.D + d) * NS + i] = h[i];
    }
}

// One token per sequence: the states are read and written once, 16 bytes at a
// time, n / 4 lanes to a channel.  h may be h0.
template <typename T, int NS>
__global__ void __launch_bounds__(kStepThreads) selective_step_kernel(const ScanArgs a) {
    constexpr int L = NS / 4;
    const long long i = (long long)blockIdx.x * kStepThreads + threadIdx.x;
    const bool on = i < (long long)a.rows.B * a.D * L;
    const long long unit = on ? i / L : 0;
    const int b = (int)(unit / a.D), d = (int)(unit - (long long)b * a.D), q = (int)(i % L) * 4;
    const float4 A = *reinterpret_cast<const float4*>(a.A + (size_t)d * NS + q);
    float4 h = on ? *reinterpret_cast<const float4*>(a.h0 + unit * NS + q) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float u = to_f32(static_cast<const T*>(a.u)[b * a.ldu + d]);
    const float delta = softplus(to_f32(static_cast<const T*>(a.dt)[b * a.lddt + d]) + (a.dt_bias ? a.dt_bias[d] : 0.f));
    const T* B = static_cast<const T*>(a.Bm) + b * a.ldb + q;
    const T* C = static_cast<const T*>(a.Cm) + b * a.ldc + q;
    const float du = delta * u;
    h.x = fmaf(expf(delta * A.x), h.x, du * to_f32(B[0]));
    h.y = fmaf(expf(delta * A.y), h.y, du * to_f32(B[1]));
    h.z = fmaf(expf(delta * A.z), h.z, du * to_f32(B[2]));
    h.w = fmaf(expf(delta * A.w), h.w, du * to_f32(B[3]));
    float y = to_f32(C[0]) * h.x + to_f32(C[1]) * h.y + to_f32(C[2]) * h.z + to_f32(C[3]) * h.w;
#pragma unroll
    for (int m = L / 2; m > 0; m >>= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
    if (!on) return;
    *reinterpret_cast<float4*>(a.h + unit * NS + q) = h;
    if (q == 0) {
        if (a.skip) y = fmaf(a.skip[d], u, y);
        if (a.z) {
            const float z = to_f32(static_cast<const T*>(a.z)[b * a.ldz + d]);
            y *= z * sigmoidf_(z);
        }
        static_cast<T*>(a.o)[unit] = from_f32<T>(y);
    }
}

template <typename T, int NS>
cudaError_t scan(ScanArgs a, cudaStream_t s) {
    a.rows.seg = a.rows.N;
    const dim3 grid((unsigned)slots_of(a.rows), (a.D + 63) / 64);
    selective_scan_kernel<T, NS><<<grid, 64, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int NS>
cudaError_t step(const ScanArgs& a, cudaStream_t s) {
    const long long threads = (long long)a.rows.B * a.D * (NS / 4);
    selective_step_kernel<T, NS><<<(unsigned)((threads + kStepThreads - 1) / kStepThreads), kStepThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

bool selective_states_supported(int n) { return n == 8 || n == 16 || n == 32 || n == 64; }

size_t selective_scan_ws_bytes(int, int, int, int, int, bool, int) { return 0; }

cudaError_t launch_selective_scan(ScanArgs a, int num_sms, cudaStream_t s) {
    (void)num_sms;
    const bool bf = a.io == GRET_BF16;
    switch (a.n) {
        case 8: return bf ? scan<__nv_bfloat16, 8>(a, s) : scan<float, 8>(a, s);
        case 16: return bf ? scan<__nv_bfloat16, 16>(a, s) : scan<float, 16>(a, s);
        case 32: return bf ? scan<__nv_bfloat16, 32>(a, s) : scan<float, 32>(a, s);
        default: return bf ? scan<__nv_bfloat16, 64>(a, s) : scan<float, 64>(a, s);
    }
}

cudaError_t launch_selective_step(const ScanArgs& a, int num_sms, cudaStream_t s) {
    (void)num_sms;
    const bool bf = a.io == GRET_BF16;
    switch (a.n) {
        case 8: return bf ? step<__nv_bfloat16, 8>(a, s) : step<float, 8>(a, s);
        case 16: return bf ? step<__nv_bfloat16, 16>(a, s) : step<float, 16>(a, s);
        case 32: return bf ? step<__nv_bfloat16, 32>(a, s) : step<float, 32>(a, s);
        default: return bf ? step<__nv_bfloat16, 64>(a, s) : step<float, 64>(a, s);
    }
}

}  // namespace gret
