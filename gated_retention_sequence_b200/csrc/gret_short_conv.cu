// Short causal convolution along the tokens, one filter of K taps per channel.
//
//   s[t,d] = bias[d] + sum_k w[d,k] x[t-K+1+k,d],   y = act(s)
//
// Rows from before a sequence's first token come from its tail (the last K-1
// inputs of the piece before, or zero).  A thread owns eight channels of one
// slot (a segment of tokens) and keeps the last K-1 inputs in registers, so
// that each input is read once, 16 bytes at a time, and K-1 more rows per slot.
#include "gret_block.cuh"

namespace gret {
namespace {

constexpr int kThreads = 128;
constexpr int kSeg = 32;

template <typename T, int K>
struct Taps {
    float w[K][kVec], b[kVec];
    __device__ __forceinline__ void load(const float* wp, const float* bp, int c) {
        float flat[K * kVec];
#pragma unroll
        for (int i = 0; i < K * kVec / 4; ++i) {
            const float4 q = reinterpret_cast<const float4*>(wp + (size_t)c * K)[i];
            flat[4 * i] = q.x; flat[4 * i + 1] = q.y; flat[4 * i + 2] = q.z; flat[4 * i + 3] = q.w;
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e)
#pragma unroll
            for (int k = 0; k < K; ++k) w[k][e] = flat[e * K + k];
        if (bp) {
            load8(bp + c, b);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) b[e] = 0.f;
        }
    }
};

// Row t (within its sequence) of the inputs; t in [-(K-1), seq_len).
template <typename T, int K>
__device__ __forceinline__ void input_row(const ConvArgs& a, const Slot& f, int t, int c, float* v) {
    if (t >= 0) {
        load8(static_cast<const T*>(a.x) + (f.row0 + t) * a.ldx + c, v);
    } else if (a.tail0) {
        load8(static_cast<const T*>(a.tail0) + ((size_t)f.b * (K - 1) + (K - 1 + t)) * a.D + c, v);
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] = 0.f;
    }
}

template <typename T, int K>
__global__ void __launch_bounds__(kThreads) short_conv_kernel(const ConvArgs a) {
    const Slot f = find_slot(a.rows, blockIdx.x);
    const int c = (blockIdx.y * kThreads + threadIdx.x) * kVec;
    if (f.b < 0 || c >= a.D) return;
    Taps<T, K> taps;
    taps.load(a.w, a.bias, c);
    float past[K - 1][kVec];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) input_row<T, K>(a, f, f.first - (K - 1) + j, c, past[j]);
    const T* x = static_cast<const T*>(a.x) + (f.row0 + f.first) * a.ldx + c;
    T* y = static_cast<T*>(a.y) + (f.row0 + f.first) * (long long)a.D + c;
#pragma unroll 4
    for (int t = 0; t < f.len; ++t) {
        float now[kVec], out[kVec];
        load8(x + t * a.ldx, now);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            float s = taps.b[e];
#pragma unroll
            for (int k = 0; k < K - 1; ++k) s = fmaf(taps.w[k][e], past[k][e], s);
            s = fmaf(taps.w[K - 1][e], now[e], s);
            out[e] = a.swish ? s * sigmoidf_(s) : s;
#pragma unroll
            for (int k = 0; k + 1 < K - 1; ++k) past[k][e] = past[k + 1][e];
            past[K - 2][e] = now[e];
        }
        store8(y + (size_t)t * a.D, out);
    }
    if (a.tail && f.s == max(f.segs, 1) - 1) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            store8(static_cast<T*>(a.tail) + ((size_t)f.b * (K - 1) + j) * a.D + c, past[j]);
    }
}

// One token per sequence.  tail may be tail0: a thread reads what it owns
// before it writes.
template <typename T, int K>
__global__ void __launch_bounds__(kThreads) short_conv_step_kernel(const ConvArgs a) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int groups = a.D / kVec;
    if (i >= (long long)a.rows.B * groups) return;
    const int b = (int)(i / groups), c = (int)(i - (long long)b * groups) * kVec;
    Taps<T, K> taps;
    taps.load(a.w, a.bias, c);
    const T* old = static_cast<const T*>(a.tail0) + (size_t)b * (K - 1) * a.D + c;
    T* next = static_cast<T*>(a.tail) + (size_t)b * (K - 1) * a.D + c;
    float v[K][kVec], out[kVec];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) load8(old + (size_t)j * a.D, v[j]);
    load8(static_cast<const T*>(a.x) + b * a.ldx + c, v[K - 1]);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        float s = taps.b[e];
#pragma unroll
        for (int k = 0; k < K; ++k) s = fmaf(taps.w[k][e], v[k][e], s);
        out[e] = a.swish ? s * sigmoidf_(s) : s;
    }
    store8(static_cast<T*>(a.y) + (size_t)b * a.D + c, out);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store8(next + (size_t)j * a.D, v[j + 1]);
}

// Gradients.  With ds[t] = dy[t] act'(s[t]) (s formed again from the inputs):
//   dx[t]   = sum_j w[K-1-j] ds[t+j]      (rows before the first token: dtail0)
//   dw[k]   = sum_t ds[t] x[t-K+1+k],  dbias = sum_t ds[t]
// and dtail adds to the last K-1 rows.  A thread walks one slot and K-1 tokens
// past its end; the slots of a block add up their dw and dbias in shared memory.
constexpr int kBackGroups = 16, kBackSlots = 8, kBackSeg = 64;

template <typename T, int K>
__global__ void __launch_bounds__(kBackGroups* kBackSlots) short_conv_backward_kernel(const ConvBackwardArgs g,
                                                                                     float* partial, int slots) {
    __shared__ float red[kBackSlots][kBackGroups * kVec + 1];
    const ConvArgs& a = g.f;
    const int slot = blockIdx.x * kBackSlots + threadIdx.y;
    const int c = (blockIdx.y * kBackGroups + threadIdx.x) * kVec;
    const bool on = slot < slots && c < a.D;
    float dw[K + 1][kVec] = {};
    if (on) {
        const Slot f = find_slot(a.rows, slot);
        Taps<T, K> taps;
        taps.load(a.w, a.bias, c);
        float past[K - 1][kVec], ds[K][kVec] = {};
#pragma unroll
        for (int j = 0; j < K - 1; ++j) input_row<T, K>(a, f, f.first - (K - 1) + j, c, past[j]);
        const T* x = static_cast<const T*>(a.x) + f.row0 * a.ldx + c;
        const T* dy = static_cast<const T*>(g.dy) + f.row0 * a.D + c;
        T* dx = static_cast<T*>(g.dx) + f.row0 * a.D + c;
        const int end = f.first + f.len, tail_at = f.seq_len - (K - 1);
        const int lo = f.first == 0 ? (g.dtail0 ? -(K - 1) : 0) : f.first;
        for (int t = f.first; t < end + K - 1; ++t) {
#pragma unroll
            for (int k = 0; k + 1 < K; ++k)
#pragma unroll
                for (int e = 0; e < kVec; ++e) ds[k][e] = ds[k + 1][e];
            if (t < f.seq_len) {
                float now[kVec], up[kVec];
                load8(x + t * a.ldx, now);
                load8(dy + (size_t)t * a.D, up);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    float s = taps.b[e];
#pragma unroll
                    for (int k = 0; k < K - 1; ++k) s = fmaf(taps.w[k][e], past[k][e], s);
                    s = fmaf(taps.w[K - 1][e], now[e], s);
                    const float d = a.swish ? up[e] * swish_slope(s, sigmoidf_(s)) : up[e];
                    ds[K - 1][e] = d;
                    if (t < end) {
#pragma unroll
                        for (int k = 0; k < K - 1; ++k) dw[k][e] = fmaf(d, past[k][e], dw[k][e]);
                        dw[K - 1][e] = fmaf(d, now[e], dw[K - 1][e]);
                        dw[K][e] += d;
                    }
#pragma unroll
                    for (int k = 0; k + 1 < K - 1; ++k) past[k][e] = past[k + 1][e];
                    past[K - 2][e] = now[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) ds[K - 1][e] = 0.f;
            }
            const int r = t - (K - 1);
            if (r < lo) continue;
            float out[kVec] = {};
            if (g.dtail && r >= tail_at)
                load8(static_cast<const T*>(g.dtail) + ((size_t)f.b * (K - 1) + (r - tail_at)) * a.D + c, out);
#pragma unroll
            for (int e = 0; e < kVec; ++e)
#pragma unroll
                for (int j = 0; j < K; ++j) out[e] = fmaf(taps.w[K - 1 - j][e], ds[j][e], out[e]);
            if (r >= 0)
                store8(dx + (size_t)r * a.D, out);
            else
                store8(static_cast<T*>(g.dtail0) + ((size_t)f.b * (K - 1) + (K - 1 + r)) * a.D + c, out);
        }
    }
    const int tid = threadIdx.y * kBackGroups + threadIdx.x;
    const int ch = blockIdx.y * kBackGroups * kVec + tid;
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kVec; ++e) red[threadIdx.y][threadIdx.x * kVec + e] = dw[k][e];
        __syncthreads();
        if (ch < a.D) {
            float s = 0.f;
#pragma unroll
            for (int y = 0; y < kBackSlots; ++y) s += red[y][tid];
            partial[((size_t)blockIdx.x * (K + 1) + k) * a.D + ch] = s;
        }
    }
}
static_assert(kBackGroups * kVec == kBackGroups * kBackSlots, "a thread of the block for each of its channels");

template <typename T, int K>
cudaError_t conv_backward(ConvBackwardArgs g, cudaStream_t s) {
    g.f.rows.seg = kBackSeg;
    const long long slots = slots_of(g.f.rows);
    const int D = g.f.D;
    const dim3 grid((unsigned)((slots + kBackSlots - 1) / kBackSlots), (D + kBackGroups * kVec - 1) / (kBackGroups * kVec));
    float* partial = static_cast<float*>(g.workspace);
    short_conv_backward_kernel<T, K><<<grid, dim3(kBackGroups, kBackSlots), 0, s>>>(g, partial, (int)slots);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || (!g.dw && !g.dbias)) return err;
    ColumnOutputs out = {};
    out.count = K + 1;
    for (int k = 0; k <= K; ++k) {
        out.offset[k] = (long long)k * D;
        out.dst[k] = k < K ? (g.dw ? g.dw + k : nullptr) : g.dbias;
        out.stride[k] = k < K ? K : 1;
    }
    out.offset[K + 1] = (long long)(K + 1) * D;
    return launch_column_sums(partial, (int)grid.x, out, s);
}

template <typename T, int K>
cudaError_t conv(const ConvArgs& a, cudaStream_t s) {
    const dim3 grid((unsigned)slots_of(a.rows), (a.D / kVec + kThreads - 1) / kThreads);
    short_conv_kernel<T, K><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int K>
cudaError_t conv_step(const ConvArgs& a, cudaStream_t s) {
    const long long threads = (long long)a.rows.B * (a.D / kVec);
    short_conv_step_kernel<T, K><<<(unsigned)((threads + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_short_conv(ConvArgs a, cudaStream_t s) {
    a.rows.seg = kSeg;
    if (a.io == GRET_BF16) {
        if (a.K == 2) return conv<__nv_bfloat16, 2>(a, s);
        return a.K == 3 ? conv<__nv_bfloat16, 3>(a, s) : conv<__nv_bfloat16, 4>(a, s);
    }
    if (a.K == 2) return conv<float, 2>(a, s);
    return a.K == 3 ? conv<float, 3>(a, s) : conv<float, 4>(a, s);
}

cudaError_t launch_short_conv_step(const ConvArgs& a, cudaStream_t s) {
    if (a.io == GRET_BF16) {
        if (a.K == 2) return conv_step<__nv_bfloat16, 2>(a, s);
        return a.K == 3 ? conv_step<__nv_bfloat16, 3>(a, s) : conv_step<__nv_bfloat16, 4>(a, s);
    }
    if (a.K == 2) return conv_step<float, 2>(a, s);
    return a.K == 3 ? conv_step<float, 3>(a, s) : conv_step<float, 4>(a, s);
}

size_t short_conv_backward_ws_bytes(int B, int N, int D, int K) {
    const long long slots = (long long)B * ((N + kBackSeg - 1) / kBackSeg);
    return align256((size_t)((slots + kBackSlots - 1) / kBackSlots) * (K + 1) * D * sizeof(float));
}

cudaError_t launch_short_conv_backward(ConvBackwardArgs g, cudaStream_t s) {
    const int K = g.f.K;
    if (g.f.io == GRET_BF16) {
        if (K == 2) return conv_backward<__nv_bfloat16, 2>(g, s);
        return K == 3 ? conv_backward<__nv_bfloat16, 3>(g, s) : conv_backward<__nv_bfloat16, 4>(g, s);
    }
    if (K == 2) return conv_backward<float, 2>(g, s);
    return K == 3 ? conv_backward<float, 3>(g, s) : conv_backward<float, 4>(g, s);
}

}  // namespace gret
