// Short causal convolution along the tokens, one filter of K taps per channel.
//
//   s[t,d] = bias[d] + sum_k w[d,k] x[t-K+1+k,d],   y = act(s)
//
// Rows from before a sequence's first token come from its tail (the last K-1
// inputs of the piece before, or zero).  A thread owns four channels of one
// slot (a segment of tokens) and keeps the last K-1 inputs in registers, so
// that each input is read once, and K-1 more rows per slot.  Rows are copied
// kBatch at a time into shared memory, a batch ahead; whole batches take a path
// without a condition per row.  Measured at 16384 packed tokens x 4096
// channels, bf16: 58 us (4.7 TB/s); 63 us with the rows held in registers
// instead, 73 us with none ahead, 104 us with eight channels a thread.
#include "gret_block.cuh"

namespace gret {
namespace {

constexpr int kThreads = 128;
constexpr int kSeg = 64, kBatch = 8, kAhead = 1, kC = 4, kP = kC / 2;

// Four channels as they lie in memory.
template <typename T> struct Four;
template <> struct Four<__nv_bfloat16> {
    uint2 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void zero() { a = make_uint2(0, 0); }
    __device__ __forceinline__ void get(float2* v) const {
        v[0] = make_float2(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u));
        v[1] = make_float2(__uint_as_float(a.y << 16), __uint_as_float(a.y & 0xffff0000u));
    }
};
template <> struct Four<float> {
    float4 a;
    __device__ __forceinline__ void load(const float* p) { a = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void zero() { a = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float2* v) const {
        v[0] = make_float2(a.x, a.y);
        v[1] = make_float2(a.z, a.w);
    }
};
// A row's four channels copied ahead into shared memory; the thread that copies
// them is the one that reads them, so no barrier is needed.
template <typename T>
__device__ __forceinline__ void copy4(Four<T>* to, const T* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
                 "n"((int)sizeof(T) * kC) : "memory");
}

__device__ __forceinline__ void store4(__nv_bfloat16* p, const float2* v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0].x, v[0].y), b = __floats2bfloat162_rn(v[1].x, v[1].y);
    *reinterpret_cast<uint2*>(p) = make_uint2(reinterpret_cast<const uint32_t&>(a), reinterpret_cast<const uint32_t&>(b));
}
__device__ __forceinline__ void store4(float* p, const float2* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
}

// Tokens of a slot: `most`, or fewer where that leaves the GPU without threads
// (some 1024 per SM), down to 16.
int slot_tokens(int most, long long tokens, int D, int num_sms) {
    int seg = most;
    while (seg > 16 && tokens / seg * (D / kC) < num_sms * 1024LL) seg /= 2;
    return seg;
}

template <int K>
struct Taps {
    float2 w[K][kP], b[kP];
    __device__ __forceinline__ void load(const float* wp, const float* bp, int c) {
        float flat[K * kC];
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const float4 q = reinterpret_cast<const float4*>(wp + (size_t)c * K)[i];
            flat[4 * i] = q.x; flat[4 * i + 1] = q.y; flat[4 * i + 2] = q.z; flat[4 * i + 3] = q.w;
        }
        const float4 q = bp ? *reinterpret_cast<const float4*>(bp + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float bias[kC] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            b[p] = make_float2(bias[2 * p], bias[2 * p + 1]);
#pragma unroll
            for (int k = 0; k < K; ++k) w[k][p] = make_float2(flat[2 * p * K + k], flat[(2 * p + 1) * K + k]);
        }
    }
    // The sum before the activation of pair p, from the K-1 rows before and the row itself.
    __device__ __forceinline__ float2 sum(const float2 (*past)[kP], float2 now, int p) const {
        float2 s = b[p];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) s = fma2(w[k][p], past[k][p], s);
        return fma2(w[K - 1][p], now, s);
    }
};

template <int K>
__device__ __forceinline__ void shift_in(float2 (*past)[kP], const float2* now) {
#pragma unroll
    for (int p = 0; p < kP; ++p) {
#pragma unroll
        for (int k = 0; k + 1 < K - 1; ++k) past[k][p] = past[k + 1][p];
        past[K - 2][p] = now[p];
    }
}

// Row t (within its sequence) of the inputs; t in [-(K-1), seq_len).
template <typename T, int K>
__device__ __forceinline__ void input_row(const ConvArgs& a, const Slot& f, int t, int c, float2* v) {
    Four<T> r;
    r.zero();
    if (t >= 0)
        r.load(static_cast<const T*>(a.x) + (f.row0 + t) * a.ldx + c);
    else if (a.tail0)
        r.load(static_cast<const T*>(a.tail0) + ((size_t)f.b * (K - 1) + (K - 1 + t)) * a.D + c);
    r.get(v);
}

template <bool B> struct Flag { static constexpr bool value = B; };

template <typename T, int K>
__global__ void __launch_bounds__(kThreads, 6) short_conv_kernel(const ConvArgs a) {
    __shared__ __align__(16) Four<T> ring[kAhead + 1][kBatch][kThreads];
    const Slot f = find_slot(a.rows, blockIdx.x);
    const int c = (blockIdx.y * kThreads + threadIdx.x) * kC;
    if (f.b < 0 || c >= a.D) return;
    Taps<K> taps;
    taps.load(a.w, a.bias, c);
    float2 past[K - 1][kP];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) input_row<T, K>(a, f, f.first - (K - 1) + j, c, past[j]);
    const T* x = static_cast<const T*>(a.x) + (f.row0 + f.first) * a.ldx + c;
    T* y = static_cast<T*>(a.y) + (f.row0 + f.first) * (long long)a.D + c;
    auto fetch = [&](int left, int slot) {                  // x points at the batch's first row
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (k < left) copy4(&ring[slot][k][threadIdx.x], x + k * a.ldx);
        copies_end();
        x += kBatch * a.ldx;
    };
    // left: rows that remain; kWhole: a batch of them at least
    auto walk = [&](int slot, int left, auto whole) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (!decltype(whole)::value && k >= left) break;
            float2 now[kP], out[kP];
            ring[slot][k][threadIdx.x].get(now);
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const float2 s = taps.sum(past, now[p], p);
                out[p] = a.swish ? mul2(s, sigmoid2(s)) : s;
            }
            shift_in<K>(past, now);
            store4(y + k * (long long)a.D, out);
        }
        y += kBatch * (long long)a.D;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(f.len - i * kBatch, i);
    int slot = 0;
    for (int left = f.len; left > 0; left -= kBatch) {
        fetch(left - kAhead * kBatch, slot == 0 ? kAhead : slot - 1);
        copies_wait<kAhead>();
        if (left >= kBatch)
            walk(slot, left, Flag<true>());
        else
            walk(slot, left, Flag<false>());
        slot = slot == kAhead ? 0 : slot + 1;
    }
    if (a.tail && f.s == max(f.segs, 1) - 1) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            store4(static_cast<T*>(a.tail) + ((size_t)f.b * (K - 1) + j) * a.D + c, past[j]);
    }
}

// One token per sequence.  tail may be tail0: a thread reads what it owns
// before it writes.
template <typename T, int K>
__global__ void __launch_bounds__(kThreads) short_conv_step_kernel(const ConvArgs a) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int groups = a.D / kC;
    if (i >= (long long)a.rows.B * groups) return;
    const int b = (int)(i / groups), c = (int)(i - (long long)b * groups) * kC;
    const T* old = static_cast<const T*>(a.tail0) + (size_t)b * (K - 1) * a.D + c;
    T* next = static_cast<T*>(a.tail) + (size_t)b * (K - 1) * a.D + c;
    Four<T> r[K];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) r[j].load(old + (size_t)j * a.D);
    r[K - 1].load(static_cast<const T*>(a.x) + b * a.ldx + c);
    Taps<K> taps;
    taps.load(a.w, a.bias, c);
    float2 v[K][kP], out[kP];
#pragma unroll
    for (int j = 0; j < K; ++j) r[j].get(v[j]);
#pragma unroll
    for (int p = 0; p < kP; ++p) {
        const float2 s = taps.sum(v, v[K - 1][p], p);
        out[p] = a.swish ? mul2(s, sigmoid2(s)) : s;
    }
    store4(static_cast<T*>(a.y) + (size_t)b * a.D + c, out);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store4(next + (size_t)j * a.D, v[j + 1]);
}

// Gradients.  With ds[t] = dy[t] act'(s[t]) (s formed again from the inputs):
//   dx[t]   = sum_j w[K-1-j] ds[t+j]      (rows before the first token: dtail0)
//   dw[k]   = sum_t ds[t] x[t-K+1+k],  dbias = sum_t ds[t]
// and dtail adds to the last K-1 rows.  A thread walks one slot and K-1 tokens
// past its end; the slots of a block add up their dw and dbias in shared memory.
// 109 us at 16384 x 4096, bf16 (150 us with a condition per row for the slot's
// ends).  No unit is full (59 % of the issue slots, 33 % of the special functions,
// 0.58 of the copy rate): at 128 registers 16 warps an SM hide too little of each
// row's chain from copy to sum.  fp32, with twice the bytes, takes 157 us.
constexpr int kBackGroups = 32, kBackSlots = 4, kBackSeg = 128, kBackBatch = 4, kBackAhead = 1;

template <typename T, int K>
__global__ void __launch_bounds__(kBackGroups* kBackSlots, 4) short_conv_backward_kernel(const ConvBackwardArgs g,
                                                                                     float* partial, int slots) {
    __shared__ float red[kBackSlots][kBackGroups * kC + 1];
    __shared__ __align__(16) Four<T> ring[kBackAhead + 1][2][kBackBatch][kBackGroups * kBackSlots];
    const int tid = threadIdx.y * kBackGroups + threadIdx.x;
    const ConvArgs& a = g.f;
    const int item = blockIdx.x * kBackSlots + threadIdx.y;
    const int c = (blockIdx.y * kBackGroups + threadIdx.x) * kC;
    float2 dw[K + 1][kP];
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
        for (int p = 0; p < kP; ++p) dw[k][p] = both(0.f);
    if (item < slots && c < a.D) {
        const Slot f = find_slot(a.rows, item);
        Taps<K> taps;
        taps.load(a.w, a.bias, c);
        float2 past[K - 1][kP], ds[K][kP];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) input_row<T, K>(a, f, f.first - (K - 1) + j, c, past[j]);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int p = 0; p < kP; ++p) ds[k][p] = both(0.f);
        const int end = f.first + f.len, tail_at = f.seq_len - (K - 1), stop = end + K - 1;
        const int lo = f.first == 0 ? (g.dtail0 ? -(K - 1) : 0) : f.first;
        const T* x = static_cast<const T*>(a.x) + (f.row0 + f.first) * a.ldx + c;
        const T* dy = static_cast<const T*>(g.dy) + (f.row0 + f.first) * (long long)a.D + c;
        T* dx = static_cast<T*>(g.dx) + (f.row0 + f.first - (K - 1)) * (long long)a.D + c;
        // x and dy point at row t0; no gradient comes from behind the last token
        auto fetch = [&](int t0, int slot) {
            const int have = min(stop, f.seq_len) - t0;
#pragma unroll
            for (int i = 0; i < kBackBatch; ++i) {
                if (i < have) {
                    copy4(&ring[slot][0][i][tid], x + i * a.ldx);
                    copy4(&ring[slot][1][i][tid], dy + i * (long long)a.D);
                } else {
                    ring[slot][0][i][tid].zero();
                    ring[slot][1][i][tid].zero();
                }
            }
            copies_end();
            x += kBackBatch * a.ldx;
            dy += kBackBatch * (long long)a.D;
        };
        // rows t0 .. of the batch; kInside: all of them the slot's own, and all rows of dx that they end too
        auto walk = [&](int t0, int slot, auto inside) {
            constexpr bool kInside = decltype(inside)::value;
#pragma unroll
            for (int i = 0; i < kBackBatch; ++i) {
                const int t = t0 + i;
                if (!kInside && t >= stop) break;
                float2 now[kP], d[kP];
                ring[slot][0][i][tid].get(now);
                ring[slot][1][i][tid].get(d);
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    const float2 s = taps.sum(past, now[p], p);
                    if (a.swish) d[p] = mul2(d[p], swish_slope2(s, sigmoid2(s)));
#pragma unroll
                    for (int k = 0; k + 1 < K; ++k) ds[k][p] = ds[k + 1][p];
                    ds[K - 1][p] = d[p];
                    if (kInside || t < end) {
#pragma unroll
                        for (int k = 0; k < K - 1; ++k) dw[k][p] = fma2(d[p], past[k][p], dw[k][p]);
                        dw[K - 1][p] = fma2(d[p], now[p], dw[K - 1][p]);
                        dw[K][p] = add2(dw[K][p], d[p]);
                    }
                }
                shift_in<K>(past, now);
                const int r = t - (K - 1);
                if (!kInside && r < lo) continue;
                float2 out[kP];
#pragma unroll
                for (int p = 0; p < kP; ++p) out[p] = both(0.f);
                if (!kInside && g.dtail && r >= tail_at) {
                    Four<T> x0;
                    x0.load(static_cast<const T*>(g.dtail) + ((size_t)f.b * (K - 1) + (r - tail_at)) * a.D + c);
                    x0.get(out);
                }
#pragma unroll
                for (int p = 0; p < kP; ++p)
#pragma unroll
                    for (int j = 0; j < K; ++j) out[p] = fma2(taps.w[K - 1 - j][p], ds[j][p], out[p]);
                if (kInside || r >= 0)
                    store4(dx + i * (long long)a.D, out);
                else
                    store4(static_cast<T*>(g.dtail0) + ((size_t)f.b * (K - 1) + (K - 1 + r)) * a.D + c, out);
            }
            dx += kBackBatch * (long long)a.D;
        };
#pragma unroll
        for (int i = 0; i < kBackAhead; ++i) fetch(f.first + i * kBackBatch, i);
        int slot = 0;
        for (int t0 = f.first; t0 < stop; t0 += kBackBatch) {
            fetch(t0 + kBackAhead * kBackBatch, slot == 0 ? kBackAhead : slot - 1);
            copies_wait<kBackAhead>();
            if (t0 >= f.first + K - 1 && t0 + kBackBatch <= end && t0 + kBackBatch - K < tail_at)
                walk(t0, slot, Flag<true>());
            else
                walk(t0, slot, Flag<false>());
            slot = slot == kBackAhead ? 0 : slot + 1;
        }
    }
    const int ch = blockIdx.y * kBackGroups * kC + tid;
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        __syncthreads();
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            red[threadIdx.y][threadIdx.x * kC + 2 * p] = dw[k][p].x;
            red[threadIdx.y][threadIdx.x * kC + 2 * p + 1] = dw[k][p].y;
        }
        __syncthreads();
        if (ch < a.D) {
            float s = 0.f;
#pragma unroll
            for (int y = 0; y < kBackSlots; ++y) s += red[y][tid];
            partial[((size_t)blockIdx.x * (K + 1) + k) * a.D + ch] = s;
        }
    }
}
static_assert(kBackGroups * kC == kBackGroups * kBackSlots, "a thread of the block for each of its channels");

template <typename T, int K>
cudaError_t conv_backward(const ConvBackwardArgs& g, cudaStream_t s) {
    const long long slots = slots_of(g.f.rows);
    const int D = g.f.D;
    const dim3 grid((unsigned)((slots + kBackSlots - 1) / kBackSlots), (D + kBackGroups * kC - 1) / (kBackGroups * kC));
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
    const dim3 grid((unsigned)slots_of(a.rows), (a.D / kC + kThreads - 1) / kThreads);
    short_conv_kernel<T, K><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int K>
cudaError_t conv_step(const ConvArgs& a, cudaStream_t s) {
    const long long threads = (long long)a.rows.B * (a.D / kC);
    short_conv_step_kernel<T, K><<<(unsigned)((threads + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_short_conv(ConvArgs a, int num_sms, cudaStream_t s) {
    a.rows.seg = slot_tokens(kSeg, a.rows.cu ? a.rows.total : (long long)a.rows.B * a.rows.N, a.D, num_sms);
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

size_t short_conv_backward_ws_bytes(int B, int N, int D, int K, int num_sms) {
    const int seg = slot_tokens(kBackSeg, (long long)B * N, D, num_sms);
    const long long slots = (long long)B * segments_of(N, seg);
    return align256((size_t)((slots + kBackSlots - 1) / kBackSlots) * (K + 1) * D * sizeof(float));
}

cudaError_t launch_short_conv_backward(ConvBackwardArgs g, int num_sms, cudaStream_t s) {
    const int K = g.f.K;
    g.f.rows.seg = slot_tokens(kBackSeg, (long long)g.f.rows.B * g.f.rows.N, g.f.D, num_sms);
    if (g.f.io == GRET_BF16) {
        if (K == 2) return conv_backward<__nv_bfloat16, 2>(g, s);
        return K == 3 ? conv_backward<__nv_bfloat16, 3>(g, s) : conv_backward<__nv_bfloat16, 4>(g, s);
    }
    if (K == 2) return conv_backward<float, 2>(g, s);
    return K == 3 ? conv_backward<float, 3>(g, s) : conv_backward<float, 4>(g, s);
}

}  // namespace gret
