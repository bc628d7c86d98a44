// The norm after a block, its gate and residual scale, and the norm before the
// next block, in one pass over the rows:
//
//   p = rms(y) (.) w_post (.) swish(gate),  r = x + scale (.) p,  n = rms(r) (.) w_next
//   rms(v) = v / sqrt(mean(v^2) + eps)
//
// A block of threads walks rows blockIdx.x, + gridDim.x, ...; each thread owns
// the same 16-byte vectors of every row and copies them asynchronously into
// shared memory kStages - 1 rows ahead.  It reads back only what it copied
// itself, so the copies need no barrier; the only ones are the row sums', which
// are taken from registers in fp32.  Every input is read once and every output
// written once, and the memory bandwidth bounds the time.  n is formed from r
// before r is rounded to its storage type.
#include "gret_block.cuh"

namespace gret {
namespace {

// Copies of one thread's vectors of a row: `Parts` 16-byte pieces of each.
template <typename T> constexpr int kParts = (int)sizeof(T) / 2;
__device__ __forceinline__ void copy_async(uint4* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from)
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void copy_vector(uint4* to, const T* from) {
#pragma unroll
    for (int p = 0; p < kParts<T>; ++p) copy_async(to + p * blockDim.x, reinterpret_cast<const uint4*>(from) + p);
}
template <typename T>
__device__ __forceinline__ void read_vector(const uint4* from, float* v) {
    Raw<T> r;
    const uint4 a = from[0];
    if constexpr (kParts<T> == 1) {
        r.a = a;
    } else {
        const uint4 b = from[blockDim.x];
        r.a = reinterpret_cast<const float4&>(a);
        r.b = reinterpret_cast<const float4&>(b);
    }
    r.get(v);
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// `red`: 32 words of shared memory; a caller takes others for the next two
// sums, so that one barrier a sum is enough.
__device__ __forceinline__ float block_sum(float v, float* red) {
    const int warps = blockDim.x >> 5;
    v = warp_sum(v);
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum((threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f);
}

// Two sums behind one barrier; `red`: 64 words.
__device__ __forceinline__ float2 block_sum(float2 v, float* red) {
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if (warps == 1) return v;
    if (lane == 0) reinterpret_cast<float2*>(red)[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? reinterpret_cast<const float2*>(red)[lane] : make_float2(0.f, 0.f);
    return make_float2(warp_sum(v.x), warp_sum(v.y));
}

// A vector as four pairs.
template <typename T>
__device__ __forceinline__ void read_pairs(const uint4* from, float2* v) {
    float x[kVec];
    read_vector<T>(from, x);
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i) v[i] = make_float2(x[2 * i], x[2 * i + 1]);
}
__device__ __forceinline__ void load_pairs(const float* p, float2* v) {
    float x[kVec];
    load8(p, x);
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i) v[i] = make_float2(x[2 * i], x[2 * i + 1]);
}

// A parameter's values for the thread's vectors, or 1.
template <int V>
__device__ __forceinline__ void load_weights(float (*w)[kVec], const float* p, int D) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = (threadIdx.x + j * blockDim.x) * kVec;
#pragma unroll
        for (int e = 0; e < kVec; ++e) w[j][e] = 1.f;
        if (p && c < D) load8(p + c, w[j]);
    }
}

// TS: the residual stream's type; T: the block's.
template <typename TS, typename T, int V, int kStages>
__global__ void __launch_bounds__(512) residual_norm_kernel(const NormArgs a) {
    extern __shared__ __align__(16) uint4 stage[];
    __shared__ float red[4][32];
    constexpr int kPieces = V * (kParts<TS> + 2 * kParts<T>);
    const int D = a.D;
    float w_post[V][kVec], w_next[V][kVec], scale[V][kVec];
    load_weights<V>(w_post, a.w_post, D);
    load_weights<V>(w_next, a.w_next, D);
    load_weights<V>(scale, a.scale, D);
    auto fetch = [&](long long t, int s) {
        if (t < a.T) {
            uint4* to = stage + (size_t)s * kPieces * blockDim.x + threadIdx.x;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (threadIdx.x + j * blockDim.x) * kVec;
                if (c < D) {
                    copy_vector(to, static_cast<const TS*>(a.x) + t * a.ldx + c);
                    if (a.y) copy_vector(to + kParts<TS> * blockDim.x, static_cast<const T*>(a.y) + t * a.ldy + c);
                    if (a.gate)
                        copy_vector(to + (kParts<TS> + kParts<T>)*blockDim.x, static_cast<const T*>(a.gate) + t * a.ldg + c);
                }
                to += (kParts<TS> + 2 * kParts<T>)*blockDim.x;
            }
        }
        copies_end();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(blockIdx.x + (long long)s * gridDim.x, s);
    int s = 0, turn = 0;
    for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
        fetch(t + (long long)(kStages - 1) * gridDim.x, s == 0 ? kStages - 1 : s - 1);
        copies_wait<kStages - 1>();
        const uint4* from = stage + (size_t)s * kPieces * blockDim.x + threadIdx.x;
        float r[V][kVec], p[V][kVec];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (threadIdx.x + j * blockDim.x) * kVec;
#pragma unroll
            for (int e = 0; e < kVec; ++e) r[j][e] = p[j][e] = 0.f;
            if (c < D) {
                read_vector<TS>(from, r[j]);
                if (a.y) read_vector<T>(from + kParts<TS> * blockDim.x, p[j]);
            }
            from += (kParts<TS> + 2 * kParts<T>)*blockDim.x;
        }
        if (a.y) {
            float k = 1.f;
            if (a.w_post) {
                float sq = 0.f;
#pragma unroll
                for (int j = 0; j < V; ++j)
#pragma unroll
                    for (int e = 0; e < kVec; ++e) sq = fmaf(p[j][e], p[j][e], sq);
                k = rsqrtf(block_sum(sq, red[turn]) / (float)D + a.eps);
            }
            from = stage + (size_t)s * kPieces * blockDim.x + threadIdx.x + (kParts<TS> + kParts<T>)*blockDim.x;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (threadIdx.x + j * blockDim.x) * kVec;
                if (c < D) {
                    float g[kVec];
                    if (a.gate) read_vector<T>(from, g);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        float v = p[j][e] * k * w_post[j][e] * scale[j][e];
                        if (a.gate) v *= g[e] * sigmoid_fast(g[e]);
                        r[j][e] += v;
                    }
                    store8(static_cast<TS*>(a.r) + t * D + c, r[j]);
                }
                from += (kParts<TS> + 2 * kParts<T>)*blockDim.x;
            }
        }
        if (a.w_next) {
            float sq = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int e = 0; e < kVec; ++e) sq = fmaf(r[j][e], r[j][e], sq);
            const float k = rsqrtf(block_sum(sq, red[turn + 1]) / (float)D + a.eps);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (threadIdx.x + j * blockDim.x) * kVec;
                if (c >= D) continue;
                float n[kVec];
#pragma unroll
                for (int e = 0; e < kVec; ++e) n[e] = w_next[j][e] * (r[j][e] * k);
                store8(static_cast<T*>(a.n) + t * D + c, n);
            }
        }
        turn ^= 2;
        s = s + 1 == kStages ? 0 : s + 1;
    }
}

// Gradients, with everything of the forward formed again from x, y and gate
// (kv = 1 / rms(v), vn = v kv, q = yn w_post, t = dn w_next):
//   dx = dr + kr (t - rn mean(t rn)),  dscale = sum dx q swish(gate),  dw_next = sum dn rn
//   dp = dx scale,  dgate = dp q swish'(gate),  dq = dp swish(gate),  dw_post = sum dq yn
//   dy = ky (dq w_post - yn mean(dq w_post yn))
// Rows as in the forward; a block keeps its share of the three parameter
// gradients in registers and leaves it to the column sums.
template <typename TS, typename T, int V, int kStages>
__global__ void __launch_bounds__(512) residual_norm_backward_kernel(const NormBackwardArgs g, float* partial) {
    extern __shared__ __align__(16) uint4 stage[];
    __shared__ __align__(16) float red[2][128];
    const NormArgs& a = g.f;
    constexpr int kPer = 2 * kParts<TS> + 3 * kParts<T>, kP = kVec / 2;    // pieces of a vector: x, dr; y, gate, dn
    const int D = a.D;
    const float2 one = both(1.f), none = both(0.f);
    // dscale, dw_post, dw_next; and the parameters, where a thread has one vector and registers for them
    constexpr bool kKeep = V == 1;
    float2 acc[3][V][kP], kept[3][kP];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
#pragma unroll
        for (int p = 0; p < V * kP; ++p) acc[i][p / kP][p % kP] = none;
#pragma unroll
        for (int p = 0; p < kP; ++p) kept[i][p] = one;
        const float* w = i == 0 ? a.scale : i == 1 ? a.w_post : a.w_next;
        if (kKeep && w && threadIdx.x * kVec < D) load_pairs(w + threadIdx.x * kVec, kept[i]);
    }
    auto weights = [&](const float* w, int i, int c, float2* to) {
#pragma unroll
        for (int p = 0; p < kP; ++p) to[p] = kKeep ? kept[i][p] : one;
        if (!kKeep && w) load_pairs(w + c, to);
    };
    auto fetch = [&](long long t, int s) {
        if (t < a.T) {
            uint4* to = stage + (size_t)s * kPer * V * blockDim.x + threadIdx.x;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (threadIdx.x + j * blockDim.x) * kVec;
                if (c < D) {
                    copy_vector(to, static_cast<const TS*>(a.x) + t * a.ldx + c);
                    if (g.dr) copy_vector(to + kParts<TS> * blockDim.x, static_cast<const TS*>(g.dr) + t * D + c);
                    uint4* rest = to + 2 * kParts<TS> * blockDim.x;
                    if (a.y) copy_vector(rest, static_cast<const T*>(a.y) + t * a.ldy + c);
                    if (a.gate) copy_vector(rest + kParts<T> * blockDim.x, static_cast<const T*>(a.gate) + t * a.ldg + c);
                    if (g.dn) copy_vector(rest + 2 * kParts<T> * blockDim.x, static_cast<const T*>(g.dn) + t * D + c);
                }
                to += kPer * blockDim.x;
            }
        }
        copies_end();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(blockIdx.x + (long long)s * gridDim.x, s);
    const float over = 1.0f / (float)D;
    int s = 0, turn = 0;
    for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
        fetch(t + (long long)(kStages - 1) * gridDim.x, s == 0 ? kStages - 1 : s - 1);
        copies_wait<kStages - 1>();
        const uint4* row = stage + (size_t)s * kPer * V * blockDim.x + threadIdx.x;
        float* sums = red[turn];
        float2 r[V][kP], y[V][kP];                          // the sum r; y, then yn
        float ky = 1.f;
        {
            float2 sq = none;
#pragma unroll
            for (int j = 0; j < V; ++j) {
#pragma unroll
                for (int p = 0; p < kP; ++p) y[j][p] = none;
                if (a.y && (threadIdx.x + j * blockDim.x) * kVec < D)
                    read_pairs<T>(row + (j * kPer + 2 * kParts<TS>)*blockDim.x, y[j]);
#pragma unroll
                for (int p = 0; p < kP; ++p) sq = fma2(y[j][p], y[j][p], sq);
            }
            if (a.w_post) ky = rsqrtf(block_sum(sq.x + sq.y, sums) * over + a.eps);
        }
        float kr = 0.f, m = 0.f;
        {
            float2 s2 = none, s3 = none;                    // r^2, t r
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (threadIdx.x + j * blockDim.x) * kVec;
                const uint4* from = row + j * kPer * blockDim.x;
#pragma unroll
                for (int p = 0; p < kP; ++p) r[j][p] = none;
                if (c >= D) continue;
                read_pairs<TS>(from, r[j]);
                from += 2 * kParts<TS> * blockDim.x;
                float2 w[kP];
                if (a.y) {
                    float2 gt[kP], sc[kP];
                    weights(a.w_post, 1, c, w);
                    weights(a.scale, 0, c, sc);
                    if (a.gate) read_pairs<T>(from + kParts<T> * blockDim.x, gt);
#pragma unroll
                    for (int p = 0; p < kP; ++p) {
                        y[j][p] = mul2(y[j][p], both(ky));
                        float2 v = mul2(y[j][p], mul2(w[p], sc[p]));
                        if (a.gate) v = mul2(v, mul2(gt[p], sigmoid2(gt[p])));
                        r[j][p] = add2(r[j][p], v);
                    }
                }
                if (a.w_next) {
                    float2 dn[kP];
                    weights(a.w_next, 2, c, w);
                    read_pairs<T>(from + 2 * kParts<T> * blockDim.x, dn);
#pragma unroll
                    for (int p = 0; p < kP; ++p) {
                        s2 = fma2(r[j][p], r[j][p], s2);
                        s3 = fma2(mul2(dn[p], w[p]), r[j][p], s3);
                    }
                }
            }
            if (a.w_next) {
                const float2 v = block_sum(make_float2(s2.x + s2.y, s3.x + s3.y), sums + 32);
                kr = rsqrtf(v.x * over + a.eps);
                m = v.y * kr * over;
            }
        }
        float2 s4 = none;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (threadIdx.x + j * blockDim.x) * kVec;
            if (c >= D) continue;
            const uint4* from = row + j * kPer * blockDim.x;
            float2 dr[kP], w[kP];
#pragma unroll
            for (int p = 0; p < kP; ++p) dr[p] = none;
            if (g.dr) read_pairs<TS>(from + kParts<TS> * blockDim.x, dr);
            from += 2 * kParts<TS> * blockDim.x;
            if (a.w_next) {
                float2 dn[kP];
                weights(a.w_next, 2, c, w);
                read_pairs<T>(from + 2 * kParts<T> * blockDim.x, dn);
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    const float2 rn = mul2(r[j][p], both(kr));
                    acc[2][j][p] = fma2(dn[p], rn, acc[2][j][p]);
                    dr[p] = fma2(both(kr), fma2(rn, both(-m), mul2(dn[p], w[p])), dr[p]);
                }
            }
            store_pairs(static_cast<TS*>(g.dx) + t * D + c, dr);
            if (!a.y) continue;
            float2 gt[kP], sc[kP], dg[kP];
            weights(a.w_post, 1, c, w);
            weights(a.scale, 0, c, sc);
            if (a.gate) read_pairs<T>(from + kParts<T> * blockDim.x, gt);
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const float2 yn = y[j][p], q = mul2(yn, w[p]);
                const float2 sig = a.gate ? sigmoid2(gt[p]) : one, sw = a.gate ? mul2(gt[p], sig) : one;
                const float2 dp = mul2(dr[p], sc[p]), dq = mul2(dp, sw);
                acc[0][j][p] = fma2(dr[p], mul2(q, sw), acc[0][j][p]);
                acc[1][j][p] = fma2(dq, yn, acc[1][j][p]);
                if (a.gate) dg[p] = mul2(mul2(dp, q), swish_slope2(gt[p], sig));
                r[j][p] = mul2(dq, w[p]);                   // the gradient of yn
                s4 = fma2(r[j][p], yn, s4);
            }
            if (a.gate) store_pairs(static_cast<T*>(g.dgate) + t * D + c, dg);
        }
        if (a.y) {
            const float m4 = a.w_post ? block_sum(s4.x + s4.y, sums + 96) * over : 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (threadIdx.x + j * blockDim.x) * kVec;
                if (c >= D) continue;
#pragma unroll
                for (int p = 0; p < kP; ++p) r[j][p] = mul2(both(ky), fma2(y[j][p], both(-m4), r[j][p]));
                store_pairs(static_cast<T*>(g.dy) + t * D + c, r[j]);
            }
        }
        turn ^= 1;
        s = s + 1 == kStages ? 0 : s + 1;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (threadIdx.x + j * blockDim.x) * kVec;
            if (c < D) store_pairs(partial + ((size_t)blockIdx.x * 3 + i) * D + c, acc[i][j]);
        }
}

// Threads of a block for D channels, V vectors each.
int block_threads(int D, int V) { return ((D / kVec + V - 1) / V + 31) & ~31; }
int rows_grid(long long T, long long most) { return (int)(T < most ? T : most); }

template <typename K>
cudaError_t shared_limit(K kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename TS, typename T, int V>
cudaError_t norm(const NormArgs& a, int num_sms, cudaStream_t s) {
    constexpr int kStages = V == 2 && sizeof(T) == 4 ? 2 : 3;   // what fits in shared memory at 8192 channels
    const int threads = block_threads(a.D, V), per_sm = (V == 1 ? 768 : 512) / threads;
    const int bytes = kStages * V * (kParts<TS> + 2 * kParts<T>)*threads * 16;
    auto k = residual_norm_kernel<TS, T, V, kStages>;
    cudaError_t err = shared_limit(k, bytes);
    if (err != cudaSuccess) return err;
    k<<<rows_grid(a.T, (long long)num_sms * (per_sm > 0 ? per_sm : 1)), threads, bytes, s>>>(a);
    return cudaGetLastError();
}

template <typename TS, typename T>
cudaError_t norm(const NormArgs& a, int num_sms, cudaStream_t s) {
    return a.D <= 2048 ? norm<TS, T, 1>(a, num_sms, s) : norm<TS, T, 2>(a, num_sms, s);
}

int backward_vectors(int D) { return D <= 4096 ? 1 : 2; }
int backward_grid(long long T, int D, int num_sms) {
    const int per_sm = 512 / block_threads(D, backward_vectors(D));
    return rows_grid(T, (long long)num_sms * per_sm);
}

template <typename TS, typename T, int V, int kStages>
cudaError_t norm_backward(const NormBackwardArgs& g, int grid, cudaStream_t s) {
    const int threads = block_threads(g.f.D, V);
    const int bytes = kStages * V * (2 * kParts<TS> + 3 * kParts<T>)*threads * 16;
    auto k = residual_norm_backward_kernel<TS, T, V, kStages>;
    float* partial = static_cast<float*>(g.workspace);
    cudaError_t err = shared_limit(k, bytes);
    if (err != cudaSuccess) return err;
    k<<<grid, threads, bytes, s>>>(g, partial);
    err = cudaGetLastError();
    if (err != cudaSuccess || (!g.dscale && !g.dw_post && !g.dw_next)) return err;
    const long long D = g.f.D;
    const ColumnOutputs out = {3, {0, D, 2 * D, 3 * D}, {g.dscale, g.dw_post, g.dw_next}, {1, 1, 1}};
    return launch_column_sums(partial, grid, out, s);
}

// Three rows in flight where they fit in shared memory.
template <typename TS, typename T>
cudaError_t norm_backward(const NormBackwardArgs& g, int grid, cudaStream_t s) {
    if (backward_vectors(g.f.D) == 1) {
        if constexpr (sizeof(T) == 2) return norm_backward<TS, T, 1, 3>(g, grid, s);
        else return norm_backward<TS, T, 1, 2>(g, grid, s);
    }
    if constexpr (sizeof(T) == 2) return norm_backward<TS, T, 2, 2>(g, grid, s);
    else return norm_backward<TS, T, 2, 1>(g, grid, s);
}

}  // namespace

cudaError_t launch_residual_norm(const NormArgs& a, int num_sms, cudaStream_t s) {
    if (a.io == GRET_F32) return norm<float, float>(a, num_sms, s);
    if (a.stream_type == GRET_F32) return norm<float, __nv_bfloat16>(a, num_sms, s);
    return norm<__nv_bfloat16, __nv_bfloat16>(a, num_sms, s);
}

size_t residual_norm_backward_ws_bytes(long long T, int D, int num_sms) {
    return align256((size_t)backward_grid(T, D, num_sms) * 3 * D * sizeof(float));
}

cudaError_t launch_residual_norm_backward(NormBackwardArgs g, int num_sms, cudaStream_t s) {
    const int grid = backward_grid(g.f.T, g.f.D, num_sms);
    if (g.f.io == GRET_F32) return norm_backward<float, float>(g, grid, s);
    if (g.f.stream_type == GRET_F32) return norm_backward<float, __nv_bfloat16>(g, grid, s);
    return norm_backward<__nv_bfloat16, __nv_bfloat16>(g, grid, s);
}

}  // namespace gret
