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
// written once, and the memory bandwidth bounds the time: 107 us at 16384 x 4096
// bf16, 0.97 of a plain copy's rate (197 us without the copies ahead).  n is
// formed from r before r is rounded to its storage type.
#include "gret_block.cuh"
#include "gret_sm100.cuh"

namespace gret {
using namespace sm100;
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

// Eight sums behind one barrier, which also orders the block's shared memory
// before and after it, in a block of one warp too (a shuffle alone does not: the
// row that a copy is about to replace has been read by all); `red`: 128 words (at
// most 16 warps).  Each
// round halves the values a lane keeps, so that a lane ends with one of the
// eight over its warp, and after the barrier with one over four warps.
__device__ __forceinline__ void block_sums(float* v, float* red) {
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 16;
        x[i] = (up ? v[i + 4] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 4], 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 8;
        x[i] = (up ? x[i + 2] : x[i]) + __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + 2], 8);
    }
    const bool up = lane & 4;
    float sum = (up ? x[1] : x[0]) + __shfl_xor_sync(0xffffffffu, up ? x[0] : x[1], 4);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    if (warps > 1) {
        // value lane / 4 of every warp: a quarter of the warps for each of its four lanes
        if ((lane & 3) == 0) red[(lane >> 2) * 16 + (threadIdx.x >> 5)] = sum;
        __syncthreads();
        const float4 q = *reinterpret_cast<const float4*>(red + (lane >> 2) * 16 + (lane & 3) * 4);
        const int left = warps - (lane & 3) * 4;
        sum = (left > 0 ? q.x : 0.f) + (left > 1 ? q.y : 0.f) + (left > 2 ? q.z : 0.f) + (left > 3 ? q.w : 0.f);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    } else {
        __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __shfl_sync(0xffffffffu, sum, 4 * i);
}

// A vector as four pairs, from a row in shared or global memory.
template <typename T>
__device__ __forceinline__ void load_pairs(const T* p, float2* v) {
    Raw<T> r;
    r.load(p);
    pairs_of(r, v);
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

// TS: the residual stream's type; T: the block's.  kFull: y, gate and both
// norms are given and the threads' vectors fill the row, so that no part's
// absence cuts the code into pieces that loads cannot cross.
template <typename TS, typename T, int V, int kStages, bool kFull>
__global__ void __launch_bounds__(512) residual_norm_kernel(const NormArgs a) {
    extern __shared__ __align__(16) uint4 stage[];
    __shared__ float red[4][32];
    constexpr int kPieces = V * (kParts<TS> + 2 * kParts<T>);
    const int D = a.D;
    const bool has_y = kFull || a.y, has_gate = kFull || a.gate, has_post = kFull || a.w_post, has_next = kFull || a.w_next;
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
                if (kFull || c < D) {
                    copy_vector(to, static_cast<const TS*>(a.x) + t * a.ldx + c);
                    if (has_y) copy_vector(to + kParts<TS> * blockDim.x, static_cast<const T*>(a.y) + t * a.ldy + c);
                    if (has_gate)
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
            if (kFull || c < D) {
                read_vector<TS>(from, r[j]);
                if (has_y) read_vector<T>(from + kParts<TS> * blockDim.x, p[j]);
            }
            from += (kParts<TS> + 2 * kParts<T>)*blockDim.x;
        }
        if (has_y) {
            float k = 1.f;
            if (has_post) {
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
                if (kFull || c < D) {
                    float g[kVec];
                    if (has_gate) read_vector<T>(from, g);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        float v = p[j][e] * k * w_post[j][e] * scale[j][e];
                        if (has_gate) v *= g[e] * sigmoid_fast(g[e]);
                        r[j][e] += v;
                    }
                    store8(static_cast<TS*>(a.r) + t * D + c, r[j]);
                }
                from += (kParts<TS> + 2 * kParts<T>)*blockDim.x;
            }
        }
        if (has_next) {
            float sq = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int e = 0; e < kVec; ++e) sq = fmaf(r[j][e], r[j][e], sq);
            const float k = rsqrtf(block_sum(sq, red[turn + 1]) / (float)D + a.eps);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (threadIdx.x + j * blockDim.x) * kVec;
                if (!kFull && c >= D) continue;
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
// A block walks rows as in the forward and keeps its share of the three
// parameter gradients in registers, which it leaves to the column sums.  Its
// rows come by bulk copies into kStages rows of shared memory, issued by one
// thread: copies by every thread, as in the forward, took 328 us instead of
// 254 at 16384 x 4096 beside an fp32 stream, as five inputs a row keep the load
// and store unit busy.  The last mean is sum(dx v) / D with v = r - x, and
// dx is linear in dr, t and r: its parts are summed with r^2 and t r, and the
// next row's y^2 with them, so that a row costs one barrier; the same sums
// carry the word that a wait gave up, and the block then returns together.
// kFull: every part is given and the threads' vectors fill the row, so that no
// part's absence cuts the code into pieces that loads cannot cross.
template <typename TS, typename T, int V, int kStages, bool kFull>
__global__ void __launch_bounds__(512) residual_norm_backward_kernel(const NormBackwardArgs g, float* partial) {
    extern __shared__ __align__(128) unsigned char rows[];
    __shared__ __align__(16) float red[2][128], first[2][32];
    __shared__ __align__(8) unsigned long long full[kStages], never;
    __shared__ volatile int gave_up;
    const NormArgs& a = g.f;
    constexpr int kP = kVec / 2;
    const int D = a.D;
    const bool has_y = kFull || a.y, has_gate = kFull || a.gate, has_next = kFull || a.w_next, has_dr = kFull || g.dr,
               has_post = kFull || a.w_post;
    const float2 one = both(1.f), none = both(0.f);
    // a row in shared memory: x, dr; y, gate, dn
    const uint32_t stream_bytes = D * (uint32_t)sizeof(TS), block_bytes = D * (uint32_t)sizeof(T);
    const uint32_t row_bytes = 2 * stream_bytes + 3 * block_bytes;
    struct Row {
        const TS *x, *dr;
        const T *y, *gate, *dn;
    };
    auto row_at = [&](int s) {
        const unsigned char* p = rows + (size_t)s * row_bytes;
        Row r;
        r.x = reinterpret_cast<const TS*>(p);
        r.dr = r.x + D;
        r.y = reinterpret_cast<const T*>(r.dr + D);
        r.gate = r.y + D;
        r.dn = r.gate + D;
        return r;
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(smem_u32(&full[s]), 1);
        mbar_init(smem_u32(&never), 1);
        gave_up = 0;
        fence_mbar_init();
        if (g.fault) mbar_wait_injected_timeout(smem_u32(&never), g.status, &gave_up);
    }
    __syncthreads();
    // the block's i-th row into stage i mod kStages (one thread)
    auto row_of = [&](long long i) { return blockIdx.x + i * gridDim.x; };
    auto fetch = [&](long long i) {
        const long long t = row_of(i);
        if (threadIdx.x != 0 || t >= a.T) return;
        const int s = (int)(i % kStages);
        const uint32_t bar = smem_u32(&full[s]);
        uint32_t to = smem_u32(rows) + s * row_bytes;
        mbar_arrive_expect_tx(bar, stream_bytes * (has_dr ? 2 : 1) +
                                       block_bytes * ((has_y ? 1 : 0) + (has_gate ? 1 : 0) + (has_next ? 1 : 0)));
        bulk_load(to, static_cast<const TS*>(a.x) + t * a.ldx, stream_bytes, bar);
        to += stream_bytes;
        if (has_dr) bulk_load(to, static_cast<const TS*>(g.dr) + t * D, stream_bytes, bar);
        to += stream_bytes;
        if (has_y) bulk_load(to, static_cast<const T*>(a.y) + t * a.ldy, block_bytes, bar);
        to += block_bytes;
        if (has_gate) bulk_load(to, static_cast<const T*>(a.gate) + t * a.ldg, block_bytes, bar);
        to += block_bytes;
        if (has_next) bulk_load(to, static_cast<const T*>(g.dn) + t * D, block_bytes, bar);
    };
    auto arrived = [&](long long i) {
        return row_of(i) >= a.T || mbar_wait(smem_u32(&full[i % kStages]), (uint32_t)(i / kStages) & 1u, g.status, &gave_up);
    };
    // dscale, dw_post, dw_next; and the parameters, where a thread has one vector and registers for them
    constexpr bool kKeep = V == 1, kAhead = kStages >= 3;
    float2 acc[3][V][kP], kept[3][kP];
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
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
    const float over = 1.0f / (float)D;
    // sum of y^2 over the thread's share of a row
    auto square = [&](const Row& row) {
        float2 sq = none;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (threadIdx.x + j * blockDim.x) * kVec;
            if (!kFull && c >= D) continue;
            float2 y[kP];
            load_pairs(row.y + c, y);
#pragma unroll
            for (int p = 0; p < kP; ++p) sq = fma2(y[p], y[p], sq);
        }
        return sq.x + sq.y;
    };
    int turn = 0;
    float y2 = 0.f;                                         // sum of y^2 of the row
    bool ok = true;
    if (kAhead && has_post) {
        ok = arrived(0);
        y2 = block_sum(square(row_at(0)), first[0]);
    }
    for (long long i = 0; row_of(i) < a.T; ++i) {
        const long long t = row_of(i);
        if (!kAhead) {
            __syncthreads();                                // everyone is done with the row before
            fetch(i + kStages - 1);
        }
        ok = arrived(i) && ok;
        if (kAhead) ok = arrived(i + 1) && ok;
        const Row row = row_at((int)(i % kStages));
        if (!kAhead && has_post) y2 = block_sum(square(row), first[turn]);
        const float ky = has_post ? rsqrtf(y2 * over + a.eps) : 1.f;
        float2 r[V][kP], yn[V][kP];
        // dr v, t v, r v, r^2, t r with v = r - x; and the next row's y^2
        float2 sum[5] = {none, none, none, none, none};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (threadIdx.x + j * blockDim.x) * kVec;
#pragma unroll
            for (int p = 0; p < kP; ++p) r[j][p] = yn[j][p] = none;
            if (!kFull && c >= D) continue;
            load_pairs(row.x + c, r[j]);
            float2 v[kP], dr[kP], w[kP], dn[kP];
#pragma unroll
            for (int p = 0; p < kP; ++p) v[p] = dr[p] = none;
            if (has_dr) load_pairs(row.dr + c, dr);
            if (has_y) {
                float2 gt[kP], sc[kP];
                load_pairs(row.y + c, yn[j]);
                weights(a.w_post, 1, c, w);
                weights(a.scale, 0, c, sc);
                if (has_gate) load_pairs(row.gate + c, gt);
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    yn[j][p] = mul2(yn[j][p], both(ky));
                    v[p] = mul2(yn[j][p], mul2(w[p], sc[p]));
                    if (has_gate) v[p] = mul2(v[p], mul2(gt[p], sigmoid2(gt[p])));
                    r[j][p] = add2(r[j][p], v[p]);
                    sum[0] = fma2(dr[p], v[p], sum[0]);
                }
            }
            if (has_next) {
                weights(a.w_next, 2, c, w);
                load_pairs(row.dn + c, dn);
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    const float2 tt = mul2(dn[p], w[p]);
                    sum[1] = fma2(tt, v[p], sum[1]);
                    sum[2] = fma2(r[j][p], v[p], sum[2]);
                    sum[3] = fma2(r[j][p], r[j][p], sum[3]);
                    sum[4] = fma2(tt, r[j][p], sum[4]);
                }
            }
        }
        float all[8] = {};
#pragma unroll
        for (int k = 0; k < 5; ++k) all[k] = sum[k].x + sum[k].y;
        all[5] = kAhead && has_post && row_of(i + 1) < a.T ? square(row_at((int)((i + 1) % kStages))) : 0.f;
        all[6] = ok ? 0.f : 1.f;
        block_sums(all, red[turn]);
        if (!(all[6] == 0.f)) {
            // a copy did not arrive: let those issued land, as far as they do, and leave
            if (threadIdx.x == 0)
                for (long long k = i; k < i + (kAhead ? kStages - 1 : kStages); ++k)
                    if (row_of(k) < a.T)
                        mbar_wait_drain(smem_u32(&full[k % kStages]), (uint32_t)(k / kStages) & 1u, kWaitCycles);
            return;
        }
        if (kAhead) fetch(i + kStages - 1);
        y2 = all[5];
        const float kr = has_next ? rsqrtf(all[3] * over + a.eps) : 0.f, m = all[4] * kr * over;
        // mean of (gradient of yn) yn: the total gradient of r is dr + kr (t - r kr m)
        const float m4 = has_post ? (all[0] + kr * (all[1] - kr * m * all[2])) * over : 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (threadIdx.x + j * blockDim.x) * kVec;
            if (!kFull && c >= D) continue;
            float2 dr[kP], w[kP];
#pragma unroll
            for (int p = 0; p < kP; ++p) dr[p] = none;
            if (has_dr) load_pairs(row.dr + c, dr);
            if (has_next) {
                float2 dn[kP];
                weights(a.w_next, 2, c, w);
                load_pairs(row.dn + c, dn);
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    const float2 rn = mul2(r[j][p], both(kr));
                    acc[2][j][p] = fma2(dn[p], rn, acc[2][j][p]);
                    dr[p] = fma2(both(kr), fma2(rn, both(-m), mul2(dn[p], w[p])), dr[p]);
                }
            }
            store_pairs(static_cast<TS*>(g.dx) + t * D + c, dr);
            if (!has_y) continue;
            float2 gt[kP], sc[kP], dy[kP];
            weights(a.w_post, 1, c, w);
            weights(a.scale, 0, c, sc);
            if (has_gate) load_pairs(row.gate + c, gt);
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const float2 q = mul2(yn[j][p], w[p]);
                const float2 sig = has_gate ? sigmoid2(gt[p]) : one, sw = has_gate ? mul2(gt[p], sig) : one;
                const float2 dp = mul2(dr[p], sc[p]), dq = mul2(dp, sw);
                acc[0][j][p] = fma2(dr[p], mul2(q, sw), acc[0][j][p]);
                acc[1][j][p] = fma2(dq, yn[j][p], acc[1][j][p]);
                dy[p] = mul2(both(ky), fma2(yn[j][p], both(-m4), mul2(dq, w[p])));
                if (has_gate) gt[p] = mul2(mul2(dp, q), swish_slope2(gt[p], sig));
            }
            if (has_gate) store_pairs(static_cast<T*>(g.dgate) + t * D + c, gt);
            store_pairs(static_cast<T*>(g.dy) + t * D + c, dy);
        }
        turn ^= 1;
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
    if (bytes <= 46 * 1024) return cudaSuccess;             // every kernel may have 48 KB, its static words included
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename TS, typename T, int V>
cudaError_t norm(const NormArgs& a, int num_sms, cudaStream_t s) {
    constexpr int kStages = V == 2 && sizeof(T) == 4 ? 2 : 3;   // what fits in shared memory at 8192 channels
    const int threads = block_threads(a.D, V), per_sm = (V == 1 ? 768 : 512) / threads;
    const int bytes = kStages * V * (kParts<TS> + 2 * kParts<T>)*threads * 16;
    const bool full = a.y && a.gate && a.w_post && a.w_next && threads * V * kVec == a.D;
    auto k = full ? residual_norm_kernel<TS, T, V, kStages, true> : residual_norm_kernel<TS, T, V, kStages, false>;
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
    const NormArgs& a = g.f;
    const int bytes = kStages * a.D * (int)(2 * sizeof(TS) + 3 * sizeof(T));
    const bool full = a.y && a.gate && a.scale && a.w_post && a.w_next && g.dr && threads * V * kVec == a.D;
    auto k = full ? residual_norm_backward_kernel<TS, T, V, kStages, true>
                  : residual_norm_backward_kernel<TS, T, V, kStages, false>;
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

// As many rows in shared memory as fit for all blocks of an SM: 512 threads'
// worth of rows take 14 bytes a channel beside an fp32 stream, so that four rows
// fit one block (3 rows 299 us, 4 rows 254 us at 16384 x 4096) but not several.
// Two rows of fp32 take 394 us there (0.85 of the copy rate).  Above 4096 channels
// two rows fit, or one of fp32, whose copy then overlaps nothing: 576, 782 and
// 1019 us at 16384 x 8192 in bf16, beside an fp32 stream and in fp32 (0.58, 0.59
// and 0.65 of the copy rate).
template <typename TS, typename T>
cudaError_t norm_backward(const NormBackwardArgs& g, int grid, cudaStream_t s) {
    constexpr bool kWide = sizeof(TS) == 4, kAll = sizeof(T) == 4;
    if (backward_vectors(g.f.D) == 2) return norm_backward<TS, T, 2, kAll ? 1 : 2>(g, grid, s);
    if constexpr (kAll) {
        return norm_backward<TS, T, 1, 2>(g, grid, s);
    } else {
        if (kWide && block_threads(g.f.D, 1) <= 256) return norm_backward<TS, T, 1, 3>(g, grid, s);
        return norm_backward<TS, T, 1, kWide ? 4 : 5>(g, grid, s);
    }
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
