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

// How a warp lays out its channels and states: a lane holds kLane states of CPL
// channels, n / kLane lanes share a channel, and the warp's kWidth channels are
// walked kTile tokens at a time.
constexpr int kLane = 4, kTile = 16, kWarps = 4;
template <int NS>
struct Layout {
    static constexpr int CPL = NS == 8 ? 2 : 4;            // channels of a lane
    static constexpr int LPC = NS / kLane;                 // lanes of a channel
    static constexpr int W = 32 / LPC * CPL;               // channels of a warp: 32, 32, 16, 8
    static constexpr int LD = W + 4;                       // shared row: 16-byte steps over the banks
    static constexpr int VR = W / kVec;                    // 16-byte vectors of a row
    static constexpr int V = (kTile * VR + 31) / 32;       // and of a lane
    static constexpr int BV = (kTile * NS / kVec + 31) / 32;   // vectors of B (of C) a lane stages
    static constexpr int FLOATS = 3 * kTile * LD + 2 * kTile * NS;   // shared floats of a warp
};

// Eight values as they lie in memory.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float* v) const { unpack8(a, v); }
};
template <> struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float* v) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// A warp walks one slot's tokens for its channels.  Each tile of tokens is
// staged first (delta and delta u of the warp's channels, B and C), then
// scanned token by token from shared memory, then gated and stored; the next
// tile's inputs are in flight meanwhile.  kFinal: the outputs, from the state
// before the slot (the folded one of a cut sequence).  Otherwise the state that
// the slot alone leaves, from zero, and the sum of its steps.
template <typename T, int NS, bool kFinal>
__global__ void __launch_bounds__(kWarps * 32, 3) selective_scan_kernel(const ScanArgs a, float* local, float* steps) {
    using L = Layout<NS>;
    constexpr int CPL = L::CPL, LPC = L::LPC, W = L::W, LD = L::LD, V = L::V, BV = L::BV, P = CPL / 2;
    __shared__ __align__(16) float smem[kWarps][L::FLOATS];
    const Slot f = find_slot(a.rows, blockIdx.x);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = a.D;
    const int d0 = (blockIdx.y * kWarps + warp) * W;
    if (f.b < 0 || d0 >= D) return;
    if (!kFinal && f.s + 1 >= f.segs) return;               // nothing comes after it
    float *sd = smem[warp], *su = sd + kTile * LD, *sy = su + kTile * LD, *sb = sy + kTile * LD, *sc = sb + kTile * NS;

    const int q = lane % LPC, g = lane / LPC;               // states 4 q .., channels d0 + g CPL ..
    float2 A[P][kLane], h[P][kLane];
    const float* h0 = nullptr;
    if (kFinal) {
        if (f.segs > 1 && f.s > 0)
            h0 = local + (size_t)(blockIdx.x - 1) * D * NS;
        else if (a.h0)
            h0 = a.h0 + (size_t)f.b * D * NS;
    }
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        const int d = d0 + g * CPL + c;
        float4 av = make_float4(0.f, 0.f, 0.f, 0.f), hv = av;
        if (d < D) {
            av = *reinterpret_cast<const float4*>(a.A + (size_t)d * NS + q * kLane);
            if (h0) hv = *reinterpret_cast<const float4*>(h0 + (size_t)d * NS + q * kLane);
        }
        const float as[4] = {av.x, av.y, av.z, av.w}, hs[4] = {hv.x, hv.y, hv.z, hv.w};
#pragma unroll
        for (int i = 0; i < kLane; ++i) {
            (c & 1 ? A[c / 2][i].y : A[c / 2][i].x) = as[i] * kLog2e;
            (c & 1 ? h[c / 2][i].y : h[c / 2][i].x) = hs[i];
        }
    }

    // staging: vector lane + 32 j of the tile is row / L::VR, always the same channels
    const int vc = d0 + (lane % L::VR) * kVec, vr = lane / L::VR;
    const bool von = vc < D && (V > 1 || lane < kTile * L::VR);
    const int bc = (lane % (NS / kVec)) * kVec, br = lane / (NS / kVec);
    constexpr int VSTEP = 32 / L::VR, BSTEP = 32 / (NS / kVec);
    const long long row0 = f.row0 + f.first;
    const T* u = static_cast<const T*>(a.u) + row0 * a.ldu + vc;
    const T* dt = static_cast<const T*>(a.dt) + row0 * a.lddt + vc;
    const T* z = static_cast<const T*>(a.z) + (a.z ? row0 * a.ldz + vc : 0);
    const T* B = static_cast<const T*>(a.Bm) + row0 * a.ldb + bc;
    const T* C = static_cast<const T*>(a.Cm) + row0 * a.ldc + bc;
    Raw<T> nu[V], nd[V], nb[BV], nc[BV];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int t = t0 + vr + j * VSTEP;
            if (von && t < f.len) {
                nu[j].load(u + t * a.ldu);
                nd[j].load(dt + t * a.lddt);
            } else {
                nu[j].zero();
                nd[j].zero();
            }
        }
#pragma unroll
        for (int j = 0; j < BV; ++j) {
            const int t = t0 + br + j * BSTEP;
            if (br + j * BSTEP < kTile && t < f.len) {
                nb[j].load(B + t * a.ldb);
                if (kFinal) nc[j].load(C + t * a.ldc);
            }
        }
    };
    fetch(0);
    float total[kVec] = {};
    for (int t0 = 0; t0 < f.len; t0 += kTile) {
        const int len = min(kTile, f.len - t0);
        Raw<T> cu[V], cz[V];
        float bias[kVec] = {};
        if (von && a.dt_bias) load8(a.dt_bias + vc, bias);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int r = vr + j * VSTEP;
            cu[j] = nu[j];
            if (kFinal && a.z && von && r < len) cz[j].load(z + (t0 + r) * a.ldz);
            float x[kVec], s[kVec];
            nu[j].get(x);
            nd[j].get(s);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                s[e] = softplus(s[e] + bias[e]);
                x[e] *= s[e];
                if (!kFinal && von && r < len) total[e] += s[e];
            }
            if (V > 1 || lane < kTile * L::VR) {
                store8(sd + r * LD + (vc - d0), s);
                store8(su + r * LD + (vc - d0), x);
            }
        }
#pragma unroll
        for (int j = 0; j < BV; ++j) {
            const int r = br + j * BSTEP;
            if (r < len) {
                float x[kVec];
                nb[j].get(x);
                store8(sb + r * NS + bc, x);
                if (kFinal) {
                    nc[j].get(x);
                    store8(sc + r * NS + bc, x);
                }
            }
        }
        __syncwarp();
        if (t0 + kTile < f.len) fetch(t0 + kTile);
#pragma unroll 4
        for (int t = 0; t < len; ++t) {
            float dv[CPL], uv[CPL];
            if (CPL == 4) {
                *reinterpret_cast<float4*>(dv) = *reinterpret_cast<const float4*>(sd + t * LD + g * CPL);
                *reinterpret_cast<float4*>(uv) = *reinterpret_cast<const float4*>(su + t * LD + g * CPL);
            } else {
                *reinterpret_cast<float2*>(dv) = *reinterpret_cast<const float2*>(sd + t * LD + g * CPL);
                *reinterpret_cast<float2*>(uv) = *reinterpret_cast<const float2*>(su + t * LD + g * CPL);
            }
            const float4 bv = *reinterpret_cast<const float4*>(sb + t * NS + q * kLane);
            const float bs[4] = {bv.x, bv.y, bv.z, bv.w};
            float4 cv = bv;
            if (kFinal) cv = *reinterpret_cast<const float4*>(sc + t * NS + q * kLane);
            const float cs[4] = {cv.x, cv.y, cv.z, cv.w};
            float2 y[P];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const float2 dd = make_float2(dv[2 * p], dv[2 * p + 1]), uu = make_float2(uv[2 * p], uv[2 * p + 1]);
                y[p] = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < kLane; ++i) {
                    const float2 x = mul2(dd, A[p][i]);
                    const float2 e = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                    h[p][i] = fma2(e, h[p][i], mul2(uu, make_float2(bs[i], bs[i])));
                    if (kFinal) y[p] = fma2(make_float2(cs[i], cs[i]), h[p][i], y[p]);
                }
            }
            if (kFinal) {
                // the lanes of a channel add up their states; lane q keeps channel q mod CPL
                float v[CPL];
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    v[2 * p] = y[p].x;
                    v[2 * p + 1] = y[p].y;
                }
                int m = LPC / 2;
#pragma unroll
                for (int half = CPL / 2; half > 0; half /= 2) {
                    if (m == 0) break;
                    const bool up = (q & m) != 0;
#pragma unroll
                    for (int c = 0; c < half; ++c) {
                        const float keep = up ? v[c + half] : v[c], send = up ? v[c] : v[c + half];
                        v[c] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                    }
                    m /= 2;
                }
                for (; m > 0; m /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
                if (LPC >= CPL) {
                    // the channel's bits are the highest of q
                    if (q % (LPC / CPL) == 0) sy[t * LD + g * CPL + q / (LPC / CPL)] = v[0];
                } else {
                    sy[t * LD + g * CPL + q] = v[0];
                }
            }
        }
        __syncwarp();
        if (kFinal) {
            float skip[kVec] = {};
            if (von && a.skip) load8(a.skip + vc, skip);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int r = vr + j * VSTEP;
                if (!von || r >= len) continue;
                float y[kVec], x[kVec];
                load8(sy + r * LD + (vc - d0), y);
                cu[j].get(x);
#pragma unroll
                for (int e = 0; e < kVec; ++e) y[e] = fmaf(skip[e], x[e], y[e]);
                if (a.z) {
                    cz[j].get(x);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) y[e] *= x[e] * sigmoidf_(x[e]);
                }
                store8(static_cast<T*>(a.o) + (row0 + t0 + r) * D + vc, y);
            }
            __syncwarp();
        }
    }
    float* to = kFinal ? (a.h && f.s == max(f.segs, 1) - 1 ? a.h + (size_t)f.b * D * NS : nullptr)
                       : local + (size_t)blockIdx.x * D * NS;
    if (to) {
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            const int d = d0 + g * CPL + c;
            float o[4];
#pragma unroll
            for (int i = 0; i < kLane; ++i) o[i] = c & 1 ? h[c / 2][i].y : h[c / 2][i].x;
            if (d < D) *reinterpret_cast<float4*>(to + (size_t)d * NS + q * kLane) = make_float4(o[0], o[1], o[2], o[3]);
        }
    }
    if (!kFinal) {
        // a channel's vectors lie in the lanes VR apart
#pragma unroll
        for (int m = L::VR; m < 32; m *= 2)
#pragma unroll
            for (int e = 0; e < kVec; ++e) total[e] += __shfl_xor_sync(0xffffffffu, total[e], m);
        if (lane < L::VR && vc < D) store8(steps + (size_t)blockIdx.x * D + vc, total);
    }
}

// The state before every segment but the first, from the local ones:
// h <- exp(A sum of the segment's steps) h + local, over local in place.
template <int NS>
__global__ void __launch_bounds__(128) fold_kernel(const ScanArgs a, float* local, const float* steps) {
    const int i = blockIdx.y * 128 + threadIdx.x, b = blockIdx.x;
    if (i >= a.D * (NS / 4)) return;
    const int d = i / (NS / 4), q = i % (NS / 4) * 4;
    int len = a.rows.N;
    if (a.rows.cu) {
        int row0;
        packed_range(a.rows.cu, b, a.rows.total, row0, len);
        len = min(len, a.rows.N);
    }
    const int cuts = (len + a.rows.seg - 1) / a.rows.seg - 1;
    if (cuts <= 0) return;
    const long long slot = slot_start(a.rows, b);
    float4 A = *reinterpret_cast<const float4*>(a.A + (size_t)d * NS + q);
    A = make_float4(A.x * kLog2e, A.y * kLog2e, A.z * kLog2e, A.w * kLog2e);
    float4 h = a.h0 ? *reinterpret_cast<const float4*>(a.h0 + ((size_t)b * a.D + d) * NS + q)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
    float* l = local + ((size_t)slot * a.D + d) * NS + q;
    const float* s = steps + (size_t)slot * a.D + d;
    constexpr int U = 8;
    for (int k = 0; k < cuts; k += U) {
        float4 v[U];
        float w[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (k + j < cuts) {
                v[j] = *reinterpret_cast<const float4*>(l + (size_t)(k + j) * a.D * NS);
                w[j] = s[(size_t)(k + j) * a.D];
            }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (k + j < cuts) {
                h.x = fmaf(exp2_approx(w[j] * A.x), h.x, v[j].x);
                h.y = fmaf(exp2_approx(w[j] * A.y), h.y, v[j].y);
                h.z = fmaf(exp2_approx(w[j] * A.z), h.z, v[j].z);
                h.w = fmaf(exp2_approx(w[j] * A.w), h.w, v[j].w);
                *reinterpret_cast<float4*>(l + (size_t)(k + j) * a.D * NS) = h;
            }
    }
}

// Tokens of a segment: the whole sequence where the channels of all sequences
// give the GPU enough warps, else as many cuts as fill it (each cut token is
// scanned twice).
int segment(int B, int N, int total, int D, int n, bool packed, int num_sms) {
    const int width = n <= 16 ? 32 : n == 32 ? 16 : 8;
    const long long tokens = packed ? total : (long long)B * N;
    const long long per_seq = ((long long)D + width - 1) / width;
    const long long want = 12LL * num_sms;
    const long long have = per_seq * B;
    if (!packed && have >= want / 2) return N;
    long long seg = (tokens * per_seq + want - 1) / want;
    seg = (seg + kTile - 1) / kTile * kTile;
    if (seg < 4 * kTile) seg = 4 * kTile;
    return seg >= N ? N : (int)seg;
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
cudaError_t scan(ScanArgs a, int num_sms, cudaStream_t s) {
    a.rows.seg = segment(a.rows.B, a.rows.N, a.rows.total, a.D, NS, a.rows.cu != nullptr, num_sms);
    const long long slots = slots_of(a.rows);
    const dim3 grid((unsigned)slots, (a.D + kWarps * Layout<NS>::W - 1) / (kWarps * Layout<NS>::W));
    float* local = static_cast<float*>(a.workspace);
    float* steps = local + (size_t)slots * a.D * NS;
    if (a.rows.seg < a.rows.N) {
        selective_scan_kernel<T, NS, false><<<grid, kWarps * 32, 0, s>>>(a, local, steps);
        fold_kernel<NS><<<dim3(a.rows.B, (a.D * (NS / 4) + 127) / 128), 128, 0, s>>>(a, local, steps);
    }
    selective_scan_kernel<T, NS, true><<<grid, kWarps * 32, 0, s>>>(a, local, steps);
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

size_t selective_scan_ws_bytes(int B, int N, int total, int D, int n, bool packed, int num_sms) {
    Rows r = {nullptr, B, N, total, segment(B, N, total, D, n, packed, num_sms)};
    if (r.seg >= N) return 0;
    const long long slots = packed ? (long long)total / r.seg + B : slots_of(r);
    return align256((size_t)slots * D * (n + 1) * sizeof(float));
}

cudaError_t launch_selective_scan(ScanArgs a, int num_sms, cudaStream_t s) {
    const bool bf = a.io == GRET_BF16;
    switch (a.n) {
        case 8: return bf ? scan<__nv_bfloat16, 8>(a, num_sms, s) : scan<float, 8>(a, num_sms, s);
        case 16: return bf ? scan<__nv_bfloat16, 16>(a, num_sms, s) : scan<float, 16>(a, num_sms, s);
        case 32: return bf ? scan<__nv_bfloat16, 32>(a, num_sms, s) : scan<float, 32>(a, num_sms, s);
        default: return bf ? scan<__nv_bfloat16, 64>(a, num_sms, s) : scan<float, 64>(a, num_sms, s);
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
