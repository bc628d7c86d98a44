// Gradients of the selective scan.  With g[t,d,i] the gradient of the state,
//
//   y = C.h + skip u,  dz = do y swish'(z),  dy = do swish(z)
//   g[t] = C[t] dy[t] + a[t+1] g[t+1],  a[t] = exp(delta[t] A),  g past the end = dh_final
//   dC[t,i] = sum_d h dy,  dB[t,i] = sum_d g delta u,  s = sum_i g B
//   du = skip dy + delta s,  ddelta = sum_i A g a h[t-1] + u s,  ddt = ddelta sigmoid(dt + dt_bias)
//   dA = sum_t delta g a h[t-1],  dskip = sum_t dy u,  ddt_bias = sum_t ddt,  dh0 = a[0] g[0]
//
// Both recurrences are linear, so the sequence is cut into short segments that
// are independent but for two states each:
//
//   ends     per segment, walked once: the state it leaves from zero, what it
//            hands back from a zero gradient past its end (sum of P C dy, P the
//            product of the decays up to t), and the sum of its steps
//   fold     per channel and state, forwards and backwards over the segments:
//            the state before each and the gradient carried into each
//   walk     per segment: a sweep keeps the state before every group of
//            kGroup tokens in shared memory; then group by group from the last,
//            the group's states and decays are formed again in registers and
//            the group is walked in reverse
//   join     dB, dC: the channel blocks' shares; the parameters' sums over the segments
//
// A sequence of one segment is walked alone, from h0 and dh_final.
//
// Three exponentials per state and token, all of them parallel over the tokens.
// 4 x 4096 tokens x 2048 channels x 16 states, bf16: 958 us, of them ends 200,
// fold 55, walk 670, join 36.  The walk issues 217 instructions per token and 16
// channels; no unit is full (60 % of the issue slots, 67 % of the shared memory's
// cycles), as 12 warps an SM hide too little; more blocks an SM, at 128 registers
// and 28 tokens a segment, took 1063 us, and blocks of two, three or eight warps
// 1015 to 1155.  With 8, 32, 64 states it takes 650, 1866, 4556 us (in fp32 828,
// 2034, 4806; 1062 with 16): at 64 states a segment is 16 tokens, whose states,
// gradients and shares alone are 2.2 GB written and read, and 8 warps fit an SM.
// The workspace, for 4 x 4096 tokens x 4096 channels and 8, 16, 32, 64 states, is
// 0.26, 0.56, 1.4 and 4.4 GB.
#include "gret_selective.cuh"

namespace gret {
namespace {

template <int NS>
struct Layout {
    static constexpr int SPL = NS == 64 ? 8 : 4;            // states of a lane
    static constexpr int LPC = NS / SPL;                    // lanes of a channel
    static constexpr int W = 32 / LPC * kPair;              // channels of a warp: 32, 16, 8, 8
    static constexpr int GROUP = NS == 64 ? 2 : 4;          // tokens walked in registers
    static constexpr int SEG = NS == 64 ? 16 : 32;          // tokens of a segment
    static constexpr int LD = 2 * W + 4, LY = W + 4;        // shared rows: 16-byte steps over the banks
    static constexpr int VR = W / kVec;                     // 16-byte vectors of a row
    static constexpr int V = (SEG * VR + 31) / 32;          // and of a lane
    static constexpr int START = 32 * kPair * SPL;          // floats of a group's start
    static constexpr int ROWS = SEG * (LD + LY);            // floats a warp stages
    static constexpr int WARP = ROWS + SEG / GROUP * START;
    static constexpr int BC = 2 * SEG * NS;                 // B and C of the segment
    static constexpr int W4 = kScanWarps * W;               // channels of a block
    static_assert(GROUP * 2 * NS <= START, "a group's dB and dC go where its start was");
};

struct Work {
    float *h, *g, *steps;   // [slots][D][n], [slots][D][n], [slots][D]
    float *bc;              // [channel blocks][rows][2 n]
    float *partial;         // [slots][D (n + 2)]
};

// Stage the segment: (delta, delta, delta u, delta u) of each two channels and
// dy, of this warp's channels; B and C for the block.  Rows past the end are
// steps of nothing.  Adds the steps to `total`.
template <typename T, int NS>
__device__ __forceinline__ void stage(const ScanBackwardArgs& g, const Slot& f, int d0, float* sd, float* sy, float* sbc,
                                      float* total) {
    using L = Layout<NS>;
    const ScanArgs& a = g.f;
    const int lane = threadIdx.x & 31;
    const long long row0 = f.row0 + f.first;
    for (int i = threadIdx.x; i < 2 * L::SEG * NS / kVec; i += kScanWarps * 32) {
        const int which = i / (L::SEG * NS / kVec), j = i % (L::SEG * NS / kVec), r = j / (NS / kVec),
                  c = j % (NS / kVec) * kVec;
        float x[kVec] = {};
        if (r < f.len)
            load8(which ? static_cast<const T*>(a.Cm) + (row0 + r) * a.ldc + c
                        : static_cast<const T*>(a.Bm) + (row0 + r) * a.ldb + c, x);
        store8(sbc + which * L::SEG * NS + r * NS + c, x);
    }
    const int vc = d0 + lane % L::VR * kVec;
    if (d0 < a.D) {
        float bias[kVec] = {};
        if (vc < a.D && a.dt_bias) load8(a.dt_bias + vc, bias);
        Raw<T> ru[L::V], rt[L::V], rg[L::V], rz[L::V];
#pragma unroll
        for (int j = 0; j < L::V; ++j) {
            const int r = lane / L::VR + j * (32 / L::VR);
            if (vc >= a.D || r >= f.len) continue;
            const long long row = row0 + r;
            rt[j].load(static_cast<const T*>(a.dt) + row * a.lddt + vc);
            ru[j].load(static_cast<const T*>(a.u) + row * a.ldu + vc);
            rg[j].load(static_cast<const T*>(g.dout) + row * a.D + vc);
            if (a.z) rz[j].load(static_cast<const T*>(a.z) + row * a.ldz + vc);
        }
#pragma unroll
        for (int j = 0; j < L::V; ++j) {
            const int r = lane / L::VR + j * (32 / L::VR);
            if (r >= L::SEG) continue;
            float u[kVec] = {}, s[kVec] = {}, dy[kVec] = {};
            if (vc < a.D && r < f.len) {
                rt[j].get(s);
                ru[j].get(u);
                rg[j].get(dy);
                if (a.z) {
                    float z[kVec];
                    rz[j].get(z);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) dy[e] *= z[e] * sigmoid_fast(z[e]);
                }
#pragma unroll
                for (int e = 0; e < kVec; e += 2) {
                    const float2 d = softplus2(make_float2(s[e] + bias[e], s[e + 1] + bias[e + 1]));
                    s[e] = d.x;
                    s[e + 1] = d.y;
                    u[e] *= d.x;
                    u[e + 1] *= d.y;
                    total[e] += d.x;
                    total[e + 1] += d.y;
                }
            }
            float* to = sd + r * L::LD + 2 * (vc - d0);
#pragma unroll
            for (int e = 0; e < kVec; e += 2)
                *reinterpret_cast<float4*>(to + 2 * e) = make_float4(s[e], s[e + 1], u[e], u[e + 1]);
            store8(sy + r * L::LY + (vc - d0), dy);
        }
    }
    __syncthreads();
}

// Eight channels' sums over the lanes that hold other rows of them.
template <int VR>
__device__ __forceinline__ void sum_rows(float* v) {
#pragma unroll
    for (int m = VR; m < 32; m *= 2)
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], m);
}

template <int H>
__device__ __forceinline__ void read_states(float2* v, const float* row) {
#pragma unroll
    for (int i = 0; i < H; i += 2) {
        const float4 x = *reinterpret_cast<const float4*>(row + 2 * i);
        v[i] = make_float2(x.x, x.y);
        v[i + 1] = make_float2(x.z, x.w);
    }
}

__device__ __forceinline__ float2 exp2_pair(float2 x) { return make_float2(exp2_approx(x.x), exp2_approx(x.y)); }

template <typename T, int NS>
__global__ void __launch_bounds__(kScanWarps * 32, 4) ends_kernel(const ScanBackwardArgs g, const Work w) {
    using L = Layout<NS>;
    constexpr int SPL = L::SPL, H = SPL / 2;
    extern __shared__ __align__(16) float shared[];
    const ScanArgs& a = g.f;
    const Slot f = find_slot(a.rows, blockIdx.x);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = a.D;
    const int d0 = blockIdx.y * L::W4 + warp * L::W;
    float *sbc = shared, *sd = shared + L::BC + warp * L::ROWS, *sy = sd + L::SEG * L::LD;
    float total[kVec] = {};
    stage<T, NS>(g, f, d0, sd, sy, sbc, total);
    if (d0 >= D) return;
    sum_rows<L::VR>(total);
    if (lane < L::VR && d0 + lane * kVec < D) store8(w.steps + (size_t)blockIdx.x * D + d0 + lane * kVec, total);

    const int q = lane % L::LPC, cg = lane / L::LPC, d = d0 + cg * kPair;
    float2 A[kPair][H], h[kPair][H], back[kPair][H], P[kPair][H];
    load_states<SPL>(A, a.A, NS, q, d, D);
#pragma unroll
    for (int c = 0; c < kPair; ++c)
#pragma unroll
        for (int i = 0; i < H; ++i) {
            A[c][i] = log2_rate(A[c][i]);
            h[c][i] = back[c][i] = both(0.f);
            P[c][i] = both(1.f);
        }
    const float *B = sbc + q * SPL, *C = B + L::SEG * NS;
#pragma unroll 4
    for (int t = 0; t < L::SEG; ++t) {
        const float4 du = *reinterpret_cast<const float4*>(sd + t * L::LD + cg * 4);
        const float2 dy = *reinterpret_cast<const float2*>(sy + t * L::LY + cg * 2);
        float2 b[H], cs[H];
        read_states<H>(b, B + t * NS);
        read_states<H>(cs, C + t * NS);
#pragma unroll
        for (int c = 0; c < kPair; ++c) {
            const float2 dd = both(c ? du.y : du.x), uu = both(c ? du.w : du.z), yy = both(c ? dy.y : dy.x);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float2 e = exp2_pair(mul2(dd, A[c][i]));
                h[c][i] = fma2(e, h[c][i], mul2(uu, b[i]));
                P[c][i] = mul2(P[c][i], e);
                back[c][i] = fma2(P[c][i], mul2(yy, cs[i]), back[c][i]);
            }
        }
    }
    const size_t state = (size_t)blockIdx.x * D * NS;
    store_states<SPL>(w.h + state, h, NS, q, d, D);
    store_states<SPL>(w.g + state, back, NS, q, d, D);
}

// h: the state before each segment; g: the gradient carried into its last token
// from behind; both over the segments' own, in place.
template <int NS, int Y>
__global__ void __launch_bounds__(kFoldThreads) fold_kernel(const ScanBackwardArgs g, const Work w, int segs) {
    __shared__ FoldShared<Y> shared;
    const ScanArgs& a = g.f;
    const int blocks = fold_blocks<Y>(a.D, NS), b = blockIdx.x / blocks;
    const int i = (blockIdx.x - b * blocks) * kFoldX<Y> + threadIdx.x;
    const bool on = i < a.D * (NS / 4);
    const int d = on ? i / (NS / 4) : 0, q = on ? i % (NS / 4) * 4 : 0;
    const long long stride = (long long)a.D * NS, first = (long long)b * segs, last = first + segs - 1;
    const size_t own = ((size_t)b * a.D + d) * NS + q, at = (size_t)d * NS + q;
    const float4 A = *reinterpret_cast<const float4*>(a.A + at), none = make_float4(0.f, 0.f, 0.f, 0.f);
    fold_segments<false, Y>(shared, on, w.h + first * stride + at, stride, w.steps + first * a.D + d, a.D, segs, A,
                         a.h0 ? *reinterpret_cast<const float4*>(a.h0 + own) : none);
    const float4 x = fold_segments<false, Y>(shared, on, w.g + last * stride + at, -stride, w.steps + last * a.D + d, -a.D,
                                          segs, A, g.dh_final ? *reinterpret_cast<const float4*>(g.dh_final + own) : none);
    if (g.dh0 && on && threadIdx.y == 0) *reinterpret_cast<float4*>(g.dh0 + own) = x;
}

template <typename T, int NS>
__global__ void __launch_bounds__(kScanWarps * 32, NS == 64 ? 2 : 3) walk_kernel(const ScanBackwardArgs g, const Work w,
                                                                                          bool alone) {
    using L = Layout<NS>;
    constexpr int SPL = L::SPL, H = SPL / 2, G = L::GROUP, LPC = L::LPC, W = L::W;
    extern __shared__ __align__(16) float shared[];
    const ScanArgs& a = g.f;
    const Slot f = find_slot(a.rows, blockIdx.x);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = a.D;
    const int d0 = blockIdx.y * L::W4 + warp * W;
    float *sbc = shared, *sd = shared + L::BC + warp * L::WARP, *sy = sd + L::SEG * L::LD, *starts = sd + L::ROWS;
    const long long row0 = f.row0 + f.first;
    const int groups = (f.len + G - 1) / G;
    const int q = lane % LPC, cg = lane / LPC, d = d0 + cg * kPair;
    const size_t state = (size_t)blockIdx.x * D * NS;
    float2 A[kPair][H], dA[kPair][H], carry[kPair][H], first[kPair][H];
    load_states<SPL>(A, a.A, NS, q, d, D);
    const size_t whole = (size_t)f.b * D * NS;              // of the sequence, when it is one segment
    load_states<SPL>(first, !alone ? w.h + state : a.h0 ? a.h0 + whole : nullptr, NS, q, d, D);
    load_states<SPL>(carry, !alone ? w.g + state : g.dh_final ? g.dh_final + whole : nullptr, NS, q, d, D);
    {
        float total[kVec] = {};
        stage<T, NS>(g, f, d0, sd, sy, sbc, total);
    }
    if (d0 < D) {
        const float *B = sbc + q * SPL, *C = B + L::SEG * NS;
#pragma unroll
        for (int c = 0; c < kPair; ++c)
#pragma unroll
            for (int i = 0; i < H; ++i) {
                A[c][i] = log2_rate(A[c][i]);
                dA[c][i] = both(0.f);
            }
        // the state before every group
        {
            float2 (&h)[kPair][H] = first;
#pragma unroll 2
            for (int k = 0; k < groups; ++k) {
                float4* to = reinterpret_cast<float4*>(starts + k * L::START) + lane;
#pragma unroll
                for (int c = 0; c < kPair; ++c)
#pragma unroll
                    for (int i = 0; i < H; i += 2)
                        to[(c * H + i) / 2 * 32] = make_float4(h[c][i].x, h[c][i].y, h[c][i + 1].x, h[c][i + 1].y);
                if (k + 1 == groups) break;
#pragma unroll
                for (int t = k * G; t < (k + 1) * G; ++t) {
                    const float4 du = *reinterpret_cast<const float4*>(sd + t * L::LD + cg * 4);
                    float2 b[H];
                    read_states<H>(b, B + t * NS);
#pragma unroll
                    for (int c = 0; c < kPair; ++c) {
                        const float2 dd = both(c ? du.y : du.x), uu = both(c ? du.w : du.z);
#pragma unroll
                        for (int i = 0; i < H; ++i)
                            h[c][i] = fma2(exp2_pair(mul2(dd, A[c][i])), h[c][i], mul2(uu, b[i]));
                    }
                }
            }
        }
        for (int k = groups - 1; k >= 0; --k) {
            // the group's states and decays
            float2 h[G + 1][kPair][H], e[G][kPair][H];
            const float4* from = reinterpret_cast<const float4*>(starts + k * L::START) + lane;
#pragma unroll
            for (int c = 0; c < kPair; ++c)
#pragma unroll
                for (int i = 0; i < H; i += 2) {
                    const float4 x = from[(c * H + i) / 2 * 32];
                    h[0][c][i] = make_float2(x.x, x.y);
                    h[0][c][i + 1] = make_float2(x.z, x.w);
                }
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const int t = k * G + j;
                const float4 du = *reinterpret_cast<const float4*>(sd + t * L::LD + cg * 4);
                float2 b[H];
                read_states<H>(b, B + t * NS);
#pragma unroll
                for (int c = 0; c < kPair; ++c) {
                    const float2 dd = both(c ? du.y : du.x), uu = both(c ? du.w : du.z);
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        e[j][c][i] = exp2_pair(mul2(dd, A[c][i]));
                        h[j + 1][c][i] = fma2(e[j][c][i], h[j][c][i], mul2(uu, b[i]));
                    }
                }
            }
            // and the way back; sums[token][channel]: y, sum of A g a h[t-1] (in log2 units), sum of g B
            float sums[G * kPair * 3];
            constexpr int kLeft = parts_left<2 * SPL, 16, LPC>();  // of the lane's dB and dC values of a token
            float left[G][kLeft];
#pragma unroll
            for (int j = G - 1; j >= 0; --j) {
                const int t = k * G + j;
                const float4 du = *reinterpret_cast<const float4*>(sd + t * L::LD + cg * 4);
                const float2 dy = *reinterpret_cast<const float2*>(sy + t * L::LY + cg * 2);
                float2 b[H], cs[H], bc[2 * H];
                read_states<H>(b, B + t * NS);
                read_states<H>(cs, C + t * NS);
#pragma unroll
                for (int c = 0; c < kPair; ++c) {
                    const float2 dd = both(c ? du.y : du.x), uu = both(c ? du.w : du.z), yy = both(c ? dy.y : dy.x);
                    float2 y, sa, sb;
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const float2 gr = fma2(cs[i], yy, carry[c][i]);
                        y = i ? fma2(cs[i], h[j + 1][c][i], y) : mul2(cs[i], h[j + 1][c][i]);
                        sb = i ? fma2(gr, b[i], sb) : mul2(gr, b[i]);
                        bc[i] = c ? fma2(gr, uu, bc[i]) : mul2(gr, uu);
                        bc[H + i] = c ? fma2(h[j + 1][c][i], yy, bc[H + i]) : mul2(h[j + 1][c][i], yy);
                        carry[c][i] = mul2(gr, e[j][c][i]);
                        const float2 through = mul2(carry[c][i], h[j][c][i]);
                        sa = i ? fma2(through, A[c][i], sa) : mul2(through, A[c][i]);
                        dA[c][i] = fma2(through, dd, dA[c][i]);
                    }
                    float* s = sums + (j * kPair + c) * 3;
                    s[0] = y.x + y.y;
                    s[1] = sa.x + sa.y;
                    s[2] = sb.x + sb.y;
                }
                // dB, dC of the warp's channels: over the lanes of other channels
                float v[2 * SPL];
#pragma unroll
                for (int i = 0; i < 2 * H; ++i) {
                    v[2 * i] = bc[i].x;
                    v[2 * i + 1] = bc[i].y;
                }
                add_parts<2 * SPL, 16, LPC>(v, lane);
#pragma unroll
                for (int i = 0; i < kLeft; ++i) left[j][i] = v[i];
            }
            add_parts<G * kPair * 3, LPC / 2, 1>(sums, lane);
            constexpr int R = parts_left<G * kPair * 3, LPC / 2, 1>();
            constexpr int TWINS = LPC * R / (G * kPair * 3);
            static_assert(R % 3 == 0, "whole channels");
            __syncwarp();
            {
                // dB, dC where the group's start was
                constexpr int HOLDERS = 32 / LPC, SAME = HOLDERS * kLeft / (2 * SPL);
                const int at = cg / SAME * kLeft;
                float* to = starts + k * L::START + (at / SPL) * NS + q * SPL + at % SPL;
                if (cg % SAME == 0)
#pragma unroll
                    for (int j = 0; j < G; ++j)
#pragma unroll
                        for (int i = 0; i < kLeft; ++i) to[j * 2 * NS + i] = left[j][i];
            }
            if (q % TWINS == 0) {
                // where the tokens' delta u and dy were: A g a h[t-1], g B, y
#pragma unroll
                for (int i = 0; i < R / 3; ++i) {
                    const int item = q / TWINS * (R / 3) + i, t = k * G + item / kPair, c = item % kPair;
                    sd[t * L::LD + cg * 4 + c] = sums[3 * i + 1];
                    sd[t * L::LD + cg * 4 + 2 + c] = sums[3 * i + 2];
                    sy[t * L::LY + cg * 2 + c] = sums[3 * i];
                }
            }
        }
        __syncwarp();
        if (alone && g.dh0) store_states<SPL>(g.dh0 + whole, carry, NS, q, d, D);
        float* partial = w.partial + (size_t)blockIdx.x * D * (NS + 2);
        store_states<SPL>(partial, dA, NS, q, d, D);

        const int vc = d0 + lane % L::VR * kVec;
        float bias[kVec] = {}, skip[kVec] = {}, dskip[kVec] = {}, dbias[kVec] = {};
        if (vc < D && a.dt_bias) load8(a.dt_bias + vc, bias);
        if (vc < D && a.skip) load8(a.skip + vc, skip);
        Raw<T> ru[L::V], rt[L::V], rg[L::V], rz[L::V];
#pragma unroll
        for (int j = 0; j < L::V; ++j) {
            const int r = lane / L::VR + j * (32 / L::VR);
            if (vc >= D || r >= f.len) continue;
            const long long row = row0 + r;
            ru[j].load(static_cast<const T*>(a.u) + row * a.ldu + vc);
            rt[j].load(static_cast<const T*>(a.dt) + row * a.lddt + vc);
            rg[j].load(static_cast<const T*>(g.dout) + row * D + vc);
            if (a.z) rz[j].load(static_cast<const T*>(a.z) + row * a.ldz + vc);
        }
#pragma unroll
        for (int j = 0; j < L::V; ++j) {
            const int r = lane / L::VR + j * (32 / L::VR);
            if (vc >= D || r >= f.len) continue;
            const long long row = row0 + r;
            float u[kVec], raw[kVec], up[kVec], z[kVec], y[kVec], du[kVec], ddt[kVec], dz[kVec];
            ru[j].get(u);
            rt[j].get(raw);
            rg[j].get(up);
            if (a.z) rz[j].get(z);
            load8(sy + r * L::LY + (vc - d0), y);
            const float* s = sd + r * L::LD + 2 * (vc - d0);
#pragma unroll
            for (int e = 0; e < kVec; e += 2) {
                const float4 ab = *reinterpret_cast<const float4*>(s + 2 * e);
                const float sa[2] = {ab.x, ab.y}, sb[2] = {ab.z, ab.w};
                raw[e] += bias[e];
                raw[e + 1] += bias[e + 1];
                const float2 dl = softplus2(make_float2(raw[e], raw[e + 1]));
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const int i = e + o;
                    float dy = up[i];
                    if (a.z) {
                        const float sig = sigmoid_fast(z[i]);
                        dz[i] = up[i] * fmaf(skip[i], u[i], y[i]) * swish_slope(z[i], sig);
                        dy *= z[i] * sig;
                    }
                    ddt[i] = fmaf(u[i], sb[o], sa[o] * 0.6931471805599453f) * sigmoid_fast(raw[i]);
                    du[i] = fmaf(o ? dl.y : dl.x, sb[o], skip[i] * dy);
                    dskip[i] = fmaf(dy, u[i], dskip[i]);
                    dbias[i] += ddt[i];
                }
            }
            store8(static_cast<T*>(g.du) + row * D + vc, du);
            store8(static_cast<T*>(g.ddt) + row * D + vc, ddt);
            if (a.z) store8(static_cast<T*>(g.dz) + row * D + vc, dz);
        }
        sum_rows<L::VR>(dskip);
        sum_rows<L::VR>(dbias);
        if (lane < L::VR && vc < D) {
            store8(partial + (size_t)D * NS + vc, dskip);
            store8(partial + (size_t)D * (NS + 1) + vc, dbias);
        }
    }
    __syncthreads();
    // the block's share of dB and dC
    const int warps = min(kScanWarps, (D - (int)blockIdx.y * L::W4 + W - 1) / W);
    float* bc = w.bc + ((size_t)blockIdx.y * a.rows.B * a.rows.N + row0) * 2 * NS;
    for (int i = threadIdx.x; i < f.len * 2 * NS; i += kScanWarps * 32) {
        const int t = i / (2 * NS);
        const float* from = shared + L::BC + L::ROWS + t / G * L::START + t % G * 2 * NS + i % (2 * NS);
        float s = 0.f;
        for (int k = 0; k < warps; ++k) s += from[k * L::WARP];
        bc[i] = s;
    }
}

// dB, dC: the channel blocks' shares, added in order, in the launch's first
// `joins` blocks; the parameters' gradients, over the segments, in the others.
template <typename T>
__global__ void __launch_bounds__(kSumThreads) join_kernel(const float* bc, int blocks, long long rows, int n, T* dB, T* dC,
                                                           long long joins, const float* partial, int groups,
                                                           ColumnOutputs out, int width) {
    if (blockIdx.x >= joins) return column_sums(partial, groups, out, width, blockIdx.x - joins);
    const long long i = ((long long)blockIdx.x * kSumThreads + threadIdx.x) * 4, all = rows * 2 * n;
    if (i >= all) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < blocks; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(bc + k * all + i);
        s.x += x.x;
        s.y += x.y;
        s.z += x.z;
        s.w += x.w;
    }
    const long long row = i / (2 * n);
    const int j = (int)(i - row * 2 * n);
    T* to = j < n ? dB + row * n + j : dC + row * n + j - n;
    to[0] = from_f32<T>(s.x);
    to[1] = from_f32<T>(s.y);
    to[2] = from_f32<T>(s.z);
    to[3] = from_f32<T>(s.w);
}

// Tokens of a segment and channels of a block for n states.
struct Cut {
    int seg, channels;
};
Cut cut_of(int n) {
    switch (n) {
        case 8: return {Layout<8>::SEG, Layout<8>::W4};
        case 16: return {Layout<16>::SEG, Layout<16>::W4};
        case 32: return {Layout<32>::SEG, Layout<32>::W4};
        default: return {Layout<64>::SEG, Layout<64>::W4};
    }
}

// Offsets of the workspace's parts, in bytes, and its size.
struct Parts {
    size_t g, steps, bc, partial, all;
};
Parts parts_of(int B, int N, int D, int n) {
    const Cut c = cut_of(n);
    const size_t slots = (size_t)B * segments_of(N, c.seg), blocks = (D + c.channels - 1) / c.channels;
    Parts p;
    p.g = align256(slots * D * n * 4);
    p.steps = 2 * p.g;
    p.bc = p.steps + align256(slots * D * 4);
    p.partial = p.bc + align256(blocks * B * N * 2 * n * 4);
    p.all = p.partial + align256(slots * D * (n + 2) * 4);
    return p;
}

template <int NS, int Y>
void launch_fold(const ScanBackwardArgs& g, const Work& w, int segs, cudaStream_t s) {
    fold_kernel<NS, Y><<<g.f.rows.B * fold_blocks<Y>(g.f.D, NS), dim3(kFoldX<Y>, Y), 0, s>>>(g, w, segs);
}

template <typename T, int NS>
cudaError_t backward(ScanBackwardArgs g, cudaStream_t s) {
    using L = Layout<NS>;
    ScanArgs& a = g.f;
    a.rows.seg = L::SEG;
    const Parts p = parts_of(a.rows.B, a.rows.N, a.D, NS);
    char* ws = static_cast<char*>(g.workspace);
    const Work w = {reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + p.g), reinterpret_cast<float*>(ws + p.steps),
                    reinterpret_cast<float*>(ws + p.bc), reinterpret_cast<float*>(ws + p.partial)};
    const long long slots = slots_of(a.rows), D = a.D, rows = (long long)a.rows.B * a.rows.N;
    const dim3 grid((unsigned)slots, (a.D + L::W4 - 1) / L::W4);
    const int ends_bytes = (L::BC + kScanWarps * L::ROWS) * 4, walk_bytes = (L::BC + kScanWarps * L::WARP) * 4;
    cudaError_t err = cudaFuncSetAttribute(ends_kernel<T, NS>, cudaFuncAttributeMaxDynamicSharedMemorySize, ends_bytes);
    if (err == cudaSuccess)
        err = cudaFuncSetAttribute(walk_kernel<T, NS>, cudaFuncAttributeMaxDynamicSharedMemorySize, walk_bytes);
    if (err != cudaSuccess) return err;
    const int segs = (int)(slots / a.rows.B);
    if (segs > 1) {
        ends_kernel<T, NS><<<grid, kScanWarps * 32, ends_bytes, s>>>(g, w);
        if (segs > kFoldSerial)
            launch_fold<NS, 8>(g, w, segs, s);
        else
            launch_fold<NS, 1>(g, w, segs, s);
    }
    walk_kernel<T, NS><<<grid, kScanWarps * 32, walk_bytes, s>>>(g, w, segs == 1);
    const ColumnOutputs out = {3, {0, D * NS, D * (NS + 1), D * (NS + 2)}, {g.dA, g.dskip, g.ddt_bias}, {1, 1, 1}};
    const long long joins = (rows * 2 * NS / 4 + kSumThreads - 1) / kSumThreads;
    const int width = column_width(out, (int)slots);
    join_kernel<T><<<(unsigned)(joins + column_blocks(out, width)), kSumThreads, 0, s>>>(
        w.bc, grid.y, rows, NS, static_cast<T*>(g.dBm), static_cast<T*>(g.dCm), joins, w.partial, (int)slots, out, width);
    return cudaGetLastError();
}

}  // namespace

size_t selective_backward_ws_bytes(int B, int N, int D, int n) { return parts_of(B, N, D, n).all; }

cudaError_t launch_selective_backward(const ScanBackwardArgs& g, cudaStream_t s) {
    const bool bf = g.f.io == GRET_BF16;
    switch (g.f.n) {
        case 8: return bf ? backward<__nv_bfloat16, 8>(g, s) : backward<float, 8>(g, s);
        case 16: return bf ? backward<__nv_bfloat16, 16>(g, s) : backward<float, 16>(g, s);
        case 32: return bf ? backward<__nv_bfloat16, 32>(g, s) : backward<float, 32>(g, s);
        default: return bf ? backward<__nv_bfloat16, 64>(g, s) : backward<float, 64>(g, s);
    }
}

}  // namespace gret
