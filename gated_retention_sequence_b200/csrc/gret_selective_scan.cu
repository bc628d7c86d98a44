// Selective state space scan: a state of n numbers per channel whose decay and
// input depend on the token.
//
//   delta[t,d] = softplus(dt[t,d] + dt_bias[d])
//   h[t,d,i]   = exp(delta[t,d] A[d,i]) h[t-1,d,i] + delta[t,d] u[t,d] B[t,i]
//   o[t,d]     = (sum_i C[t,i] h[t,d,i] + skip[d] u[t,d]) swish(z[t,d])
//
// B and C are shared by all channels of a token.  One exponential per token,
// channel and state is all but unavoidable, as A is any matrix, and bounds the
// time: at 16 a clock and SM they take 239 us for 16384 tokens x 4096 channels x
// 16 states, whose bytes take 87.  38 packed sequences of that size take 398 us
// (564 in fp32), with the special function unit 72 % busy; evaluating a quarter of
// the powers by a polynomial instead made it slower (379 -> 408 us at 64 x 256 x
// 4096), as the instructions then bound it.  The shared memory's data path comes
// next, hence two channels a lane that share their B and C, and those in their
// own type.
#include <math.h>

#include "gret_selective.cuh"

namespace gret {
namespace {

constexpr int kStepThreads = 128;

// How a warp lays out its channels and states: a lane holds SPL states of two
// channels, n / SPL lanes share a channel, and the warp's W channels are walked
// kTile tokens at a time, kGroup of them between two rounds of shuffles.
constexpr int kTile = 16, kWarps = kScanWarps, kGroup = 4;
template <int NS>
struct Layout {
    static constexpr int SPL = NS >= 32 ? 8 : 4;            // states of a lane
    static constexpr int LPC = NS / SPL;                    // lanes of a channel
    static constexpr int W = 32 / LPC * kPair;              // channels of a warp: 32, 16, 16, 8
    static constexpr int LD = 2 * W + 4, LY = W + 4;        // shared rows: 16-byte steps over the banks
    static constexpr int VR = W / kVec;                     // 16-byte vectors of a row
    static constexpr int V = (kTile * VR + 31) / 32;        // and of a lane
    static constexpr int BV = (kTile * NS / kVec + 31) / 32;    // vectors of B (of C) a lane stages
    static constexpr int FLOATS = kTile * (LD + 2 * NS + LY);   // shared floats of a warp, at most
};

// B and C of a tile in shared memory, in their own type, so that a lane's
// states of both take as few bytes as they can: the shared memory's data path
// is what the scan's warps load most.  A lane's states of B, four at a time,
// are followed by the same of C.
template <typename T> struct Words;
template <> struct Words<__nv_bfloat16> {
    static constexpr int kFour = 2;                         // 32-bit words of four states
    static __device__ __forceinline__ void put(uint32_t* to, const Raw<__nv_bfloat16>& r) {
        *reinterpret_cast<uint2*>(to) = make_uint2(r.a.x, r.a.y);
        *reinterpret_cast<uint2*>(to + 2 * kFour) = make_uint2(r.a.z, r.a.w);
    }
    // the first two pairs of B and C
    static __device__ __forceinline__ void get(const uint32_t* from, float2* b, float2* c) {
        const uint4 v = *reinterpret_cast<const uint4*>(from);
        b[0] = make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
        b[1] = make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
        c[0] = make_float2(__uint_as_float(v.z << 16), __uint_as_float(v.z & 0xffff0000u));
        c[1] = make_float2(__uint_as_float(v.w << 16), __uint_as_float(v.w & 0xffff0000u));
    }
};
template <> struct Words<float> {
    static constexpr int kFour = 4;
    static __device__ __forceinline__ void put(uint32_t* to, const Raw<float>& r) {
        *reinterpret_cast<float4*>(to) = r.a;
        *reinterpret_cast<float4*>(to + 2 * kFour) = r.b;
    }
    static __device__ __forceinline__ void get(const uint32_t* from, float2* b, float2* c) {
        const float4 x = reinterpret_cast<const float4*>(from)[0], y = reinterpret_cast<const float4*>(from)[1];
        b[0] = make_float2(x.x, x.y);
        b[1] = make_float2(x.z, x.w);
        c[0] = make_float2(y.x, y.y);
        c[1] = make_float2(y.z, y.w);
    }
};

// A warp walks one slot's tokens for its channels.  Each tile of tokens is
// staged first (delta and delta u of the warp's channels, B and C), then
// scanned from shared memory, then gated and stored; the next tile's inputs are
// in flight meanwhile.  kFinal: the outputs, from the state before the slot.
// Otherwise the state that the slot alone leaves, from zero, and the sum of its
// steps.  `before`: the state that the slot starts from, or the one `apart`
// segments before it, whose own states and steps follow.  `leave`: where the
// state after the slot goes as well.
template <typename T, int NS, bool kFinal>
__device__ __forceinline__ void walk(const ScanArgs& a, const Slot& f, int block, float* shared, const float* before,
                                     int apart, float* leave, float* steps) {
    using L = Layout<NS>;
    constexpr int SPL = L::SPL, LPC = L::LPC, W = L::W, LD = L::LD, LY = L::LY, V = L::V, BV = L::BV, H = SPL / 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = a.D;
    const int d0 = (block * kWarps + warp) * W;
    if (d0 >= D) return;
    // per token: (delta, delta, delta u, delta u) of each two channels; the sums over the states; B and C
    constexpr int FOUR = Words<T>::kFour, LB = NS / 4 * 2 * FOUR;   // words of B and C for four states, and of a token
    float *sd = shared + warp * L::FLOATS, *sy = sd + kTile * LD;
    uint32_t* sbc = reinterpret_cast<uint32_t*>(sy + kTile * LY);

    const int q = lane % LPC, g = lane / LPC;               // states q SPL .., channels d0 + 2 g ..
    float2 A[kPair][H], h[kPair][H];                        // two states each
    load_states<SPL>(A, a.A, NS, q, d0 + g * kPair, D);
    load_states<SPL>(h, before, NS, q, d0 + g * kPair, D);
#pragma unroll
    for (int c = 0; c < kPair; ++c)
#pragma unroll
        for (int i = 0; i < H; ++i) A[c][i] = log2_rate(A[c][i]);
    if (kFinal) {
#pragma unroll 2
        for (int k = 1; k <= apart; ++k) {
            const int d = d0 + g * kPair;
            float2 own[kPair][H];
            load_states<SPL>(own, before + (size_t)k * D * NS, NS, q, d, D);
            const float2 sum = d < D ? *reinterpret_cast<const float2*>(steps + (size_t)k * D + d) : both(0.f);
#pragma unroll
            for (int c = 0; c < kPair; ++c)
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const float2 x = mul2(both(c ? sum.y : sum.x), A[c][i]);
                    h[c][i] = fma2(make_float2(exp2_approx(x.x), exp2_approx(x.y)), h[c][i], own[c][i]);
                }
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
            } else {
                nb[j].zero();
                nc[j].zero();
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
            for (int e = 0; e < kVec; e += 2) {
                const float2 d = softplus2(make_float2(s[e] + bias[e], s[e + 1] + bias[e + 1]));
                s[e] = d.x;
                s[e + 1] = d.y;
                x[e] *= d.x;
                x[e + 1] *= d.y;
                if (!kFinal && von && r < len) {
                    total[e] += d.x;
                    total[e + 1] += d.y;
                }
            }
            if (r >= len) {                                 // past the end: a step of nothing
#pragma unroll
                for (int e = 0; e < kVec; ++e) s[e] = x[e] = 0.f;
            }
            if (V > 1 || lane < kTile * L::VR) {
                float* to = sd + r * LD + 2 * (vc - d0);
#pragma unroll
                for (int e = 0; e < kVec; e += 2)
                    *reinterpret_cast<float4*>(to + 2 * e) = make_float4(s[e], s[e + 1], x[e], x[e + 1]);
            }
        }
#pragma unroll
        for (int j = 0; j < BV; ++j) {
            const int r = br + j * BSTEP;
            if (r < kTile) {
                uint32_t* to = sbc + r * LB + bc / 4 * 2 * FOUR;
                Words<T>::put(to, nb[j]);
                if (kFinal) Words<T>::put(to + FOUR, nc[j]);
            }
        }
        __syncwarp();
        if (t0 + kTile < f.len) fetch(t0 + kTile);
        for (int t1 = 0; t1 < len; t1 += kGroup) {
            float v[kGroup * kPair];
#pragma unroll
            for (int k = 0; k < kGroup; ++k) {
                const int t = t1 + k;
                const float4 du = *reinterpret_cast<const float4*>(sd + t * LD + g * 4);
                const float dv[2] = {du.x, du.y}, uv[2] = {du.z, du.w};
                float2 bs[H], cs[H], y[kPair];
#pragma unroll
                for (int i = 0; i < H; i += 2) Words<T>::get(sbc + t * LB + (q * SPL / 4 + i / 2) * 2 * FOUR, bs + i, cs + i);
#pragma unroll
                for (int c = 0; c < kPair; ++c) {
                    const float2 dd = both(dv[c]), uu = both(uv[c]);
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const float2 x = mul2(dd, A[c][i]);
                        const float2 e = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                        h[c][i] = fma2(e, h[c][i], mul2(uu, bs[i]));
                        if (kFinal) y[c] = i == 0 ? mul2(cs[i], h[c][i]) : fma2(cs[i], h[c][i], y[c]);
                    }
                    if (kFinal) v[k * kPair + c] = y[c].x + y[c].y;
                }
            }
            if (kFinal) {
                // the lanes of a channel add up their states; lane q keeps the group's values q R ..
                constexpr int R = kGroup * kPair / LPC;
                add_parts<kGroup * kPair, LPC / 2, 1>(v, q);
#pragma unroll
                for (int k = 0; k < R; ++k)
                    sy[(t1 + (q * R + k) / kPair) * LY + g * kPair + (q * R + k) % kPair] = v[k];
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
                load8(sy + r * LY + (vc - d0), y);
                cu[j].get(x);
#pragma unroll
                for (int e = 0; e < kVec; ++e) y[e] = fmaf(skip[e], x[e], y[e]);
                if (a.z) {
                    cz[j].get(x);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) y[e] *= x[e] * sigmoid_fast(x[e]);
                }
                store8(static_cast<T*>(a.o) + (row0 + t0 + r) * D + vc, y);
            }
            __syncwarp();
        }
    }
    if (leave) store_states<SPL>(leave, h, NS, q, d0 + g * kPair, D);
    if (!kFinal) {
        // a channel's vectors lie in the lanes VR apart
#pragma unroll
        for (int m = L::VR; m < 32; m *= 2)
#pragma unroll
            for (int e = 0; e < kVec; ++e) total[e] += __shfl_xor_sync(0xffffffffu, total[e], m);
        if (lane < L::VR && vc < D) store8(steps + vc, total);
    }
}

// The rank-th segment of a packed batch in the order in which they are walked:
// all whole segments first, then what is left of each sequence, the longest
// first, so that the launch does not end on long ones.  All 32 lanes call it
// together and go over the offsets 32 at a time.  More than kSorted sequences
// leave their rests in the order of the batch, and more than kRanked take
// find_slot's order, as the search itself would cost too much.  In us, at 16384
// tokens x 4096 channels x 16 states: 64 sequences with the rests by length 414, in
// the batch's order 660; 128 sequences 613 and 508 (the search grows with the square
// of their number).  Whole segments first against find_slot's order: 65 sequences
// 515 and 555, 128 sequences 508 and 499, 256 sequences 511 and 461, 512 sequences
// 748 and 532; at 512 channels, where the batch is cut, 256 sequences take 121 and
// 109.  The two cross between 65 and 128 sequences, below the border.
constexpr int kRanked = 256, kSorted = 64;
__device__ __forceinline__ Slot find_ranked(const Rows& r, int rank) {
    if (!r.cu || r.B > kRanked) return find_slot(r, rank);
    const int lane = threadIdx.x & 31;
    auto tokens = [&](int b) {
        int row0 = 0, len = 0;
        if (b < r.B) packed_range(r.cu, b, r.total, row0, len);
        return min(len, r.N);
    };
    Slot f;
    f.b = -1; f.s = 0; f.segs = 0; f.first = 0; f.len = 0; f.seq_len = 0; f.row0 = 0;
    int b = -1, s = -1, base = 0;
    for (int b0 = 0; b0 < r.B; b0 += 32) {
        const int whole = tokens(b0 + lane) / r.seg;
        int upto = whole;
#pragma unroll
        for (int m = 1; m < 32; m *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += v;
        }
        const unsigned past = __ballot_sync(0xffffffffu, base + upto > rank);
        if (past) {
            const int at = __ffs(past) - 1;
            b = b0 + at;
            s = rank - base - __shfl_sync(0xffffffffu, upto - whole, at);
            break;
        }
        base += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (b < 0) {
        const int j = rank - base;
        if (j >= r.B) return f;
        b = j;
        if (r.B <= kSorted) {
            // the sequence that j others come before: those with more left, or as much and a lower number
            constexpr int kEach = kSorted / 32;
            int rest[kEach], before[kEach] = {};
#pragma unroll
            for (int k = 0; k < kEach; ++k) rest[k] = lane + 32 * k < r.B ? tokens(lane + 32 * k) % r.seg : -1;
#pragma unroll
            for (int o = 0; o < kEach; ++o)
                for (int l = 0; l < 32; ++l) {
                    const int v = __shfl_sync(0xffffffffu, rest[o], l);
#pragma unroll
                    for (int k = 0; k < kEach; ++k)
                        before[k] += v > rest[k] || (v == rest[k] && l + 32 * o < lane + 32 * k);
                }
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const unsigned hit = __ballot_sync(0xffffffffu, lane + 32 * k < r.B && before[k] == j);
                if (hit) b = __ffs(hit) - 1 + 32 * k;
            }
        }
    }
    int row0, len;
    packed_range(r.cu, b, r.total, row0, len);
    len = min(len, r.N);
    const int whole = len / r.seg;
    if (s < 0) {
        if (whole > 0 && whole * r.seg == len) return f;
        s = whole;
    }
    f.b = b;
    f.s = s;
    f.segs = segments_of(len, r.seg);
    f.seq_len = len;
    f.row0 = row0;
    f.first = s * r.seg;
    f.len = min(r.seg, len - f.first);
    return f;
}

// A sequence that is cut is walked in two launches.  The first gives the first
// segment's outputs, whose state before is known, and the local states of the
// segments between the first and the last; the second the other segments'
// outputs.  So two segments cost no token twice.  Up to kFoldSerial segments
// are folded by the second launch's warps themselves, each from the first to
// its own, which costs less than a launch; more are folded in between.  The
// blocks of a segment, which read the same rows, are next to one another.
template <typename T, int NS, bool kFirst>
__global__ void __launch_bounds__(kWarps * 32, NS >= 32 ? 3 : 4) selective_scan_kernel(const ScanArgs a, float* local,
                                                                                       float* steps, int blocks,
                                                                                       bool folded) {
    __shared__ __align__(16) float shared[kWarps * Layout<NS>::FLOATS];
    const int rank = blockIdx.x / blocks, block = blockIdx.x - rank * blocks;
    const Slot f = find_ranked(a.rows, rank);
    const bool last = f.s + 1 >= f.segs;
    if (f.b < 0 || (kFirst ? f.s > 0 && last : f.s == 0)) return;
    const size_t state = (size_t)a.D * NS, slot = slot_start(a.rows, f.b) + f.s;
    float* leave = !last ? local + slot * state : a.h ? a.h + f.b * state : nullptr;
    if (!kFirst) {
        const int apart = folded ? 0 : f.s - 1;
        const size_t from = slot - 1 - apart;
        walk<T, NS, true>(a, f, block, shared, local + from * state, apart, last ? leave : nullptr, steps + from * a.D);
    } else if (f.s == 0) {
        walk<T, NS, true>(a, f, block, shared, a.h0 ? a.h0 + f.b * state : nullptr, 0, leave, nullptr);
    } else {
        walk<T, NS, false>(a, f, block, shared, nullptr, 0, leave, steps + slot * a.D);
    }
}

// The state after every segment but the last, from the first one's and the
// local ones of the others, over the local ones in place.
template <int NS>
__global__ void __launch_bounds__(kFoldThreads) fold_kernel(const ScanArgs a, float* local, const float* steps) {
    constexpr int Y = 8;
    __shared__ FoldShared<Y> shared;
    const int blocks = fold_blocks<Y>(a.D, NS), b = blockIdx.x / blocks;
    const int i = (blockIdx.x - b * blocks) * kFoldX<Y> + threadIdx.x;
    const bool on = i < a.D * (NS / 4);
    const int d = on ? i / (NS / 4) : 0, q = on ? i % (NS / 4) * 4 : 0;
    int len = a.rows.N;
    if (a.rows.cu) {
        int row0;
        packed_range(a.rows.cu, b, a.rows.total, row0, len);
        len = min(len, a.rows.N);
    }
    const int cuts = segments_of(len, a.rows.seg) - 1;
    if (cuts <= 1) return;
    const long long slot = slot_start(a.rows, b), stride = (long long)a.D * NS;
    float* first = local + slot * stride + (size_t)d * NS + q;
    fold_segments<true, Y>(shared, on, first + stride, stride, steps + (slot + 1) * a.D + d, a.D, cuts - 1,
                        *reinterpret_cast<const float4*>(a.A + (size_t)d * NS + q), *reinterpret_cast<const float4*>(first));
}

// Tokens of a segment: N leaves the sequences whole.  Measured with 16 states,
// a token costs a warp 88 ns when it has its scheduler to itself, 62 ns a warp
// when two share it, and with many warps 53 ns; cut sequences pay the last for
// most of their tokens twice.  Whole packed sequences, the longest first, take
// a tenth more than that, or 127 ns for each token of the longest; in the order
// of the batch the two may come one after the other.  For example, in us whole
// / cut: 1 x 4096 tokens x 4096 channels 358 / 189, 2 x 1024 x 4096 94 / 100,
// 4 x 4096 x 4096 514 / 594, 38 packed sequences of 16384 tokens, the longest
// of 2470, x 4096 channels 412 / 493 and x 2048 channels 314 / 283.  The segment
// gives some 4096 warps, about twice what the GPU holds: fewer leave it idle at
// the end, more cost staging.  The second launch and its workspace count 16 us,
// 10 on the GPU and as much again for the host that has to issue them.  A lane of
// 8 states takes twice as long a token.  A segment has 64 tokens, or down to a
// tile where all warps still fit the GPU at once (900 tokens x 256 channels x 16
// states: 64, 32, 16 tokens a segment take 21, 15 and 13 us).
int segment(int B, int N, int total, int D, int n, bool packed, int num_sms) {
    const int width = n == 8 ? 32 : n == 64 ? 8 : 16;
    const double warps = (D + width - 1) / width, tokens = packed ? (double)total : (double)B * N;
    const double lane = n >= 32 ? 2 : 1;                    // states of a lane, in fours
    const double schedulers = 4.0 * num_sms, filled = lane * 53e-3 * tokens * warps / schedulers;
    const double shared = B * warps / schedulers;
    const double whole = !packed ? lane * N * (shared <= 1 ? 88e-3 : 62e-3 * ceil(shared))
                         : B <= kSorted ? fmax(1.1 * filled, lane * 127e-3 * N) : filled + lane * 127e-3 * N;
    long long seg = (long long)ceil(tokens * warps / 4096 / kTile) * kTile;
    int least = 4 * kTile;
    while (least > kTile && tokens * warps / (least / 2) <= 12.0 * num_sms) least /= 2;
    if (seg < least) seg = least;
    if (seg >= N) return N;
    const double cut = (packed ? 1.45 : 1.1 * (2.0 - (double)seg / N)) * filled + 16;
    return whole <= cut ? N : (int)seg;
}

// Four values next to one another.
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
}

// One token per sequence: the states are read and written once, 16 bytes at a
// time, n / 4 lanes to a channel, and the memory bandwidth bounds the time.  A
// thread takes its states of kStepSeqs sequences, whose loads are all in flight
// together and which share A: 27 us, 5.2 TB/s, at 256 sequences x 4096 channels x
// 16 states (one sequence a thread 39 us).  h may be h0.
constexpr int kStepSeqs = 4;
template <typename T, int NS>
__global__ void __launch_bounds__(kStepThreads) selective_step_kernel(const ScanArgs a) {
    constexpr int L = NS / 4;
    const int D = a.D, S = a.rows.B, blocks = (D * L + kStepThreads - 1) / kStepThreads;   // of a group of sequences
    const int i = blockIdx.x % blocks * kStepThreads + threadIdx.x;
    const bool on = i < D * L;
    const int d = on ? i / L : 0, q = i % L * 4;
    const long long b0 = (long long)(blockIdx.x / blocks) * kStepSeqs;
    float4 h[kStepSeqs], B[kStepSeqs], C[kStepSeqs];
    float u[kStepSeqs], raw[kStepSeqs], z[kStepSeqs];
#pragma unroll
    for (int k = 0; k < kStepSeqs; ++k) {
        const long long b = b0 + k < S ? b0 + k : S - 1;
        h[k] = __ldcs(reinterpret_cast<const float4*>(a.h0 + (b * D + d) * NS + q));
        B[k] = load4(static_cast<const T*>(a.Bm) + b * a.ldb + q);
        C[k] = load4(static_cast<const T*>(a.Cm) + b * a.ldc + q);
        u[k] = to_f32(static_cast<const T*>(a.u)[b * a.ldu + d]);
        raw[k] = to_f32(static_cast<const T*>(a.dt)[b * a.lddt + d]);
        z[k] = a.z ? to_f32(static_cast<const T*>(a.z)[b * a.ldz + d]) : 0.f;
    }
    const float4 A = log2_rate(*reinterpret_cast<const float4*>(a.A + (size_t)d * NS + q));
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f, skip = a.skip ? a.skip[d] : 0.f;
#pragma unroll
    for (int k = 0; k < kStepSeqs; k += 2) {
        const float2 pair = softplus2(make_float2(raw[k] + bias, raw[k + 1] + bias));
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const int j = k + o;
            const long long b = b0 + j;
            const float delta = o ? pair.y : pair.x, du = delta * u[j];
            h[j].x = fmaf(exp2_approx(delta * A.x), h[j].x, du * B[j].x);
            h[j].y = fmaf(exp2_approx(delta * A.y), h[j].y, du * B[j].y);
            h[j].z = fmaf(exp2_approx(delta * A.z), h[j].z, du * B[j].z);
            h[j].w = fmaf(exp2_approx(delta * A.w), h[j].w, du * B[j].w);
            float y = C[j].x * h[j].x + C[j].y * h[j].y + C[j].z * h[j].z + C[j].w * h[j].w;
#pragma unroll
            for (int m = L / 2; m > 0; m >>= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
            if (!on || b >= S) continue;
            __stcs(reinterpret_cast<float4*>(a.h + (b * D + d) * NS + q), h[j]);
            if (q == 0) {
                y = fmaf(skip, u[j], y);
                if (a.z) y *= z[j] * sigmoid_fast(z[j]);
                static_cast<T*>(a.o)[b * D + d] = from_f32<T>(y);
            }
        }
    }
}

template <typename T, int NS>
cudaError_t scan(const ScanArgs& a, cudaStream_t s) {
    constexpr int W = Layout<NS>::W;
    const long long slots = slots_of(a.rows);
    const int blocks = (a.D + kWarps * W - 1) / (kWarps * W);
    const unsigned grid = (unsigned)(slots * blocks);
    float* local = static_cast<float*>(a.workspace);
    float* steps = local + (size_t)slots * a.D * NS;
    selective_scan_kernel<T, NS, true><<<grid, kWarps * 32, 0, s>>>(a, local, steps, blocks, false);
    if (a.rows.seg < a.rows.N) {
        const bool fold = (long long)kFoldSerial * a.rows.seg < a.rows.N;
        if (fold)
            fold_kernel<NS><<<a.rows.B * fold_blocks<8>(a.D, NS), dim3(kFoldX<8>, 8), 0, s>>>(a, local, steps);
        selective_scan_kernel<T, NS, false><<<grid, kWarps * 32, 0, s>>>(a, local, steps, blocks, fold);
    }
    return cudaGetLastError();
}

template <typename T, int NS>
cudaError_t step(const ScanArgs& a, cudaStream_t s) {
    const long long blocks = (a.D * (NS / 4) + kStepThreads - 1) / kStepThreads;
    const long long groups = ((long long)a.rows.B + kStepSeqs - 1) / kStepSeqs;
    selective_step_kernel<T, NS><<<(unsigned)(blocks * groups), kStepThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

bool selective_states_supported(int n) { return n == 8 || n == 16 || n == 32 || n == 64; }

size_t selective_scan_ws_bytes(int B, int N, int total, int D, int n, bool packed, int num_sms) {
    const int seg = segment(B, N, total, D, n, packed, num_sms);
    if (seg >= N) return 0;
    const long long slots = packed ? (long long)total / seg + B : (long long)B * segments_of(N, seg);
    return align256((size_t)slots * D * (n + 1) * sizeof(float));
}

cudaError_t launch_selective_scan(ScanArgs a, int num_sms, cudaStream_t s) {
    a.rows.seg = segment(a.rows.B, a.rows.N, a.rows.total, a.D, a.n, a.rows.cu != nullptr, num_sms);
    const bool bf = a.io == GRET_BF16;
    switch (a.n) {
        case 8: return bf ? scan<__nv_bfloat16, 8>(a, s) : scan<float, 8>(a, s);
        case 16: return bf ? scan<__nv_bfloat16, 16>(a, s) : scan<float, 16>(a, s);
        case 32: return bf ? scan<__nv_bfloat16, 32>(a, s) : scan<float, 32>(a, s);
        default: return bf ? scan<__nv_bfloat16, 64>(a, s) : scan<float, 64>(a, s);
    }
}

cudaError_t launch_selective_step(const ScanArgs& a, cudaStream_t s) {
    const bool bf = a.io == GRET_BF16;
    switch (a.n) {
        case 8: return bf ? step<__nv_bfloat16, 8>(a, s) : step<float, 8>(a, s);
        case 16: return bf ? step<__nv_bfloat16, 16>(a, s) : step<float, 16>(a, s);
        case 32: return bf ? step<__nv_bfloat16, 32>(a, s) : step<float, 32>(a, s);
        default: return bf ? step<__nv_bfloat16, 64>(a, s) : step<float, 64>(a, s);
    }
}

}  // namespace gret
