// What the selective scan and its gradients share: the way a warp holds
// channels and states.
#pragma once

#include <float.h>

#include "gret_block.cuh"

namespace gret {

constexpr int kScanWarps = 4;       // warps of a block: neighbouring channels, the same tokens
constexpr int kPair = 2;            // channels of a lane

// A in powers of two a unit step.  A = -inf, which keeps nothing of the tokens
// before, and an A whose product with log2 e passes fp32 are the lowest finite
// number: a step of zero, as the tokens that fill a group have, then leaves the
// state as it is instead of giving 0 x inf.  NaN stays NaN.
__device__ __forceinline__ float log2_rate(float A) {
    const float x = A * kLog2e;
    return x < -FLT_MAX ? -FLT_MAX : x;
}
__device__ __forceinline__ float2 log2_rate(float2 A) { return make_float2(log2_rate(A.x), log2_rate(A.y)); }
__device__ __forceinline__ float4 log2_rate(float4 A) {
    return make_float4(log2_rate(A.x), log2_rate(A.y), log2_rate(A.z), log2_rate(A.w));
}

// The values of a lane's two channels x SPL states, as pairs of states, from
// or to rows of n per channel; a channel from `end` on reads as zero.
template <int SPL>
__device__ __forceinline__ void load_states(float2 (*v)[SPL / 2], const float* from, int n, int q, int d, int end) {
#pragma unroll
    for (int c = 0; c < kPair; ++c)
#pragma unroll
        for (int i = 0; i < SPL / 2; i += 2) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (from && d + c < end) x = *reinterpret_cast<const float4*>(from + (size_t)(d + c) * n + q * SPL + 2 * i);
            v[c][i] = make_float2(x.x, x.y);
            v[c][i + 1] = make_float2(x.z, x.w);
        }
}
template <int SPL>
__device__ __forceinline__ void store_states(float* to, const float2 (*v)[SPL / 2], int n, int q, int d, int end) {
#pragma unroll
    for (int c = 0; c < kPair; ++c)
#pragma unroll
        for (int i = 0; i < SPL / 2; i += 2)
            if (d + c < end)
                *reinterpret_cast<float4*>(to + (size_t)(d + c) * n + q * SPL + 2 * i) =
                    make_float4(v[c][i].x, v[c][i].y, v[c][i + 1].x, v[c][i + 1].y);
}

// The fold that joins segments: x <- exp(A s_k) x + v_k for k = 0 .. count - 1,
// four states a thread.  v_k, kFoldX threads next to one another, lies at
// v + k stride and s_k at sums + k step; each is replaced by x after it
// (kAfter) or before it.  Few threads walk many segments here, and one after
// another their loads would bound the time, so Y threads take kFoldU segments
// each: every thread folds its own from zero, the block (128 / Y, Y) carries x
// through the parts, and each thread goes over its own again.  All threads of
// the block call it; x has to be the same for all of a column, and is returned
// after the last segment.  Y is 8 for sequences of more than kFoldSerial
// segments: 127 segments of 512 channels x 16 states take 10 us, and 31 with
// one thread for all of a state's segments.
constexpr int kFoldU = 8, kFoldSerial = 16, kFoldThreads = 128;
template <int Y> constexpr int kFoldX = kFoldThreads / Y;
// Blocks of a sequence's fold.  A sequence has up to 65536 of them (65536
// channels x 64 states), one more than a grid's second dimension takes, so that
// a launch counts them all in its first.
template <int Y>
__host__ __device__ __forceinline__ int fold_blocks(int D, int n) {
    return (D * (n / 4) + kFoldX<Y> - 1) / kFoldX<Y>;
}
template <int Y>
struct FoldShared {
    float4 decay[Y][kFoldX<Y>], local[Y][kFoldX<Y>];
};
__device__ __forceinline__ float4 fma4(float4 a, float4 b, float4 c) {
    return make_float4(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y), fmaf(a.z, b.z, c.z), fmaf(a.w, b.w, c.w));
}
template <bool kAfter, int Y>
__device__ __forceinline__ float4 fold_segments(FoldShared<Y>& shared, bool on, float* v, long long stride, const float* sums,
                                                long long step, int count, float4 A, float4 x) {
    const int tx = threadIdx.x, ty = threadIdx.y;
    A = log2_rate(A);
    for (int base = 0; base < count; base += Y * kFoldU) {
        const int first = base + ty * kFoldU, mine = on ? min(kFoldU, count - first) : 0;
        float4 l[kFoldU];
        float s[kFoldU];
#pragma unroll
        for (int j = 0; j < kFoldU; ++j)
            if (j < mine) {
                l[j] = *reinterpret_cast<const float4*>(v + (first + j) * stride);
                s[j] = sums[(first + j) * step];
            }
        float4 here = x;
        if constexpr (Y > 1) {
            float4 own = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < kFoldU; ++j)
                if (j < mine) {
                    own = fma4(make_float4(exp2_approx(s[j] * A.x), exp2_approx(s[j] * A.y), exp2_approx(s[j] * A.z),
                                           exp2_approx(s[j] * A.w)), own, l[j]);
                    sum += s[j];
                }
            shared.decay[ty][tx] = make_float4(exp2_approx(sum * A.x), exp2_approx(sum * A.y), exp2_approx(sum * A.z),
                                               exp2_approx(sum * A.w));
            shared.local[ty][tx] = own;
            __syncthreads();
#pragma unroll
            for (int y = 0; y < Y; ++y) {
                if (y == ty) here = x;
                x = fma4(shared.decay[y][tx], x, shared.local[y][tx]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < kFoldU; ++j)
            if (j < mine) {
                float4* to = reinterpret_cast<float4*>(v + (first + j) * stride);
                if (!kAfter) *to = here;
                here = fma4(make_float4(exp2_approx(s[j] * A.x), exp2_approx(s[j] * A.y), exp2_approx(s[j] * A.z),
                                        exp2_approx(s[j] * A.w)), here, l[j]);
                if (kAfter) *to = here;
            }
        if (Y == 1) x = here;
    }
    return x;
}

// COUNT values, each held in parts by the lanes that differ in the bits First,
// First / 2, ... Last of the lane: every round halves what a lane keeps, by the
// bit, while the count is even, and otherwise adds all of it.  Returns how many
// values a lane has left, from v[0]; the bits of the halving rounds, the first
// the highest, count the parts.
template <int COUNT, int First, int Last>
__device__ __forceinline__ constexpr int parts_left() {
    int n = COUNT;
    for (int m = First; m >= Last; m /= 2)
        if (n % 2 == 0) n /= 2;
    return n;
}
template <int COUNT, int First, int Last>
__device__ __forceinline__ void add_parts(float* v, int lane) {
    if constexpr (First >= Last) {
        if constexpr (COUNT % 2 == 0) {
            const bool up = (lane & First) != 0;
#pragma unroll
            for (int i = 0; i < COUNT / 2; ++i) {
                const float keep = up ? v[i + COUNT / 2] : v[i], send = up ? v[i] : v[i + COUNT / 2];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, First);
            }
            add_parts<COUNT / 2, First / 2, Last>(v, lane);
        } else {
#pragma unroll
            for (int i = 0; i < COUNT; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], First);
            add_parts<COUNT, First / 2, Last>(v, lane);
        }
    }
}

}  // namespace gret
