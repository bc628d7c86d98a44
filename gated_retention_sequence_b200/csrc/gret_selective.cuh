// What the selective scan and its gradients share: the way a warp holds
// channels and states.
#pragma once

#include "gret_block.cuh"

namespace gret {

constexpr int kScanWarps = 4;       // warps of a block: neighbouring channels, the same tokens
constexpr int kPair = 2;            // channels of a lane

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
