// Operators of the selective state space block (internal header): the short
// causal convolution, the selective scan and the residual norm.
//
// Tokens come as rows.  A uniform batch has B sequences of N rows each; a
// packed one has `total` rows, cut by cu_seqlens (device).  Either way the
// kernels walk slots: a slot is one segment of at most `seg` consecutive tokens
// of one sequence.  Sequence b's slots start at b * ceil(N / seg) in a uniform
// batch and at floor(cu_seqlens[b] / seg) + b in a packed one: that leaves
// every sequence room for ceil(len / seg) slots (at least one, so an empty
// sequence has a slot that hands its state on), and total / seg + B slots hold
// them all, without a plan and without a host copy of the offsets.
#pragma once

#include "gret_common.cuh"

namespace gret {

// Device status word and SM count of the current device.
bool device_info(unsigned int** status, int* num_sms);
// Take one injected timeout, if any is pending (gret_debug_inject_timeout).
int take_injected_timeout();

struct Rows {
    const int* cu;      // device offsets [B + 1], or null for a uniform batch
    int B, N;           // sequences; tokens of each, or the longest (at most `total`)
    int total;          // rows of a packed batch
    int seg;            // tokens of a slot
};

// Segments of `len` tokens, without a sum that could pass 31 bits.
__host__ __device__ __forceinline__ int segments_of(int len, int seg) { return len > 0 ? (len - 1) / seg + 1 : 0; }
inline long long slots_of(const Rows& r) {
    return r.cu ? (long long)r.total / r.seg + r.B : (long long)r.B * segments_of(r.N, r.seg);
}

struct Slot {
    int b;              // sequence, or -1 for a slot that holds nothing
    int s;              // segment of the sequence
    int segs;           // segments the sequence has (0 when it is empty)
    int first;          // first token of the segment within its sequence
    int len;            // tokens of the segment
    int seq_len;        // tokens of the sequence
    long long row0;     // row of the sequence's first token
};

__device__ __forceinline__ long long slot_start(const Rows& r, int b) {
    if (!r.cu) return (long long)b * segments_of(r.N, r.seg);
    int c = r.cu[b];
    c = c < 0 ? 0 : (c > r.total ? r.total : c);
    return (long long)(c / r.seg) + b;
}

// The segment a slot holds.  All 32 lanes call it together: in a packed batch
// they search the offsets 32 at a time.  Offsets that are not in order give
// slots without tokens or rows that another slot has too, never a row outside
// the tensors (packed_range clamps both ends).
__device__ __forceinline__ Slot find_slot(const Rows& r, int slot) {
    Slot f;
    f.b = -1; f.s = 0; f.segs = 0; f.first = 0; f.len = 0; f.seq_len = 0; f.row0 = 0;
    if (!r.cu) {
        const int per = segments_of(r.N, r.seg);
        f.b = slot / per;
        f.s = slot - f.b * per;
        f.segs = per;
        f.seq_len = r.N;
        f.row0 = (long long)f.b * r.N;
    } else {
        const int lane = threadIdx.x & 31;
        int lo = 0, n = r.B;
        while (true) {
            const int step = (n + 31) / 32;
            const int at = lo + lane * step;
            const bool before = at < lo + n && slot_start(r, at) <= slot;
            const int hits = __popc(__ballot_sync(0xffffffffu, before));
            if (hits == 0) return f;
            lo += (hits - 1) * step;
            n = min(step, n - (hits - 1) * step);
            if (n <= 1 || step == 1) break;
        }
        int row0, len;
        packed_range(r.cu, lo, r.total, row0, len);
        len = min(len, r.N);
        f.s = (int)(slot - slot_start(r, lo));
        f.segs = segments_of(len, r.seg);
        if (f.s < 0 || f.s >= max(f.segs, 1)) return f;
        f.b = lo;
        f.seq_len = len;
        f.row0 = row0;
    }
    f.first = f.s * r.seg;
    f.len = min(r.seg, f.seq_len - f.first);
    return f;
}

// Eight consecutive channels: 16 bytes of bf16 or 32 of fp32, 16-byte aligned.
constexpr int kVec = 8;
__device__ __forceinline__ void unpack8(const uint4& p, float* v) {
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
    unpack8(*reinterpret_cast<const uint4*>(p), v);
}
__device__ __forceinline__ void load8(const float* p, float* v) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
    *reinterpret_cast<uint4*>(p) = pack8(v);
}
__device__ __forceinline__ void store8(float* p, const float* v) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

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
template <typename T>
__device__ __forceinline__ void pairs_of(const Raw<T>& r, float2* v) {
    float x[kVec];
    r.get(x);
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i) v[i] = make_float2(x[2 * i], x[2 * i + 1]);
}

// Asynchronous copies into shared memory: the end of a group, and the wait until
// at most N groups are under way.
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<unsigned long long&>(r))
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
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// One special function each: 2^x (2 units in the last place) and 1/x.
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// sigmoid with two special functions: 1 / (1 + 2^(-x log2 e)).  An overflow of
// the power gives 0, as it should.
__device__ __forceinline__ float sigmoid_fast(float x) { return rcp_approx(1.0f + exp2_approx(-kLog2e * x)); }

__device__ __forceinline__ float2 sigmoid2(float2 x) { return make_float2(sigmoid_fast(x.x), sigmoid_fast(x.y)); }

// softplus of two numbers, max(x, 0) + log1p(e), e = exp(-|x|) in (0, 1].
// log1p(e) = e P(e) with P of degree 9, the minimax fit of log1p(e) / e on
// [0, 1] in relative error by Remez exchange, so that small steps keep their
// relative precision; one special function each instead of two.  In units of
// 2^-24 over the interval: P of these fp32 coefficients is off by 0.56, and e P(e)
// formed in fp32 by 2.6.
__device__ __forceinline__ float2 softplus2(float2 x) {
    const float2 e = make_float2(exp2_approx(-kLog2e * fabsf(x.x)), exp2_approx(-kLog2e * fabsf(x.y)));
    float2 p = both(-0.0032440251670777798f);
    p = fma2(p, e, both(0.01985146291553974f));
    p = fma2(p, e, both(-0.05695953592658043f));
    p = fma2(p, e, both(0.10603655129671097f));
    p = fma2(p, e, both(-0.15305592119693756f));
    p = fma2(p, e, both(0.1967593878507614f));
    p = fma2(p, e, both(-0.24954134225845337f));
    p = fma2(p, e, both(0.3332996368408203f));
    p = fma2(p, e, both(-0.4999990165233612f));
    p = fma2(p, e, both(1.0f));
    return fma2(p, e, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}

// d/dv of v sigmoid(v)
__device__ __forceinline__ float swish_slope(float v, float sig) { return sig * (1.0f + v * (1.0f - sig)); }
__device__ __forceinline__ float2 swish_slope2(float2 v, float2 sig) {
    return mul2(sig, fma2(v, fma2(sig, both(-1.f), both(1.f)), both(1.f)));
}

template <typename T>
__device__ __forceinline__ void store_pairs(T* p, const float2* v) {
    const float x[kVec] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
    store8(p, x);
}

// partial [groups][offset[count]] summed over the groups; columns offset[j] ..
// offset[j + 1] - 1 go to dst[j], stride[j] floats apart (null: not wanted).
struct ColumnOutputs {
    int count;
    long long offset[6];
    float* dst[5];
    int stride[5];
};
cudaError_t launch_column_sums(const float* partial, int groups, const ColumnOutputs& out, cudaStream_t s);

// A block's share of them: `width` columns, whose groups kSumThreads / width
// lanes take in turn; 32 columns, or 8 where these are few blocks with many
// groups each (2368 groups of 216 columns: some 40 us with 32 columns a block,
// 11 with 8).  The order is fixed, so that the result does not depend on which
// blocks ended first.
constexpr int kSumThreads = 256;
inline int column_width(const ColumnOutputs& out, int groups) {
    return groups >= 64 && out.offset[out.count] < 32 * 256 ? 8 : 32;
}
inline long long column_blocks(const ColumnOutputs& out, int width) { return (out.offset[out.count] + width - 1) / width; }
__device__ __forceinline__ void column_sums(const float* partial, int groups, const ColumnOutputs& out, int width,
                                            long long block) {
    __shared__ float red[kSumThreads];
    const int x = threadIdx.x % width, y = threadIdx.x / width, lanes = kSumThreads / width;
    const long long c = block * width + x, cols = out.offset[out.count];
    float s = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int g = y; g < groups; g += lanes) s += partial[g * cols + c];
    }
    red[threadIdx.x] = s;
    __syncthreads();
    if (y != 0 || c >= cols) return;
    s = 0.f;
    for (int i = 0; i < lanes; ++i) s += red[i * width + x];
    int j = 0;
    while (j + 1 < out.count && c >= out.offset[j + 1]) ++j;
    if (out.dst[j]) out.dst[j][(c - out.offset[j]) * out.stride[j]] = s;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct ConvArgs {
    const void* x;
    long long ldx;
    const float *w, *bias;
    const void* tail0;
    void *y, *tail;
    Rows rows;
    int D, K;
    int swish;
    gret_dtype io;
};
cudaError_t launch_short_conv(ConvArgs a, int num_sms, cudaStream_t s);
cudaError_t launch_short_conv_step(const ConvArgs& a, cudaStream_t s);   // tail0 -> tail, B rows

struct ConvBackwardArgs {
    ConvArgs f;          // x, w, bias, tail0 of the forward
    const void *dy, *dtail;
    void *dx, *dtail0;
    float *dw, *dbias;
    void* workspace;
};
size_t short_conv_backward_ws_bytes(int B, int N, int D, int K, int num_sms);
cudaError_t launch_short_conv_backward(ConvBackwardArgs a, int num_sms, cudaStream_t s);

struct ScanArgs {
    const void *u, *dt, *Bm, *Cm, *z;
    long long ldu, lddt, ldb, ldc, ldz;
    const float *A, *skip, *dt_bias, *h0;
    void* o;
    float* h;
    Rows rows;
    int D, n;
    gret_dtype io;
    void* workspace;
};
bool selective_states_supported(int n);
size_t selective_scan_ws_bytes(int B, int N, int total, int D, int n, bool packed, int num_sms);
cudaError_t launch_selective_scan(ScanArgs a, int num_sms, cudaStream_t s);
cudaError_t launch_selective_step(const ScanArgs& a, cudaStream_t s);   // h0 -> h, B rows

struct ScanBackwardArgs {
    ScanArgs f;          // inputs of the forward
    const void* dout;
    const float* dh_final;
    void *du, *ddt, *dBm, *dCm, *dz;
    float *dA, *dskip, *ddt_bias, *dh0;
    void* workspace;
};
size_t selective_backward_ws_bytes(int B, int N, int D, int n);
cudaError_t launch_selective_backward(const ScanBackwardArgs& a, cudaStream_t s);

struct NormArgs {
    const void *x, *y, *gate;
    long long ldx, ldy, ldg;
    const float *scale, *w_post, *w_next;
    void *r, *n;
    long long T;
    int D;
    float eps;
    gret_dtype stream_type, io;
};
cudaError_t launch_residual_norm(const NormArgs& a, int num_sms, cudaStream_t s);

struct NormBackwardArgs {
    NormArgs f;
    const void *dr, *dn;
    void *dx, *dy, *dgate;
    float *dscale, *dw_post, *dw_next;
    void* workspace;
    unsigned int* status;       // device status word
    int fault;                  // test only: inject a timed-out wait
};
constexpr int kNormMaxChannels = 8192;
size_t residual_norm_backward_ws_bytes(long long T, int D, int num_sms);
cudaError_t launch_residual_norm_backward(NormBackwardArgs a, int num_sms, cudaStream_t s);

}  // namespace gret
