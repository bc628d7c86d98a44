// C ABI of the selective state space block's operators: argument validation
// and launch.  As in gret_api.cu nothing is allocated, copied or read here, and
// a bad call returns before any launch.
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "gret_block.cuh"

using namespace gret;

namespace {

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename... P>
bool all_set(P... p) {
    return (... && (p != nullptr));
}

template <typename... P>
bool all_aligned(P... p) {
    return (... && aligned(p));
}

size_t size_of(gret_dtype t) { return t == GRET_BF16 ? 2 : 4; }
bool type_ok(gret_dtype t) { return t == GRET_F32 || t == GRET_BF16; }

// A row stride: at least the row, rows on 16-byte boundaries.
bool stride_ok(long long ld, int width, gret_dtype t) {
    return ld >= width && ld <= (1LL << 40) && ld * (long long)size_of(t) % 16 == 0;
}

// What a pointer names: `bytes` from p on (nothing where p is null).
struct Region {
    const void* p;
    size_t bytes;
};
bool overlap(const Region& x, const Region& y) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
    return x.p && y.p && a < b + y.bytes && b < a + x.bytes;
}
// No output meets an input or another output.
bool apart(std::initializer_list<Region> outputs, std::initializer_list<Region> inputs) {
    for (const Region* o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Region& i : inputs)
            if (overlap(*o, i)) return false;
        for (const Region* p = outputs.begin(); p != o; ++p)
            if (overlap(*o, *p)) return false;
    }
    return true;
}

// Bytes from a tensor's first row to the end of its last.
size_t span(long long rows, long long ld, int width, gret_dtype t) {
    return ((size_t)(rows - 1) * ld + width) * size_of(t);
}
size_t floats(long long a, long long b = 1, long long c = 1) { return (size_t)a * b * c * sizeof(float); }
Region offsets(const Rows& r) { return {r.cu, ((size_t)r.B + 1) * sizeof(int)}; }
long long rows_of(const Rows& r) { return r.cu ? (long long)r.total : (long long)r.B * r.N; }

constexpr long long kMaxRows = (1LL << 31) - (1 << 20);     // a walk may count a few rows past the end in 31 bits
constexpr int kMaxChannels = 1 << 16;       // channel blocks are a grid's second dimension

Rows uniform(int B, int N) { return Rows{nullptr, B, N, 0, 0}; }
// No sequence of a packed batch is longer than all its rows.
Rows packed(const int* cu, int num_seqs, int max_seqlen, int total) {
    return Rows{cu, num_seqs, max_seqlen < total ? max_seqlen : total, total, 0};
}

gret_status rows_ok(const Rows& r, bool packed) {
    if (r.B <= 0 || r.N <= 0 || (packed && r.total <= 0)) return GRET_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(r.cu) & 3u) != 0) return GRET_ERR_INVALID_ARG;
    // rows, and slots of at least one token and one more a sequence
    if ((packed ? (long long)r.total + r.B : (long long)r.B * r.N) >= kMaxRows) return GRET_ERR_UNSUPPORTED;
    return GRET_OK;
}
gret_status rows_ok(const Rows& r) { return rows_ok(r, r.cu != nullptr); }

gret_status done(cudaError_t e) { return e == cudaSuccess ? GRET_OK : GRET_ERR_CUDA; }

cudaStream_t cu_stream(gret_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// ------------------------------------------------------------ short convolution
gret_status conv_sizes(const Rows& r, int D, int K) {
    if (D <= 0 || K <= 0) return GRET_ERR_INVALID_ARG;
    if (gret_status e = rows_ok(r)) return e;
    return D % kVec != 0 || D > kMaxChannels || K < 2 || K > 4 ? GRET_ERR_UNSUPPORTED : GRET_OK;
}

gret_status conv_check(const ConvArgs& a) {
    if (!all_set(a.x, a.w, a.y) || !type_ok(a.io)) return GRET_ERR_INVALID_ARG;
    if (!all_aligned(a.x, a.w, a.bias, a.tail0, a.y, a.tail)) return GRET_ERR_INVALID_ARG;
    if (gret_status e = conv_sizes(a.rows, a.D, a.K)) return e;
    if (!stride_ok(a.ldx, a.D, a.io)) return GRET_ERR_INVALID_ARG;
    return GRET_OK;
}

// What a convolution's arguments name, and whether its outputs are apart from what it reads.
Region conv_rows(const ConvArgs& a, const void* p, long long ld) { return {p, span(rows_of(a.rows), ld, a.D, a.io)}; }
Region conv_tail(const ConvArgs& a, const void* p) {
    return {p, (size_t)a.rows.B * (a.K - 1) * a.D * size_of(a.io)};
}
bool conv_apart(const ConvArgs& a, const void* tail0) {
    return apart({conv_rows(a, a.y, a.D), conv_tail(a, a.tail)},
                 {conv_rows(a, a.x, a.ldx), conv_tail(a, tail0), {a.w, floats(a.D, a.K)}, {a.bias, floats(a.D)}, offsets(a.rows)});
}

gret_status conv(const void* x, long long ldx, const float* w, const float* bias, const void* tail0, void* y,
                 void* tail, Rows rows, int D, int K, gret_dtype io, gret_activation act, gret_stream_t stream) {
    if (act != GRET_ACT_NONE && act != GRET_ACT_SWISH) return GRET_ERR_INVALID_ARG;
    const ConvArgs a = {x, ldx, w, bias, tail0, y, tail, rows, D, K, act == GRET_ACT_SWISH, io};
    if (gret_status e = conv_check(a)) return e;
    if (!conv_apart(a, tail0)) return GRET_ERR_INVALID_ARG;
    int sms = 0;
    if (!device_info(nullptr, &sms)) return GRET_ERR_CUDA;
    return done(launch_short_conv(a, sms, cu_stream(stream)));
}

// --------------------------------------------------------------- selective scan
gret_status scan_sizes(const Rows& r, bool packed, int D, int n) {
    if (D <= 0 || n <= 0) return GRET_ERR_INVALID_ARG;
    if (gret_status e = rows_ok(r, packed)) return e;
    if (D % kVec != 0 || D > kMaxChannels || !selective_states_supported(n)) return GRET_ERR_UNSUPPORTED;
    const long long rows = packed ? (long long)r.total : (long long)r.B * r.N;
    return (long long)r.B * D * n > (1LL << 38) || rows * D > (1LL << 40) ? GRET_ERR_UNSUPPORTED : GRET_OK;
}

gret_status scan_check(const ScanArgs& a) {
    if (!all_set(a.u, a.dt, a.A, a.Bm, a.Cm, a.o) || !type_ok(a.io)) return GRET_ERR_INVALID_ARG;
    if (!all_aligned(a.u, a.dt, a.A, a.Bm, a.Cm, a.skip, a.z, a.dt_bias, a.h0, a.o, a.h)) return GRET_ERR_INVALID_ARG;
    if (gret_status e = scan_sizes(a.rows, a.rows.cu != nullptr, a.D, a.n)) return e;
    if (!stride_ok(a.ldu, a.D, a.io) || !stride_ok(a.lddt, a.D, a.io) || !stride_ok(a.ldb, a.n, a.io) ||
        !stride_ok(a.ldc, a.n, a.io) || (a.z && !stride_ok(a.ldz, a.D, a.io)))
        return GRET_ERR_INVALID_ARG;
    return GRET_OK;
}

// What a scan's arguments name, and whether its outputs are apart from what it reads.
Region scan_rows(const ScanArgs& a, const void* p, long long ld, int width) {
    return {p, span(rows_of(a.rows), ld, width, a.io)};
}
Region scan_state(const ScanArgs& a, const void* p) { return {p, floats(a.rows.B, a.D, a.n)}; }
bool scan_apart(const ScanArgs& a, const float* h0, size_t workspace_bytes) {
    return apart({scan_rows(a, a.o, a.D, a.D), scan_state(a, a.h), {workspace_bytes ? a.workspace : nullptr, workspace_bytes}},
                 {scan_rows(a, a.u, a.ldu, a.D), scan_rows(a, a.dt, a.lddt, a.D), scan_rows(a, a.z, a.ldz, a.D),
                  scan_rows(a, a.Bm, a.ldb, a.n), scan_rows(a, a.Cm, a.ldc, a.n), {a.A, floats(a.D, a.n)},
                  {a.skip, floats(a.D)}, {a.dt_bias, floats(a.D)}, scan_state(a, h0), offsets(a.rows)});
}

bool workspace_ok(const void* ws, size_t have, size_t need) {
    return need == 0 || (ws && have >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0);
}

gret_status scan(ScanArgs a, size_t workspace_bytes, gret_stream_t stream) {
    if (gret_status e = scan_check(a)) return e;
    int sms = 148;
    const bool device = device_info(nullptr, &sms);
    const size_t need = selective_scan_ws_bytes(a.rows.B, a.rows.N, a.rows.total, a.D, a.n, a.rows.cu != nullptr, sms);
    if (!workspace_ok(a.workspace, workspace_bytes, need) || !scan_apart(a, a.h0, need)) return GRET_ERR_INVALID_ARG;
    if (!device) return GRET_ERR_CUDA;
    return done(launch_selective_scan(a, sms, cu_stream(stream)));
}

size_t scan_workspace(const Rows& r, int D, int n, bool packed, gret_dtype io) {
    if (!type_ok(io) || scan_sizes(r, packed, D, n)) return 0;
    int sms = 148;
    device_info(nullptr, &sms);
    return selective_scan_ws_bytes(r.B, r.N, r.total, D, n, packed, sms);
}

// ---------------------------------------------------------------- residual norm
gret_status norm_check(const NormArgs& a) {
    if (!type_ok(a.io) || !type_ok(a.stream_type) || (a.io == GRET_F32 && a.stream_type != GRET_F32))
        return GRET_ERR_INVALID_ARG;
    if (!a.x || (!a.y && (a.gate || a.scale || a.w_post)) || (!a.y && !a.w_next)) return GRET_ERR_INVALID_ARG;
    if (a.T <= 0 || a.D <= 0 || !(a.eps >= 0.f) || !isfinite(a.eps)) return GRET_ERR_INVALID_ARG;
    if (!all_aligned(a.x, a.y, a.gate, a.scale, a.w_post, a.w_next, a.r, a.n)) return GRET_ERR_INVALID_ARG;
    if (a.D % kVec != 0 || a.D > kNormMaxChannels || a.T > 0x7fffffffLL) return GRET_ERR_UNSUPPORTED;
    if (!stride_ok(a.ldx, a.D, a.stream_type) || (a.y && !stride_ok(a.ldy, a.D, a.io)) ||
        (a.gate && !stride_ok(a.ldg, a.D, a.io)))
        return GRET_ERR_INVALID_ARG;
    return GRET_OK;
}

}  // namespace

extern "C" {

gret_status gret_short_conv(const void* x, long long ldx, const float* w, const float* bias, const void* tail0,
                            void* y, void* tail, int B, int N, int D, int K, gret_dtype io_dtype, gret_activation act,
                            gret_stream_t stream) {
    return conv(x, ldx, w, bias, tail0, y, tail, uniform(B, N), D, K, io_dtype, act, stream);
}

gret_status gret_short_conv_varlen(const void* x, long long ldx, const float* w, const float* bias, const void* tail0,
                                   const int* cu_seqlens, int num_seqs, int total_tokens, int max_seqlen, void* y,
                                   void* tail, int D, int K, gret_dtype io_dtype, gret_activation act,
                                   gret_stream_t stream) {
    if (!cu_seqlens) return GRET_ERR_INVALID_ARG;
    return conv(x, ldx, w, bias, tail0, y, tail, packed(cu_seqlens, num_seqs, max_seqlen, total_tokens), D, K,
                io_dtype, act, stream);
}

gret_status gret_short_conv_step(const void* x, long long ldx, const float* w, const float* bias, const void* tail_in,
                                 void* tail_out, void* y, int num_seqs, int D, int K, gret_dtype io_dtype,
                                 gret_activation act, gret_stream_t stream) {
    if (!all_set(tail_in, tail_out) || (act != GRET_ACT_NONE && act != GRET_ACT_SWISH)) return GRET_ERR_INVALID_ARG;
    const ConvArgs a = {x, ldx, w, bias, tail_in, y, tail_out, uniform(num_seqs, 1), D, K,
                        act == GRET_ACT_SWISH, io_dtype};
    if (gret_status e = conv_check(a)) return e;
    if (!conv_apart(a, tail_in == tail_out ? nullptr : tail_in)) return GRET_ERR_INVALID_ARG;
    return done(launch_short_conv_step(a, cu_stream(stream)));
}

size_t gret_selective_scan_workspace_size(int B, int N, int D, int n, gret_dtype io_dtype) {
    return scan_workspace(uniform(B, N), D, n, false, io_dtype);
}

gret_status gret_selective_scan(const void* u, long long ldu, const void* dt, long long lddt, const float* A,
                                const void* Bm, long long ldb, const void* Cm, long long ldc, const float* skip,
                                const void* z, long long ldz, const float* dt_bias, const float* h0, void* o,
                                float* h_final, int B, int N, int D, int n, gret_dtype io_dtype, void* workspace,
                                size_t workspace_bytes, gret_stream_t stream) {
    return scan(ScanArgs{u, dt, Bm, Cm, z, ldu, lddt, ldb, ldc, ldz, A, skip, dt_bias, h0, o, h_final,
                         uniform(B, N), D, n, io_dtype, workspace},
                workspace_bytes, stream);
}

size_t gret_selective_scan_varlen_workspace_size(int num_seqs, int total_tokens, int max_seqlen, int D, int n,
                                                 gret_dtype io_dtype) {
    return scan_workspace(packed(nullptr, num_seqs, max_seqlen, total_tokens), D, n, true, io_dtype);
}

gret_status gret_selective_scan_varlen(const void* u, long long ldu, const void* dt, long long lddt, const float* A,
                                       const void* Bm, long long ldb, const void* Cm, long long ldc, const float* skip,
                                       const void* z, long long ldz, const float* dt_bias, const float* h0,
                                       const int* cu_seqlens, int num_seqs, int total_tokens, int max_seqlen, void* o,
                                       float* h_final, int D, int n, gret_dtype io_dtype, void* workspace,
                                       size_t workspace_bytes, gret_stream_t stream) {
    if (!cu_seqlens) return GRET_ERR_INVALID_ARG;
    return scan(ScanArgs{u, dt, Bm, Cm, z, ldu, lddt, ldb, ldc, ldz, A, skip, dt_bias, h0, o, h_final,
                         packed(cu_seqlens, num_seqs, max_seqlen, total_tokens), D, n, io_dtype, workspace},
                workspace_bytes, stream);
}

gret_status gret_selective_step(const void* u, long long ldu, const void* dt, long long lddt, const float* A,
                                const void* Bm, long long ldb, const void* Cm, long long ldc, const float* skip,
                                const void* z, long long ldz, const float* dt_bias, const float* h_in, float* h_out,
                                void* o, int num_seqs, int D, int n, gret_dtype io_dtype, gret_stream_t stream) {
    if (!all_set(h_in, h_out)) return GRET_ERR_INVALID_ARG;
    const ScanArgs a = {u, dt, Bm, Cm, z, ldu, lddt, ldb, ldc, ldz, A, skip, dt_bias, h_in, o, h_out,
                        uniform(num_seqs, 1), D, n, io_dtype, nullptr};
    if (gret_status e = scan_check(a)) return e;
    if (!scan_apart(a, h_in == h_out ? nullptr : h_in, 0)) return GRET_ERR_INVALID_ARG;
    return done(launch_selective_step(a, cu_stream(stream)));
}

gret_status gret_residual_norm(const void* x, long long ldx, const void* y, long long ldy, const void* gate,
                               long long ldg, const float* scale, const float* w_post, const float* w_next, void* r,
                               void* n, long long T, int D, float eps, gret_dtype stream_dtype, gret_dtype io_dtype,
                               gret_stream_t stream) {
    const NormArgs a = {x, y, gate, ldx, ldy, ldg, scale, w_post, w_next, r, n, T, D, eps, stream_dtype, io_dtype};
    if (gret_status e = norm_check(a)) return e;
    if ((y && !r) || (w_next && !n)) return GRET_ERR_INVALID_ARG;
    // r may be x itself
    const bool in_place = y && r == x && ldx == D;
    if (!apart({{y ? r : nullptr, span(T, D, D, stream_dtype)}, {w_next ? n : nullptr, span(T, D, D, io_dtype)}},
               {{in_place ? nullptr : x, span(T, ldx, D, stream_dtype)}, {y, span(T, ldy, D, io_dtype)},
                {gate, span(T, ldg, D, io_dtype)}, {scale, floats(D)}, {w_post, floats(D)}, {w_next, floats(D)}}))
        return GRET_ERR_INVALID_ARG;
    int sms = 0;
    if (!device_info(nullptr, &sms)) return GRET_ERR_CUDA;
    return done(launch_residual_norm(a, sms, cu_stream(stream)));
}

size_t gret_short_conv_backward_workspace_size(int B, int N, int D, int K, gret_dtype io_dtype) {
    if (conv_sizes(uniform(B, N), D, K) || !type_ok(io_dtype)) return 0;
    int sms = 148;
    device_info(nullptr, &sms);
    return short_conv_backward_ws_bytes(B, N, D, K, sms);
}

gret_status gret_short_conv_backward(const void* x, long long ldx, const float* w, const float* bias,
                                     const void* tail0, const void* dy, const void* dtail, void* dx, float* dw,
                                     float* dbias, void* dtail0, int B, int N, int D, int K, gret_dtype io_dtype,
                                     gret_activation act, void* workspace, size_t workspace_bytes,
                                     gret_stream_t stream) {
    if (act != GRET_ACT_NONE && act != GRET_ACT_SWISH) return GRET_ERR_INVALID_ARG;
    if (!all_set(dy, dx) || !all_aligned(dy, dtail, dx, dw, dbias, dtail0)) return GRET_ERR_INVALID_ARG;
    ConvBackwardArgs g = {};
    g.f = ConvArgs{x, ldx, w, bias, tail0, dx, nullptr, uniform(B, N), D, K, act == GRET_ACT_SWISH, io_dtype};
    if (gret_status e = conv_check(g.f)) return e;
    int sms = 148;
    const bool device = device_info(nullptr, &sms);
    const size_t need = short_conv_backward_ws_bytes(B, N, D, K, sms);
    if (!workspace_ok(workspace, workspace_bytes, need)) return GRET_ERR_INVALID_ARG;
    if (!apart({conv_rows(g.f, dx, D), {dw, floats(D, K)}, {dbias, floats(D)}, conv_tail(g.f, dtail0), {workspace, need}},
               {conv_rows(g.f, x, ldx), {w, floats(D, K)}, {bias, floats(D)}, conv_tail(g.f, tail0),
                conv_rows(g.f, dy, D), conv_tail(g.f, dtail)}))
        return GRET_ERR_INVALID_ARG;
    if (!device) return GRET_ERR_CUDA;
    g.dy = dy; g.dtail = dtail; g.dx = dx; g.dtail0 = dtail0; g.dw = dw; g.dbias = dbias; g.workspace = workspace;
    return done(launch_short_conv_backward(g, sms, cu_stream(stream)));
}

size_t gret_selective_scan_backward_workspace_size(int B, int N, int D, int n, gret_dtype io_dtype) {
    if (scan_sizes(uniform(B, N), false, D, n) || !type_ok(io_dtype)) return 0;
    return selective_backward_ws_bytes(B, N, D, n);
}

gret_status gret_selective_scan_backward(const void* u, long long ldu, const void* dt, long long lddt, const float* A,
                                         const void* Bm, long long ldb, const void* Cm, long long ldc,
                                         const float* skip, const void* z, long long ldz, const float* dt_bias,
                                         const float* h0, const void* dout, const float* dh_final, void* du, void* ddt,
                                         float* dA, void* dBm, void* dCm, float* dskip, void* dz, float* ddt_bias,
                                         float* dh0, int B, int N, int D, int n, gret_dtype io_dtype, void* workspace,
                                         size_t workspace_bytes, gret_stream_t stream) {
    if (!all_set(dout, du, ddt, dA, dBm, dCm) || (z && !dz)) return GRET_ERR_INVALID_ARG;
    if (!all_aligned(dout, dh_final, du, ddt, dA, dBm, dCm, dskip, dz, ddt_bias, dh0)) return GRET_ERR_INVALID_ARG;
    ScanBackwardArgs g = {};
    g.f = ScanArgs{u, dt, Bm, Cm, z, ldu, lddt, ldb, ldc, ldz, A, skip, dt_bias, h0, du, nullptr,
                   uniform(B, N), D, n, io_dtype, nullptr};
    if (gret_status e = scan_check(g.f)) return e;
    const size_t need = selective_backward_ws_bytes(B, N, D, n);
    if (!workspace_ok(workspace, workspace_bytes, need)) return GRET_ERR_INVALID_ARG;
    const ScanArgs& f = g.f;
    if (!apart({scan_rows(f, du, D, D), scan_rows(f, ddt, D, D), scan_rows(f, z ? dz : nullptr, D, D),
                scan_rows(f, dBm, n, n), scan_rows(f, dCm, n, n), {dA, floats(D, n)}, {dskip, floats(D)},
                {ddt_bias, floats(D)}, scan_state(f, dh0), {workspace, need}},
               {scan_rows(f, u, ldu, D), scan_rows(f, dt, lddt, D), scan_rows(f, z, ldz, D), scan_rows(f, Bm, ldb, n),
                scan_rows(f, Cm, ldc, n), {A, floats(D, n)}, {skip, floats(D)}, {dt_bias, floats(D)}, scan_state(f, h0),
                scan_rows(f, dout, D, D), scan_state(f, dh_final)}))
        return GRET_ERR_INVALID_ARG;
    g.dout = dout; g.dh_final = dh_final; g.du = du; g.ddt = ddt; g.dBm = dBm; g.dCm = dCm; g.dz = dz;
    g.dA = dA; g.dskip = dskip; g.ddt_bias = ddt_bias; g.dh0 = dh0; g.workspace = workspace;
    return done(launch_selective_backward(g, cu_stream(stream)));
}

size_t gret_residual_norm_backward_workspace_size(long long T, int D) {
    if (T <= 0 || T > 0x7fffffffLL || D <= 0 || D % kVec != 0 || D > kNormMaxChannels) return 0;
    int sms = 148;
    device_info(nullptr, &sms);
    return residual_norm_backward_ws_bytes(T, D, sms);
}

gret_status gret_residual_norm_backward(const void* x, long long ldx, const void* y, long long ldy, const void* gate,
                                        long long ldg, const float* scale, const float* w_post, const float* w_next,
                                        const void* dr, const void* dn, void* dx, void* dy, void* dgate, float* dscale,
                                        float* dw_post, float* dw_next, long long T, int D, float eps,
                                        gret_dtype stream_dtype, gret_dtype io_dtype, void* workspace,
                                        size_t workspace_bytes, gret_stream_t stream) {
    NormBackwardArgs g = {};
    g.f = NormArgs{x, y, gate, ldx, ldy, ldg, scale, w_post, w_next, nullptr, nullptr, T, D, eps, stream_dtype, io_dtype};
    if (gret_status e = norm_check(g.f)) return e;
    if (!dx || (y && !dy) || (gate && !dgate) || (w_next != nullptr) != (dn != nullptr) || (!dr && !dn))
        return GRET_ERR_INVALID_ARG;
    if (!all_aligned(dr, dn, dx, dy, dgate, dscale, dw_post, dw_next)) return GRET_ERR_INVALID_ARG;
    int sms = 148;
    const bool device = device_info(&g.status, &sms);
    const size_t need = residual_norm_backward_ws_bytes(T, D, sms), stream_row = span(T, D, D, stream_dtype),
                 block_row = span(T, D, D, io_dtype);
    if (!workspace_ok(workspace, workspace_bytes, need)) return GRET_ERR_INVALID_ARG;
    if (!apart({{dx, stream_row}, {y ? dy : nullptr, block_row}, {gate ? dgate : nullptr, block_row}, {dscale, floats(D)},
                {dw_post, floats(D)}, {dw_next, floats(D)}, {workspace, need}},
               {{x, span(T, ldx, D, stream_dtype)}, {y, span(T, ldy, D, io_dtype)}, {gate, span(T, ldg, D, io_dtype)},
                {scale, floats(D)}, {w_post, floats(D)}, {w_next, floats(D)}, {dr, stream_row}, {dn, block_row}}))
        return GRET_ERR_INVALID_ARG;
    if (!device) return GRET_ERR_CUDA;
    g.dr = dr; g.dn = dn; g.dx = dx; g.dy = dy; g.dgate = dgate;
    g.dscale = dscale; g.dw_post = dw_post; g.dw_next = dw_next; g.workspace = workspace;
    g.fault = take_injected_timeout();
    return done(launch_residual_norm_backward(g, sms, cu_stream(stream)));
}

}  // extern "C"
