"""Host-side checks of the selective state space block's entry points: bad arguments are refused before any launch
(the pointers are never used, so this runs without a GPU)."""
import pytest
import torch

import gated_retention_sequence_b200 as gret

P, Q, R = 0x100000, 0x10000000, 0x20000000      # aligned addresses apart; validation fails before they are used
INVALID, UNSUPPORTED = gret.Status.ERR_INVALID_ARG, gret.Status.ERR_UNSUPPORTED
BF = gret.Dtype.BF16


@pytest.fixture(scope="module", autouse=True)
def lib():
    from gated_retention_sequence_b200 import build
    build.build()
    return gret.load()


CONV = dict(x=P, ldx=64, w=P, bias=None, tail0=None, y=Q, tail=None, B=2, N=5, D=64, K=4, io_dtype=BF,
            act=gret.Activation.SWISH, stream=None)
SCAN = dict(u=P, ldu=64, dt=P, lddt=64, A=P, Bm=P, ldb=16, Cm=P, ldc=16, skip=None, z=None, ldz=0, dt_bias=None, h0=None,
            o=Q, h_final=None, B=2, N=5, D=64, n=16, io_dtype=BF, workspace=None, workspace_bytes=0, stream=None)
NORM = dict(x=P, ldx=64, y=P, ldy=64, gate=None, ldg=0, scale=None, w_post=None, w_next=P, r=Q, n=R, T=3, D=64, eps=1e-5,
            stream_dtype=BF, io_dtype=BF, stream=None)

ROWS_BAD = [(dict(B=0), INVALID), (dict(N=0), INVALID), (dict(N=-1), INVALID), (dict(B=1 << 16, N=1 << 16), UNSUPPORTED)]


@pytest.mark.parametrize("over,expect", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(x=P + 2), INVALID),
    (dict(tail0=P + 8), INVALID), (dict(D=0), INVALID), (dict(io_dtype=7), INVALID), (dict(act=9), INVALID),
    (dict(ldx=63), INVALID), (dict(ldx=65), INVALID), (dict(ldx=-64), INVALID), (dict(D=60, ldx=64), UNSUPPORTED),
    (dict(K=1), UNSUPPORTED), (dict(K=5), UNSUPPORTED), (dict(K=0), INVALID),
    (dict(tail0=P, tail=P), INVALID), (dict(tail0=P, tail=P + 2 * 3 * 64 * 2 - 16), INVALID),
    (dict(y=P), INVALID), (dict(ldx=128, y=P + (9 * 128 + 64) * 2 - 16), INVALID)] + ROWS_BAD)
def test_conv_refuses(over, expect):
    assert gret.gret_short_conv(**dict(CONV, **over)) == expect


def test_conv_step_and_varlen_refuse():
    step = dict(x=P, ldx=64, w=P, bias=None, tail_in=P, tail_out=P, y=Q, num_seqs=2, D=64, K=4, io_dtype=BF, act=1,
                stream=None)
    for over in (dict(tail_in=None), dict(tail_out=None), dict(num_seqs=0), dict(tail_out=P + 16)):
        assert gret.gret_short_conv_step(**dict(step, **over)) == INVALID, over
    var = dict(x=P, ldx=64, w=P, bias=None, tail0=None, cu_seqlens=P, num_seqs=2, total_tokens=10, max_seqlen=6, y=Q,
               tail=None, D=64, K=4, io_dtype=BF, act=1, stream=None)
    for over in (dict(cu_seqlens=None), dict(cu_seqlens=P + 2), dict(num_seqs=0), dict(total_tokens=0),
                 dict(max_seqlen=0)):
        assert gret.gret_short_conv_varlen(**dict(var, **over)) == INVALID, over


@pytest.mark.parametrize("over,expect", [
    (dict(u=None), INVALID), (dict(dt=None), INVALID), (dict(A=None), INVALID), (dict(Bm=None), INVALID),
    (dict(Cm=None), INVALID), (dict(o=None), INVALID), (dict(A=P + 4), INVALID), (dict(z=P + 2, ldz=64), INVALID),
    (dict(z=P, ldz=0), INVALID), (dict(ldb=8), INVALID), (dict(ldc=17), INVALID), (dict(lddt=32), INVALID),
    (dict(o=P), INVALID), (dict(z=Q + 16, ldz=64), INVALID), (dict(Cm=Q + 10 * 64 * 2 - 16), INVALID),
    (dict(n=12), UNSUPPORTED), (dict(n=128), UNSUPPORTED), (dict(n=0), INVALID), (dict(D=60), UNSUPPORTED),
    (dict(D=65544, ldu=65544, lddt=65544), UNSUPPORTED), (dict(io_dtype=3), INVALID), (dict(h0=P, h_final=P), INVALID), (dict(h0=P, h_final=P + 2 * 64 * 16 * 4 - 16), INVALID),
    ] + ROWS_BAD)
def test_scan_refuses(over, expect):
    assert gret.gret_selective_scan(**dict(SCAN, **over)) == expect


def test_scan_step_and_varlen_refuse():
    step = {k: v for k, v in SCAN.items() if k not in ("h0", "h_final", "B", "N", "workspace", "workspace_bytes")}
    step.update(h_in=P, h_out=P, num_seqs=2)
    for over in (dict(h_in=None), dict(h_out=None), dict(num_seqs=0), dict(h_out=P + 64), dict(u=None)):
        assert gret.gret_selective_step(**dict(step, **over)) == INVALID, over
    var = {k: v for k, v in SCAN.items() if k not in ("B", "N")}
    var.update(cu_seqlens=P, num_seqs=2, total_tokens=9, max_seqlen=5)
    for over in (dict(cu_seqlens=None), dict(cu_seqlens=P + 1), dict(total_tokens=0), dict(max_seqlen=-1)):
        assert gret.gret_selective_scan_varlen(**dict(var, **over)) == INVALID, over
    assert gret.gret_selective_scan_varlen(**dict(var, num_seqs=1 << 30, total_tokens=1 << 30)) == UNSUPPORTED


@pytest.mark.parametrize("over,expect", [
    (dict(x=None), INVALID), (dict(r=None), INVALID), (dict(n=None), INVALID), (dict(y=None, w_next=None), INVALID),
    (dict(y=None, gate=P, ldg=64), INVALID), (dict(y=None, scale=P), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(T=0), INVALID), (dict(D=0), INVALID), (dict(ldx=60), INVALID),
    (dict(gate=P, ldg=0), INVALID), (dict(n=Q), INVALID), (dict(n=P), INVALID), (dict(r=P + 16), INVALID),
    (dict(x=Q, ldx=72), INVALID), (dict(y=Q), INVALID), (dict(gate=R + 128, ldg=64), INVALID), (dict(y=P + 4), INVALID), (dict(io_dtype=gret.Dtype.F32), INVALID),
    (dict(D=8200, ldx=8200, ldy=8200), UNSUPPORTED), (dict(D=60), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED)])
def test_norm_refuses(over, expect):
    assert gret.gret_residual_norm(**dict(NORM, **over)) == expect


def test_backwards_refuse():
    ws = dict(workspace=P, workspace_bytes=1 << 40)
    conv = dict({k: v for k, v in CONV.items() if k not in ("y", "tail")}, dy=P, dtail=None, dx=Q, dw=P, dbias=None,
                dtail0=None, **ws)
    for over in (dict(dy=None), dict(dx=None), dict(dw=P + 4), dict(dtail=P + 8), dict(workspace=None),
                 dict(workspace=P + 128), dict(workspace_bytes=0), dict(act=4), dict(N=0)):
        assert gret.gret_short_conv_backward(**dict(conv, **over)) == INVALID, over
    assert gret.gret_short_conv_backward(**dict(conv, K=7)) == UNSUPPORTED
    scan = dict({k: v for k, v in SCAN.items() if k not in ("o", "h_final")}, dout=P, dh_final=None, du=Q, ddt=P, dA=P,
                dBm=P, dCm=P, dskip=None, dz=None, ddt_bias=None, dh0=None, **ws)
    for over in (dict(dout=None), dict(du=None), dict(ddt=None), dict(dA=None), dict(dBm=None), dict(dCm=None),
                 dict(z=P, ldz=64), dict(dh0=P + 4), dict(workspace=None), dict(workspace_bytes=0), dict(B=0)):
        assert gret.gret_selective_scan_backward(**dict(scan, **over)) == INVALID, over
    assert gret.gret_selective_scan_backward(**dict(scan, n=24)) == UNSUPPORTED
    norm = dict({k: v for k, v in NORM.items() if k not in ("r", "n")}, dr=P, dn=P, dx=P, dy=P, dgate=None, dscale=None,
                dw_post=None, dw_next=None, **ws)
    for over in (dict(dx=None), dict(dy=None), dict(dn=None), dict(w_next=None), dict(gate=P, ldg=64),
                 dict(dr=P + 2), dict(workspace_bytes=0), dict(T=0), dict(eps=float("inf"))):
        assert gret.gret_residual_norm_backward(**dict(norm, **over)) == INVALID, over
    assert gret.gret_residual_norm_backward(**dict(norm, D=8200, ldx=8200, ldy=8200)) == UNSUPPORTED


def test_workspace_sizes_of_refused_arguments():
    assert gret.gret_selective_scan_workspace_size(0, 5, 64, 16, BF) == 0
    assert gret.gret_selective_scan_workspace_size(1, 5, 64, 12, BF) == 0
    assert gret.gret_selective_scan_varlen_workspace_size(2, 0, 5, 64, 16, BF) == 0
    assert gret.gret_selective_scan_backward_workspace_size(1, 0, 64, 16, BF) == 0
    assert gret.gret_short_conv_backward_workspace_size(1, 5, 64, 5, BF) == 0
    assert gret.gret_residual_norm_backward_workspace_size(5, 60) == 0


def test_python_checks():
    x = torch.zeros(2, 5, 64)
    w = torch.zeros(64, 4)
    with pytest.raises(ValueError, match="CUDA"):
        gret.short_conv(x, w)
    with pytest.raises(TypeError, match="unsupported io dtype"):
        gret.short_conv(x.half(), w)
    with pytest.raises(ValueError, match="go with y"):
        gret.residual_norm(x, gate=x)
    with pytest.raises(ValueError, match="y or w_next"):
        gret.residual_norm(x)


def test_row_strides():
    """What a row stride may be: dense rows, equally far apart, on 16-byte boundaries."""
    from gated_retention_sequence_b200.block import _rows

    class Cuda(torch.Tensor):
        is_cuda = True

    def ld(t):
        t = t.as_subclass(Cuda)
        return _rows(t, "x", t.dtype, t.shape, t.device)

    wide = torch.zeros(4, 6, 64, dtype=torch.bfloat16)
    assert ld(wide) == 64 and ld(wide[..., 16:32]) == 64 and ld(wide[:1, :, :8]) == 64
    assert ld(wide[:, ::2]) == 128 and ld(wide[:, :1, :8]) == 6 * 64 and ld(wide[:1, :1, 8:16]) == 8 and ld(wide[0, ::2, :8]) == 128
    for bad, what in ((wide[:, :4:2], "equally"), (wide[:, :3, :8], "equally"), (wide.transpose(1, 2), "dense"),
                      (wide[..., ::2], "dense"), (wide[:1].expand(4, 6, 64), "equally"),
                      (torch.zeros(4, 12, dtype=torch.bfloat16)[:, :8], "16-byte")):
        with pytest.raises(ValueError, match=what):
            ld(bad)


@pytest.mark.parametrize("shape", [(6, 64), (4, 6, 64), (4, 3, 5, 64), (1, 6, 64), (4, 1, 64)])
def test_broadcast_rows_are_refused(shape):
    """A tensor broadcast along rows has fewer rows in memory than its shape says, wherever the dimension stands."""
    from gated_retention_sequence_b200.block import _rows

    class Cuda(torch.Tensor):
        is_cuda = True

    def ld(t):
        t = t.as_subclass(Cuda)
        return _rows(t, "x", t.dtype, t.shape, t.device)

    outer = len(shape) - 1
    for mask in range(1, 1 << outer):
        small = [1 if mask >> i & 1 else shape[i] for i in range(outer)]
        broadcast = tuple(small) != shape[:-1]
        for t in (torch.zeros(*small, 64), torch.zeros(*small, 96)[..., 16:80], torch.zeros(*small, 5, 64)[..., 2, :]):
            if broadcast:
                with pytest.raises(ValueError, match="equally"):
                    ld(t.expand(shape))
        for i in range(outer):                  # cut from a tensor whose entries would otherwise be rows of their own
            if mask >> i & 1 and shape[i] > 1:
                with pytest.raises(ValueError, match="equally"):
                    ld(torch.zeros(shape).narrow(i, 0, 1).expand(shape))
    assert ld(torch.zeros(shape)) == 64


def test_no_call_takes_broadcast_rows():
    """Every activation of every call is checked."""
    class Cuda(torch.Tensor):
        is_cuda = True

    def cuda(*s):
        return torch.zeros(s).as_subclass(Cuda)

    B, N, D, n = 2, 5, 64, 16
    flat = cuda(B, 1, D).expand(B, N, D)
    x, w, A = cuda(B, N, D), cuda(D, 4), cuda(D, n)
    few, flatn = cuda(B, N, n), cuda(B, 1, n).expand(B, N, n)
    scan = dict(u=x, dt=x, A=A, B=few, C=few, z=x)
    for k, v in (("u", flat), ("dt", flat), ("B", flatn), ("C", flatn), ("z", flat)):
        for call in (gret.selective_scan, lambda **q: gret.selective_scan_backward(do=x, **q)):
            with pytest.raises(ValueError, match=f"rows of {k} must"):
                call(**dict(scan, **{k: v}))
    norm = dict(x=x, y=x, gate=x, w_next=cuda(D))
    for k in ("x", "y", "gate"):
        for call in (gret.residual_norm, lambda **q: gret.residual_norm_backward(dn=x, **q)):
            with pytest.raises(ValueError, match=f"rows of {k} must"):
                call(**dict(norm, **{k: flat}))
    for call in (gret.short_conv, lambda x, w: gret.short_conv_backward(x, w, None, x)):
        with pytest.raises(ValueError, match="rows of x must"):
            call(flat, w)
    flat, flatn = cuda(1, D).expand(N, D), cuda(1, n).expand(N, n)
    cu = torch.zeros(3, dtype=torch.int32).as_subclass(Cuda)
    h, tail, x, few = cuda(N, D, n), cuda(N, 3, D), cuda(N, D), cuda(N, n)
    scan = dict(u=x, dt=x, A=A, B=few, C=few, z=x)
    for k, v in (("u", flat), ("dt", flat), ("B", flatn), ("C", flatn), ("z", flat)):
        for call in (lambda **q: gret.selective_scan_varlen(cu_seqlens=cu, max_seqlen=3, **q),
                     lambda **q: gret.selective_step(h=h, **q)):
            with pytest.raises(ValueError, match=f"rows of {k} must"):
                call(**dict(scan, **{k: v}))
    for call in (lambda: gret.short_conv_varlen(flat, w, None, cu, 3), lambda: gret.short_conv_step(flat, w, None, tail)):
        with pytest.raises(ValueError, match="rows of x must"):
            call()


def test_workspace_must_be_contiguous():
    """A broadcast or strided workspace has other bytes between its entries, or fewer than it counts."""
    from gated_retention_sequence_b200.block import _workspace

    class Cuda(torch.Tensor):
        is_cuda = True

    dense = torch.zeros(1024, dtype=torch.uint8).as_subclass(Cuda)
    assert _workspace(dense, 1024, dense.device) is dense
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(1024), torch.zeros(2048, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            _workspace(bad.as_subclass(Cuda), 1024, dense.device)


MOST = 2 ** 31 - 2 ** 20                         # rows that no call takes


def test_counts_next_to_31_bits():
    """Row counts next to the limit neither wrap nor pass it."""
    assert gret.gret_short_conv(**dict(CONV, B=1, N=MOST)) == UNSUPPORTED
    assert gret.gret_selective_scan(**dict(SCAN, B=1, N=2 ** 31 - 1)) == UNSUPPORTED
    back = {k: v for k, v in CONV.items() if k not in ("y", "tail")}
    assert gret.gret_short_conv_backward(**dict(back, B=1, N=MOST, dy=P, dtail=None, dx=Q, dw=P, dbias=None, dtail0=None,
                                                workspace=P, workspace_bytes=1 << 50)) == UNSUPPORTED
    # the longest sequence that is taken: some 512 segments of 2^22 rows and a state of 17 words each
    size = gret.gret_selective_scan_workspace_size(1, MOST - 1, 128, 16, BF)
    assert 0 < size < 1024 * 128 * 17 * 4
    assert 0 < gret.gret_selective_scan_varlen_workspace_size(1, MOST - 2, 2 ** 31 - 1, 128, 16, BF) < 1024 * 128 * 17 * 4
    assert gret.gret_selective_scan_workspace_size(1, MOST, 128, 16, BF) == 0
    assert gret.gret_selective_scan_varlen_workspace_size(2, MOST - 2, 5, 128, 16, BF) == 0


def test_longest_sequence_is_a_bound_from_above():
    """A bound past all rows says no more than the rows do."""
    for T in (300, 5000):
        want = gret.gret_selective_scan_varlen_workspace_size(4, T, T, 64, 16, BF)
        for bound in (T + 1, 1 << 20, 2 ** 31 - 1):
            assert gret.gret_selective_scan_varlen_workspace_size(4, T, bound, 64, 16, BF) == want


def test_python_sizes_past_31_bits():
    """Sizes that do not fit the library's counts are refused, not cut."""
    class Cuda(torch.Tensor):
        is_cuda = True

    def cuda(*s, dtype=torch.bfloat16):
        return torch.empty(s, dtype=dtype, device="meta").as_subclass(Cuda)

    N = 2 ** 32 + 5
    x, few, w, A = cuda(1, N, 8), cuda(1, N, 16), cuda(8, 4, dtype=torch.float32), cuda(8, 16, dtype=torch.float32)
    for call in (lambda: gret.short_conv(x, w), lambda: gret.short_conv_backward(x, w, None, x),
                 lambda: gret.selective_scan(x, x, A, few, few), lambda: gret.residual_norm(x, w_next=w[:, 0])):
        with pytest.raises(gret.GretError) as e:
            call()
        assert e.value.status == UNSUPPORTED


# Every pointer of every call: its bytes, and whether the call writes there.  Pointers may be moved onto one another.
def _regions():
    B, N, D, K, n, T = 2, 40, 64, 4, 16, 80
    row, tail, state, par, ab = T * D * 2, B * (K - 1) * D * 2, B * D * n * 4, D * 4, T * n * 2
    conv_in = dict(x=row, w=D * K * 4, bias=par, tail0=tail)
    scan_in = dict(u=row, dt=row, A=D * n * 4, Bm=ab, Cm=ab, skip=par, z=row, dt_bias=par, h0=state)
    norm_in = dict(x=row, y=row, gate=row, scale=par, w_post=par, w_next=par)
    lds = dict(ldu=D, lddt=D, ldb=n, ldc=n, ldz=D)
    conv = dict(ldx=D, D=D, K=K, io_dtype=BF, act=1, stream=None)
    scan = dict(lds, D=D, n=n, io_dtype=BF, stream=None)
    norm = dict(ldx=D, ldy=D, ldg=D, T=T, D=D, eps=1e-5, stream_dtype=BF, io_dtype=BF, stream=None)
    cu = dict(cu_seqlens=(B + 1) * 4)
    packed = dict(num_seqs=B, total_tokens=T, max_seqlen=N)
    step_row, step_ab = B * D * 2, B * n * 2
    size = gret.gret_selective_scan_workspace_size
    # few channels and many tokens, so that the sequence is cut and needs a workspace
    cut = dict(lds, ldu=8, lddt=8, ldz=8, B=1, N=4000, D=8, n=n, io_dtype=BF, stream=None)
    cut_row, cut_ab, cut_ws = 4000 * 8 * 2, 4000 * n * 2, size(1, 4000, 8, n, BF)
    cut_in = dict(u=cut_row, dt=cut_row, A=8 * n * 4, Bm=cut_ab, Cm=cut_ab, skip=32, z=cut_row, dt_bias=32, h0=8 * n * 4)
    conv_ws = gret.gret_short_conv_backward_workspace_size(B, N, D, K, BF)
    scan_ws = gret.gret_selective_scan_backward_workspace_size(B, N, D, n, BF)
    norm_ws = gret.gret_residual_norm_backward_workspace_size(T, D)
    assert cut_ws and conv_ws and scan_ws and norm_ws
    return {
        "conv": (gret.gret_short_conv, conv_in, dict(y=row, tail=tail), dict(conv, B=B, N=N)),
        "conv_varlen": (gret.gret_short_conv_varlen, dict(conv_in, **cu), dict(y=row, tail=tail), dict(conv, **packed)),
        "conv_step": (gret.gret_short_conv_step, dict(x=step_row, w=D * K * 4, bias=par, tail_in=tail),
                      dict(y=step_row, tail_out=tail), dict(conv, num_seqs=B)),
        "conv_backward": (gret.gret_short_conv_backward, dict(conv_in, dy=row, dtail=tail),
                          dict(dx=row, dw=D * K * 4, dbias=par, dtail0=tail, workspace=conv_ws),
                          dict(conv, B=B, N=N, workspace_bytes=conv_ws)),
        "scan": (gret.gret_selective_scan, cut_in, dict(o=cut_row, h_final=8 * n * 4, workspace=cut_ws),
                 dict(cut, workspace_bytes=cut_ws)),
        "scan_varlen": (gret.gret_selective_scan_varlen, dict(scan_in, **cu), dict(o=row, h_final=state),
                        dict(scan, **packed, workspace=1 << 40, workspace_bytes=1 << 30)),
        "step": (gret.gret_selective_step,
                 dict(u=step_row, dt=step_row, A=D * n * 4, Bm=step_ab, Cm=step_ab, skip=par, z=step_row, dt_bias=par,
                      h_in=state), dict(o=step_row, h_out=state), dict(scan, num_seqs=B)),
        "scan_backward": (gret.gret_selective_scan_backward, dict(scan_in, dout=row, dh_final=state),
                          dict(du=row, ddt=row, dA=D * n * 4, dBm=ab, dCm=ab, dskip=par, dz=row, ddt_bias=par, dh0=state,
                               workspace=scan_ws), dict(scan, B=B, N=N, workspace_bytes=scan_ws)),
        "norm": (gret.gret_residual_norm, norm_in, dict(r=row, n=row), norm),
        "norm_backward": (gret.gret_residual_norm_backward, dict(norm_in, dr=row, dn=row),
                          dict(dx=row, dy=row, dgate=row, dscale=par, dw_post=par, dw_next=par, workspace=norm_ws),
                          dict(norm, workspace_bytes=norm_ws)),
    }


IN_PLACE = {("norm", "r", "x"), ("conv_step", "tail_out", "tail_in"), ("step", "h_out", "h_in")}


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers name no memory: only where nothing can be launched")
@pytest.mark.parametrize("name", ["conv", "conv_varlen", "conv_step", "conv_backward", "scan", "scan_varlen", "step",
                                  "scan_backward", "norm", "norm_backward"])
def test_outputs_apart_from_inputs_and_one_another(name):
    """An output that meets an input or another output by 16 bytes is refused, one that ends where it begins is not."""
    call, inputs, outputs, rest = _regions()[name]
    sizes = dict(inputs, **outputs)
    at = {k: (i + 1) << 28 for i, k in enumerate(sizes)}
    ok = gret.Status.ERR_CUDA                    # past all checks: there is no device to launch on
    assert call(**at, **rest) == ok
    for out in outputs:
        for other in sizes:
            if other == out:
                continue
            step = 256 if out == "workspace" else 16
            behind, before = at[other] + sizes[other], at[other] - sizes[out]
            near = behind - 1 & -step            # the last place that still meets it
            assert call(**dict(at, **{out: near}), **rest) == INVALID, (out, other)
            assert call(**dict(at, **{out: -(-behind // step) * step}), **rest) == ok, (out, other)
            assert call(**dict(at, **{out: before & -step}), **rest) == ok, (out, other)
            if sizes[out] >= step:
                assert call(**dict(at, **{out: (before & -step) + step}), **rest) == INVALID, (out, other)
            same = dict(at, **{out: at[other]})
            assert call(**same, **rest) == (ok if (name, out, other) in IN_PLACE else INVALID), (out, other)


def test_norm_buffers_that_nothing_would_write_are_refused():
    class Cuda(torch.Tensor):
        is_cuda = True

    x, other, w = (torch.zeros(s).as_subclass(Cuda) for s in ((3, 64), (3, 64), (64,)))
    with pytest.raises(ValueError, match="n goes with w_next"):
        gret.residual_norm(x, y=other, n=torch.zeros(3, 64).as_subclass(Cuda))
    with pytest.raises(ValueError, match="r goes with y"):
        gret.residual_norm(x, w_next=w, r=other)


def test_stream_of_another_device_is_refused():
    """A launch would go to the stream's device, with pointers of the tensors'."""
    from types import SimpleNamespace

    from gated_retention_sequence_b200.block import _on

    with pytest.raises(ValueError, match="stream is on cuda:1"):
        _on(torch.device("cuda", 0), SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0))


@pytest.mark.parametrize("D,B,N", [(65544, 1, 4000), (1 << 24, 1, 400), (64, 1 << 16, 1 << 16), (65536, 1 << 18, 2),
                                   (60, 2, 4000), (0, 2, 4000), (-64, 2, 4000)])
def test_workspace_sizes_are_zero_where_the_call_is_refused(D, B, N):
    """What a call refuses needs no memory: a caller that asks first would else allocate it."""
    ld = max(D, 8) * 4
    over = dict(B=B, N=N, D=D, n=64, ldu=ld, lddt=ld, ldb=64, ldc=64)
    assert gret.gret_selective_scan(**dict(SCAN, **over)) in (INVALID, UNSUPPORTED)
    assert gret.gret_selective_scan_workspace_size(B, N, D, 64, BF) == 0
    assert gret.gret_selective_scan_backward_workspace_size(B, N, D, 64, BF) == 0
    assert gret.gret_selective_scan_varlen_workspace_size(B, min(B * N, 2 ** 31 - 1), N, D, 64, BF) == 0
    if (D, B) != (65536, 1 << 18):
        assert gret.gret_short_conv_backward_workspace_size(B, N, D, 4, BF) == 0
    assert gret.gret_residual_norm_backward_workspace_size(1 << 31, 64) == 0
