"""GPU parity of the selective state space block's operators with the 64-bit oracle, element by element within the
error bound that the oracle carries (``oracle/block_oracle.py``)."""
import numpy as np
import pytest
import torch

import gated_retention_sequence_b200 as gret
import gret_inputs as gi
from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_retention_sequence_b200 import build
    build.build()
    gret.load()


def draw(tid, shape, io="f32", mean=0.0, std=1.0, seed=91):
    """A seeded normal tensor on the GPU."""
    n = int(np.prod(shape))
    flat = gi.random_unit(seed, tid, (n,), mean, std * std, io) if n else torch.empty(0, dtype=TYPES[io])
    return flat.view(shape).cuda()


def columns(t, left=8, right=16):
    """The same values as columns of a wider tensor, whose other columns are NaN."""
    wide = torch.full(t.shape[:-1] + (left + t.shape[-1] + right,), float("nan"), dtype=t.dtype, device=t.device)
    view = wide[..., left:left + t.shape[-1]]
    view.copy_(t)
    return view


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ short convolution
def conv_inputs(io, rows, D, K, seqs, seed=1):
    return dict(x=draw(1, (rows, D), io, seed=seed), w=draw(2, (D, K), std=0.5, seed=seed), bias=draw(3, (D,), seed=seed),
                tail0=draw(4, (seqs, K - 1, D), io, seed=seed))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("B,N,D", [(1, 1, 8), (3, 2, 72), (2, 33, 264), (1, 131, 1032)])
def test_conv_prompts(io, K, B, N, D):
    p = conv_inputs(io, B * N, D, K, B)
    y, tail = gret.short_conv(p["x"].view(B, N, D), p["w"], p["bias"], tail0=p["tail0"])
    for b in range(B):
        ry, rt = bo.short_conv(p["x"][b * N:(b + 1) * N], p["w"], p["bias"], p["tail0"][b])
        bo.check(y[b], ry, io, f"y of sequence {b}")
        assert (tail[b].double().cpu().numpy() == rt.v).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_conv_from_zero_without_bias_or_activation(io):
    B, N, D = 2, 40, 40
    p = conv_inputs(io, B * N, D, 4, B)
    x = columns(p["x"].view(B, N, D))
    y, tail = gret.short_conv(x, p["w"], activation="none", want_tail=False)
    assert tail is None
    for b in range(B):
        bo.check(y[b], bo.short_conv(x[b], p["w"], swish=False)[0], io)


LENS = [[1], [5, 0, 1, 33, 64, 2], [0, 0, 3], [300, 1, 0, 31], [2] * 70, [0, 1, 4] * 100]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens", LENS)
def test_conv_packed(io, lens):
    D, K, T = 136, 4, sum(lens) + 3                 # three rows behind the last sequence
    p = conv_inputs(io, T, D, K, len(lens))
    y = torch.full((T, D), 7.0, dtype=TYPES[io], device="cuda")
    _, tail = gret.short_conv_varlen(columns(p["x"]), p["w"], p["bias"], offsets(lens), max(lens), tail0=p["tail0"], y=y)
    at = 0
    for b, n in enumerate(lens):
        ry, rt = bo.short_conv(p["x"][at:at + n], p["w"], p["bias"], p["tail0"][b])
        bo.check(y[at:at + n], ry, io, f"y of sequence {b}")
        assert (tail[b].double().cpu().numpy() == rt.v).all()
        at += n
    assert (y[at:] == 7).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("S,D", [(1, 8), (5, 264), (129, 72)])
def test_conv_step(io, K, S, D):
    p = conv_inputs(io, S, D, K, S)
    apart = torch.empty_like(p["tail0"])
    y, t = gret.short_conv_step(columns(p["x"]), p["w"], p["bias"], p["tail0"], tail_out=apart)
    assert t is apart
    for b in range(S):
        ry, rt = bo.short_conv(p["x"][b:b + 1], p["w"], p["bias"], p["tail0"][b])
        bo.check(y[b:b + 1], ry, io)
        assert (t[b].double().cpu().numpy() == rt.v).all()
    y2, t2 = gret.short_conv_step(p["x"], p["w"], p["bias"], p["tail0"])          # in place
    assert t2 is p["tail0"] and torch.equal(t2, apart) and torch.equal(y, y2)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("B,N,D", [(1, 1, 8), (3, 2, 72), (2, 65, 264), (1, 300, 136), (20, 7, 8)])
def test_conv_backward(io, K, B, N, D):
    p = conv_inputs(io, B * N, D, K, B)
    dy, dtail = draw(5, (B, N, D), io), draw(6, (B, K - 1, D), io)
    g = gret.short_conv_backward(columns(p["x"].view(B, N, D)), p["w"], p["bias"], dy, tail0=p["tail0"], dtail=dtail)
    total = None
    for b in range(B):
        want = bo.short_conv(p["x"][b * N:(b + 1) * N], p["w"], p["bias"], p["tail0"][b], dy=dy[b], dtail=dtail[b])
        bo.check(g["dx"][b], want["dx"], io, f"dx of sequence {b}")
        bo.check(g["dtail0"][b], want["dtail0"], io, f"dtail0 of sequence {b}")
        part = {k: want[k] for k in ("dw", "dbias")}
        total = part if total is None else {k: total[k] + part[k] for k in part}
    for k, v in total.items():
        bo.check(g[k], v, "f32", k)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_conv_backward_left_out(io):
    p = conv_inputs(io, 90, 40, 4, 1)
    dy = draw(5, (1, 90, 40), io)
    g = gret.short_conv_backward(p["x"][None], p["w"], None, dy, activation="none")
    want = bo.short_conv(p["x"], p["w"], swish=False, dy=dy[0])
    assert g["dbias"] is None and g["dtail0"] is None
    bo.check(g["dx"][0], want["dx"], io, "dx")
    bo.check(g["dw"], want["dw"], "f32", "dw")


# --------------------------------------------------------------- selective scan
def scan_inputs(io, rows, D, n, seqs, seed=2):
    return dict(u=draw(1, (rows, D), io, seed=seed), dt=draw(2, (rows, D), io, seed=seed),
                A=-torch.exp(draw(3, (D, n), seed=seed)), B=draw(4, (rows, n), io, seed=seed),
                C=draw(5, (rows, n), io, seed=seed), skip=draw(6, (D,), seed=seed), z=draw(7, (rows, D), io, seed=seed),
                dt_bias=draw(8, (D,), mean=-3.0, seed=seed), h0=draw(9, (seqs, D, n), seed=seed))


ROWS = ("u", "dt", "B", "C", "z")


def scan_rows(p, a, b, s):
    q = {k: v[a:b] if k in ROWS and v is not None else v for k, v in p.items()}
    if q["h0"] is not None:
        q["h0"] = q["h0"][s]
    return q


def scan_call(p, B, N, **kw):
    q = {k: v.unflatten(0, (B, N)) if k in ROWS and v is not None else v for k, v in p.items()}
    return gret.selective_scan(**q, **kw)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
@pytest.mark.parametrize("B,N,D", [(1, 1, 8), (2, 17, 72), (1, 200, 40)])
def test_scan_prompts(io, n, B, N, D):
    p = scan_inputs(io, B * N, D, n, B)
    o, h = scan_call(p, B, N)
    for b in range(B):
        ro, rh = bo.selective_scan(**scan_rows(p, b * N, (b + 1) * N, b))
        bo.check(o[b], ro, io, f"o of sequence {b}")
        bo.check(h[b], rh, "f32", f"h of sequence {b}")


@pytest.mark.parametrize("n", [8, 16, 32, 64])
@pytest.mark.parametrize("N", [700, 1200])
def test_scan_prompts_cut(n, N):
    # few channels: the sequences are cut, into few segments and into many, and joined in their two ways
    B, D = 3, 16
    assert gret.gret_selective_scan_workspace_size(B, N, D, n, gret.Dtype.F32) > 0
    p = scan_inputs("f32", B * N, D, n, B)
    o, h = scan_call(p, B, N)
    for b in range(B):
        ro, rh = bo.selective_scan(**scan_rows(p, b * N, (b + 1) * N, b))
        bo.check(o[b], ro, "f32", f"o of sequence {b}")
        bo.check(h[b], rh, "f32", f"h of sequence {b}")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("without", ["skip", "z", "dt_bias", "h0"])
def test_scan_left_out_and_strided(io, without):
    B, N, D, n = 3, 50, 264, 16
    p = scan_inputs(io, B * N, D, n, B)
    p[without] = None
    q = {k: columns(v) if k in ROWS and v is not None else v for k, v in p.items()}
    o, h = scan_call(q, B, N)
    for b in range(B):
        ro, rh = bo.selective_scan(**scan_rows(p, b * N, (b + 1) * N, b))
        bo.check(o[b], ro, io)
        bo.check(h[b], rh, "f32")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("n", [16, 64])
def test_scan_packed(io, lens, n):
    D, T = 72, sum(lens) + 5
    p = scan_inputs(io, T, D, n, len(lens))
    o = torch.full((T, D), 7.0, dtype=TYPES[io], device="cuda")
    _, h = gret.selective_scan_varlen(**p, cu_seqlens=offsets(lens), max_seqlen=max(lens), o=o)
    at = 0
    for b, m in enumerate(lens):
        if m:
            ro, rh = bo.selective_scan(**scan_rows(p, at, at + m, b))
            bo.check(o[at:at + m], ro, io, f"o of sequence {b}")
            bo.check(h[b], rh, "f32", f"h of sequence {b}")
        else:
            assert torch.equal(h[b], p["h0"][b])
        at += m
    assert (o[at:] == 7).all()


def test_scan_long_and_cut():
    # long enough for the sequence to be cut into segments, which are joined again; few channels
    N, D, n = 3000, 16, 16
    p = scan_inputs("f32", N, D, n, 1)
    o, h = scan_call(p, 1, N)
    ro, rh = bo.selective_scan(**scan_rows(p, 0, N, 0))
    bo.check(o[0], ro, "f32")
    bo.check(h[0], rh, "f32")
    # the same tokens as two sequences of one packed batch
    cu = offsets([1700, 1300])
    h0 = torch.cat([p["h0"], p["h0"]])
    o2, h2 = gret.selective_scan_varlen(**dict(p, h0=h0), cu_seqlens=cu, max_seqlen=1700)
    for b, (a, e) in enumerate([(0, 1700), (1700, 3000)]):
        ro, rh = bo.selective_scan(**scan_rows(dict(p, h0=h0), a, e, b))
        bo.check(o2[a:e], ro, "f32")
        bo.check(h2[b], rh, "f32")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
def test_scan_packed_and_cut(io, n):
    # long sequences among empty and short ones, few channels: cut into segments
    lens, D = [700, 0, 1500, 64, 1, 0, 333], 24
    T = sum(lens) + 2
    assert gret.gret_selective_scan_varlen_workspace_size(len(lens), T, max(lens), D, n, gret.Dtype.BF16) > 0
    p = scan_inputs(io, T, D, n, len(lens))
    o = torch.full((T, D), 7.0, dtype=TYPES[io], device="cuda")
    _, h = gret.selective_scan_varlen(**p, cu_seqlens=offsets(lens), max_seqlen=max(lens), o=o)
    at = 0
    for b, m in enumerate(lens):
        if m:
            ro, rh = bo.selective_scan(**scan_rows(p, at, at + m, b))
            bo.check(o[at:at + m], ro, io, f"o of sequence {b}")
            bo.check(h[b], rh, "f32", f"h of sequence {b}")
        else:
            assert torch.equal(h[b], p["h0"][b])
        at += m
    assert (o[at:] == 7).all()


def test_offsets_out_of_order():
    # offsets that are no partition: nothing outside the rows they name is written, and no error is left behind
    T, D, n = 400, 24, 16
    p = scan_inputs("f32", T, D, n, 5)
    c = conv_inputs("f32", T, D, 4, 5)
    o = torch.full((T + 8, D), 7.0, device="cuda")
    y = torch.full((T + 8, D), 7.0, device="cuda")
    for cu in ([0, 900, 100, 380, -5, 390], [-3, -2, -1, 0, 0, 0], [400, 300, 200, 100, 50, 0], [2 ** 31 - 1] * 6):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        gret.selective_scan_varlen(**p, cu_seqlens=cu, max_seqlen=T, o=o[:T])
        gret.short_conv_varlen(c["x"], c["w"], c["bias"], cu, T, tail0=c["tail0"], y=y[:T])
        assert (o[T:] == 7).all() and (y[T:] == 7).all()
    gret.check_device_status()


def test_sequences_longer_than_max_seqlen_are_not_walked_on():
    lens, D, n = [50, 30], 24, 16
    p = scan_inputs("f32", 80, D, n, 2)
    o = torch.full((80, D), 7.0, device="cuda")
    _, h = gret.selective_scan_varlen(**p, cu_seqlens=offsets(lens), max_seqlen=40, o=o)
    ro, rh = bo.selective_scan(**scan_rows(p, 0, 40, 0))
    bo.check(o[:40], ro, "f32")
    bo.check(h[0], rh, "f32")
    assert (o[40:50] == 7).all()
    bo.check(o[50:], bo.selective_scan(**scan_rows(p, 50, 80, 1))[0], "f32")


def test_values_outside_the_rows_do_not_matter():
    # NaN and infinity in rows behind the last sequence and in the states of other sequences stay where they are
    lens, D, n = [37, 90], 24, 16
    T = sum(lens) + 40
    p = scan_inputs("bf16", T, D, n, 2)
    c = conv_inputs("bf16", T, D, 4, 2)
    cu = offsets(lens)
    want, wh = gret.selective_scan_varlen(**p, cu_seqlens=cu, max_seqlen=90)
    wy, _ = gret.short_conv_varlen(c["x"], c["w"], c["bias"], cu, 90, tail0=c["tail0"])
    for k in ROWS:
        p[k][sum(lens):] = float("nan")
    c["x"][sum(lens):] = float("inf")
    p["h0"][1] = float("inf")
    c["tail0"][1] = float("nan")
    got, gh = gret.selective_scan_varlen(**p, cu_seqlens=cu, max_seqlen=90)
    gy, _ = gret.short_conv_varlen(c["x"], c["w"], c["bias"], cu, 90, tail0=c["tail0"])
    assert torch.equal(got[:37], want[:37]) and torch.equal(gh[0], wh[0]) and torch.equal(gy[:37], wy[:37])
    assert torch.equal(gy[40:127], wy[40:127])       # the tail reaches three rows


def test_scan_extreme_steps():
    # steps from nothing (softplus of -90) to all (a decay that underflows), and decays of zero and one
    N, D, n = 64, 16, 16
    p = scan_inputs("f32", N, D, n, 1)
    p["dt_bias"][0::4] = -90.0
    p["dt_bias"][1::4] = 60.0
    p["A"][2] = 0.0
    p["A"][5] = -1e30
    p["B"][7] = 0.0
    o, h = scan_call(p, 1, N)
    ro, rh = bo.selective_scan(**scan_rows(p, 0, N, 0))
    # a decay of exp(-1e30 delta) is zero in both: its bound must not count the argument
    for r in (ro, rh):
        r.e = np.where(np.isfinite(r.e), r.e, 0)
    keep = [d for d in range(D) if d != 5]
    bo.check(o[0][:, keep], ro[:, keep], "f32")
    bo.check(h[0][keep], rh[keep], "f32")
    b5 = torch.nn.functional.softplus(p["dt"][-1, 5] + p["dt_bias"][5]) * p["u"][-1, 5] * p["B"][-1]
    torch.testing.assert_close(h[0, 5], b5, rtol=1e-5, atol=0)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
@pytest.mark.parametrize("S,D", [(1, 8), (3, 72), (70, 264)])
def test_scan_step(io, n, S, D):
    p = scan_inputs(io, S, D, n, S)
    h0 = p.pop("h0")
    apart = torch.empty_like(h0)
    q = {k: columns(v) if k in ROWS else v for k, v in p.items()}
    o, h = gret.selective_step(**q, h=h0, h_out=apart)
    assert h is apart
    for b in range(S):
        ro, rh = bo.selective_scan(**scan_rows(dict(p, h0=h0), b, b + 1, b))
        bo.check(o[b:b + 1], ro, io)
        bo.check(h[b], rh, "f32")
    o2, h2 = gret.selective_step(**p, h=h0)                                       # in place
    assert h2 is h0 and torch.equal(h0, apart) and torch.equal(o, o2)


SUMS = ("dA", "dskip", "ddt_bias")


def check_scan_backward(io, p, do, dh, g, B, N):
    total = None
    for b in range(B):
        want = bo.selective_scan(**scan_rows(p, b * N, (b + 1) * N, b), do=do[b], dh_final=None if dh is None else dh[b])
        for k in ("du", "ddt", "dB", "dC", "dz"):
            if g[k] is not None:
                bo.check(g[k][b], want[k], io, f"{k} of sequence {b}")
        if g["dh0"] is not None:
            bo.check(g["dh0"][b], want["dh0"], "f32", f"dh0 of sequence {b}")
        total = {k: want[k] if total is None else total[k] + want[k] for k in SUMS}
    for k in SUMS:
        if g[k] is not None:
            bo.check(g[k], total[k], "f32", k)


def scan_backward_call(p, do, B, N, **kw):
    q = {k: v.unflatten(0, (B, N)) if k in ROWS and v is not None else v for k, v in p.items()}
    return gret.selective_scan_backward(**q, do=do, **kw)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
@pytest.mark.parametrize("B,N,D", [(1, 1, 8), (2, 33, 72), (1, 150, 40), (3, 16, 136)])
def test_scan_backward(io, n, B, N, D):
    p = scan_inputs(io, B * N, D, n, B)
    do, dh = draw(10, (B, N, D), io), draw(11, (B, D, n))
    g = scan_backward_call(p, do, B, N, dh_final=dh)
    check_scan_backward(io, p, do, dh, g, B, N)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("without", ["skip", "z", "dt_bias", "h0"])
def test_scan_backward_left_out_and_strided(io, without):
    B, N, D, n = 2, 70, 136, 16
    p = scan_inputs(io, B * N, D, n, B)
    p[without] = None
    do = draw(10, (B, N, D), io)
    q = {k: columns(v) if k in ROWS and v is not None else v for k, v in p.items()}
    g = scan_backward_call(q, do, B, N)
    assert (g["dh0"] is None) == (without == "h0") and (g["dz"] is None) == (without == "z")
    check_scan_backward(io, p, do, None, g, B, N)
    again = scan_backward_call(q, do, B, N)
    for k, v in g.items():
        assert v is None or torch.equal(v, again[k]), k          # the same bits every time


def test_scan_backward_long():
    p = scan_inputs("f32", 1500, 16, 16, 1)
    do, dh = draw(10, (1, 1500, 16)), draw(11, (1, 16, 16))
    check_scan_backward("f32", p, do, dh, scan_backward_call(p, do, 1, 1500, dh_final=dh), 1, 1500)


# ---------------------------------------------------------------- residual norm
def norm_inputs(io, stream, T, D, seed=3):
    p = dict(x=draw(1, (T, D), stream, std=2.0, seed=seed), y=draw(2, (T, D), io, seed=seed),
             gate=draw(3, (T, D), io, seed=seed))
    p.update({k: draw(4 + i, (D,), mean=1.0, std=0.2, seed=seed) for i, k in enumerate(("scale", "w_post", "w_next"))})
    return p


KINDS = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("io,stream", KINDS)
@pytest.mark.parametrize("T,D", [(1, 8), (3, 72), (5, 2048), (130, 264), (2, 4104), (3, 8192)])
def test_norm(io, stream, T, D):
    p = norm_inputs(io, stream, T, D)
    r, n = gret.residual_norm(**p)
    rr, rn = bo.residual_norm(**p)
    bo.check(r, rr, stream, "r")
    bo.check(n, rn, io, "n")


@pytest.mark.parametrize("io,stream", KINDS)
@pytest.mark.parametrize("without", [("gate",), ("scale",), ("w_post",), ("w_next",), ("gate", "scale", "w_post"),
                                     ("gate", "scale", "w_post", "y")])
def test_norm_left_out_and_strided(io, stream, without):
    T, D = 7, 264
    p = norm_inputs(io, stream, T, D)
    for k in without:
        p[k] = None
    q = {k: columns(v) if k in ("x", "y", "gate") and v is not None else v for k, v in p.items()}
    if p["y"] is None:
        q["n"] = torch.empty(T, D, dtype=TYPES[io], device="cuda")
    r, n = gret.residual_norm(**q)
    rr, rn = bo.residual_norm(**p)
    if p["y"] is None:
        assert r is q["x"]
    else:
        bo.check(r, rr, stream, "r")
    assert (n is None) == (p["w_next"] is None)
    if n is not None:
        bo.check(n, rn, io, "n")


def test_norm_in_place_and_empty_rows():
    # a row of zeros has rms sqrt(eps); the stream updated over itself gives what a copy gives
    p = norm_inputs("bf16", "f32", 6, 520)
    for k in ("x", "y"):
        p[k][2] = 0
    r, n = gret.residual_norm(**p)
    rr, rn = bo.residual_norm(**p)
    bo.check(r, rr, "f32")
    bo.check(n, rn, "bf16")
    x = p["x"].clone()
    r2, n2 = gret.residual_norm(**dict(p, x=x), r=x)
    assert r2 is x and torch.equal(x, r) and torch.equal(n, n2)


@pytest.mark.parametrize("io,stream", KINDS)
@pytest.mark.parametrize("T,D", [(1, 8), (3, 72), (700, 264), (5, 2048), (2, 4104), (3, 8192)])
def test_norm_backward(io, stream, T, D):
    p = norm_inputs(io, stream, T, D)
    dr, dn = draw(8, (T, D), stream), draw(9, (T, D), io)
    g = gret.residual_norm_backward(**p, dr=dr, dn=dn)
    want = bo.residual_norm(**p, dr=dr, dn=dn)
    for k, v in want.items():
        bo.check(g[k], v, stream if k == "dx" else io if k in ("dy", "dgate") else "f32", k)


@pytest.mark.parametrize("io,stream", KINDS)
@pytest.mark.parametrize("without", [("gate",), ("scale",), ("w_post",), ("w_next", "dn"), ("dr",),
                                     ("gate", "scale", "w_post"), ("gate", "scale", "w_post", "y")])
def test_norm_backward_left_out_and_strided(io, stream, without):
    T, D = 37, 264
    p = dict(norm_inputs(io, stream, T, D), dr=draw(8, (T, D), stream), dn=draw(9, (T, D), io))
    for k in without:
        p[k] = None
    q = {k: columns(v) if k in ("x", "y", "gate") and v is not None else v for k, v in p.items()}
    g = gret.residual_norm_backward(**q)
    want = bo.residual_norm(**p)
    for k, v in want.items():
        if p[k[1:]] is None:
            assert g[k] is None
        else:
            bo.check(g[k], v, stream if k == "dx" else io if k in ("dy", "dgate") else "f32", k)


@pytest.mark.parametrize("io,stream", KINDS)
@pytest.mark.parametrize("D", [264, 4096, 8192])
def test_norm_backward_gives_up(io, stream, D):
    """A wait that runs out is reported once, the call returns, and the next call is right again."""
    T = 300
    p = dict(norm_inputs(io, stream, T, D), dr=draw(8, (T, D), stream), dn=draw(9, (T, D), io))
    want = gret.residual_norm_backward(**p)
    gret.check_device_status()
    gret.gret_debug_inject_timeout(1)
    try:
        gret.residual_norm_backward(**p)
        with pytest.raises(gret.GretError) as e:
            gret.check_device_status()
        assert e.value.status == gret.Status.ERR_TIMEOUT
    finally:
        gret.gret_debug_inject_timeout(0)
    got = gret.residual_norm_backward(**p)
    gret.check_device_status()
    for k, v in want.items():
        assert torch.equal(v, got[k]), k


# --------------------------------------------------------------------- together
def block_weights(D, n, R, K=4):
    g = lambda i, *s, std=1.0, mean=0.0: draw(20 + i, s, std=std, mean=mean)  # noqa: E731
    return dict(w_in=g(0, D, 2 * D, std=D ** -0.5), conv_w=g(1, D, K, std=0.5), conv_b=g(2, D, std=0.1),
                w_x=g(3, D, R + 2 * n, std=D ** -0.5), w_dt=g(4, R, D, std=R ** -0.5), dt_bias=g(5, D, mean=-3.0),
                A=-torch.exp(g(6, D, n)), skip=g(7, D, mean=1.0, std=0.1), w_out=g(8, D, D, std=D ** -0.5),
                w_post=g(9, D, mean=1.0, std=0.1), w_next=g(10, D, mean=1.0, std=0.1), scale=g(11, D, mean=0.5, std=0.1))


def block_prompt(x, W, n, R, tail=None, h=None, gate=None):
    _, v = gret.residual_norm(x, w_next=W["w_next"])
    xz = v @ W["w_in"]
    D = x.shape[-1]
    c, tail = gret.short_conv(xz[..., :D], W["conv_w"], W["conv_b"], tail0=tail)
    q = c @ W["w_x"]
    o, h = gret.selective_scan(c, q[..., :R] @ W["w_dt"], W["A"], q[..., R:R + n], q[..., R + n:], skip=W["skip"],
                               z=xz[..., D:], dt_bias=W["dt_bias"], h0=h)
    r, v = gret.residual_norm(x, o @ W["w_out"], gate=xz[..., D:], scale=W["scale"], w_post=W["w_post"],
                              w_next=W["w_next"])
    return r, v, tail, h


def block_step(x, W, n, R, tail, h):
    _, v = gret.residual_norm(x, w_next=W["w_next"])
    xz = v @ W["w_in"]
    D = x.shape[-1]
    c, _ = gret.short_conv_step(xz[:, :D], W["conv_w"], W["conv_b"], tail)
    q = c @ W["w_x"]
    o, _ = gret.selective_step(c, q[:, :R] @ W["w_dt"], W["A"], q[:, R:R + n], q[:, R + n:], h, skip=W["skip"],
                               z=xz[:, D:], dt_bias=W["dt_bias"])
    return gret.residual_norm(x, o @ W["w_out"], gate=xz[:, D:], scale=W["scale"], w_post=W["w_post"],
                              w_next=W["w_next"])


def test_block_prompt_then_steps_is_the_longer_prompt():
    """A prompt, a second piece of it and single tokens give what one pass over all tokens gives."""
    B, D, n, R, cuts = 2, 64, 16, 8, (37, 90, 96)
    W = block_weights(D, n, R)
    x = draw(40, (B, cuts[2], D))
    r, v, tail, h = block_prompt(x, W, n, R)
    r1, v1, t1, h1 = block_prompt(x[:, :cuts[0]].contiguous(), W, n, R)
    r2, v2, t2, h2 = block_prompt(x[:, cuts[0]:cuts[1]].contiguous(), W, n, R, t1, h1)
    rs, vs = [r1, r2], [v1, v2]
    for t in range(cuts[1], cuts[2]):
        a, b = block_step(x[:, t].contiguous(), W, n, R, t2, h2)
        rs.append(a[:, None])
        vs.append(b[:, None])
    # the matrix products round differently for other row counts: fp32 with its default products, tens of units
    for got, want in ((torch.cat(rs, 1), r), (torch.cat(vs, 1), v), (h2, h), (t2, tail)):
        torch.testing.assert_close(got, want, rtol=2e-4, atol=2e-4)


def test_block_step_in_a_graph_and_on_another_stream():
    """Steps captured once and replayed, on a stream of their own, move the state as direct calls do."""
    S, D, n, R = 3, 64, 16, 8
    W = block_weights(D, n, R)
    xs = draw(41, (4, S, D))
    tail, h = draw(42, (S, 3, D)), draw(43, (S, D, n))
    want_t, want_h = tail.clone(), h.clone()
    want = [block_step(x, W, n, R, want_t, want_h)[0].clone() for x in xs]
    x = torch.empty(S, D, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        keep_t, keep_h = tail.clone(), h.clone()
        x.copy_(xs[0])
        block_step(x, W, n, R, tail, h)              # warm up
        tail.copy_(keep_t)
        h.copy_(keep_h)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, _ = block_step(x, W, n, R, tail, h)
    for i in range(4):
        x.copy_(xs[i])
        graph.replay()
        torch.testing.assert_close(r, want[i], rtol=1e-4, atol=1e-4)
    torch.testing.assert_close(h, want_h, rtol=1e-4, atol=1e-4)


def test_row_offsets_past_31_bits():
    """Columns of a tensor of more than 2^31 entries give what dense copies give."""
    T, D, n = 70000, 64, 16
    wide = torch.empty(T, 32768, dtype=torch.bfloat16, device="cuda")
    p, c, m = scan_inputs("bf16", T, D, n, 1), conv_inputs("bf16", T, D, 4, 1), norm_inputs("bf16", "bf16", T, D)

    def far(t, at):
        view = wide[:, at:at + t.shape[-1]]
        view.copy_(t)
        return view

    q = {k: far(v, 1024 * (i + 1)) if k in ROWS else v for i, (k, v) in enumerate(p.items())}
    do = draw(10, (1, T, D), "bf16")
    cu = offsets([T - 9, 9])
    p2, q2 = (dict(x, h0=torch.cat([x["h0"]] * 2)) for x in (p, q))
    x = far(c["x"], 16384)
    y = far(m["y"], 20480)
    for a, b in ((scan_call(p, 1, T), scan_call(q, 1, T)),
                 (gret.selective_scan_varlen(**p2, cu_seqlens=cu, max_seqlen=T),
                  gret.selective_scan_varlen(**q2, cu_seqlens=cu, max_seqlen=T)),
                 (scan_backward_call(p, do, 1, T).values(), scan_backward_call(q, do, 1, T).values()),
                 (gret.short_conv(c["x"][None], c["w"]), gret.short_conv(x[None], c["w"])),
                 (gret.short_conv_backward(c["x"][None], c["w"], None, do).values(),
                  gret.short_conv_backward(x[None], c["w"], None, do).values()),
                 (gret.residual_norm(**m), gret.residual_norm(**dict(m, y=y))),
                 (gret.residual_norm_backward(**m, dr=do[0], dn=do[0]).values(),
                  gret.residual_norm_backward(**dict(m, y=y), dr=do[0], dn=do[0]).values())):
        for s, t in zip(a, b):
            assert s is None and t is None or torch.equal(s, t)


def test_calls_on_a_given_stream():
    side = torch.cuda.Stream()
    p = scan_inputs("bf16", 600, 264, 16, 1)
    c = conv_inputs("bf16", 600, 264, 4, 1)
    m = norm_inputs("bf16", "bf16", 600, 264)
    want = [scan_call(p, 1, 600), gret.short_conv(c["x"][None], c["w"], c["bias"]), gret.residual_norm(**m)]
    torch.cuda.synchronize()
    got = [scan_call(p, 1, 600, stream=side), gret.short_conv(c["x"][None], c["w"], c["bias"], stream=side),
           gret.residual_norm(**m, stream=side)]
    side.synchronize()
    for a, b in zip(want, got):
        for s, t in zip(a, b):
            assert torch.equal(s, t)


def test_gradients_in_two_graphs_and_beside_one_another():
    """Two captured training passes, each with what it allocated, replayed in turn and after new inputs; and two
    streams at work at once."""
    B, N, D, n = 2, 90, 72, 16
    sets = []
    for seed in (5, 6):
        p = scan_inputs("bf16", B * N, D, n, B, seed=seed)
        c = conv_inputs("bf16", B * N, D, 4, B, seed=seed)
        m = norm_inputs("bf16", "f32", B * N, D, seed=seed)
        do, dr = draw(10, (B, N, D), "bf16", seed=seed), draw(11, (B * N, D), seed=seed)
        sets.append((p, c, m, do, dr))

    def one(s, stream=None):
        p, c, m, do, dr = s
        a = scan_backward_call(p, do, B, N, stream=stream)
        b = gret.short_conv_backward(c["x"].view(B, N, D), c["w"], c["bias"], do, tail0=c["tail0"], stream=stream)
        e = gret.residual_norm_backward(**m, dr=dr, dn=do.view(B * N, D), stream=stream)
        o, h = scan_call(p, B, N, stream=stream)
        return [v for g in (a, b, e) for v in g.values() if v is not None] + [o, h]

    want = [[t.clone() for t in one(s)] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    both = [one(s, st) for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(one(s))
        graphs.append(g)
    for i in (0, 1, 1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    for w, b, o in zip(want, both, outs):
        for x, y, z in zip(w, b, o):
            assert torch.equal(x, y) and torch.equal(x, z)
    sets[0][0]["u"].mul_(0.5)                        # new values in the captured inputs
    graphs[0].replay()
    again = one(sets[0])
    torch.cuda.synchronize()
    for x, y in zip(again, outs[0]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("bound", [2 ** 31 - 1, 2 ** 32 + 3])
def test_packed_with_a_bound_past_all_rows(bound):
    """The longest sequence may be given as any bound from above."""
    lens, D, n = [300, 0, 5, 91], 24, 16
    T = sum(lens) + 3
    p, c, cu = scan_inputs("f32", T, D, n, len(lens)), conv_inputs("f32", T, D, 4, len(lens)), offsets(lens)
    o, y = torch.full((T, D), 7.0, device="cuda"), torch.full((T, D), 7.0, device="cuda")
    _, h = gret.selective_scan_varlen(**p, cu_seqlens=cu, max_seqlen=bound, o=o)
    gret.short_conv_varlen(c["x"], c["w"], c["bias"], cu, bound, tail0=c["tail0"], y=y)
    at = 0
    for b, m in enumerate(lens):
        if m:
            ro, rh = bo.selective_scan(**scan_rows(p, at, at + m, b))
            bo.check(o[at:at + m], ro, "f32", f"o of sequence {b}")
            bo.check(h[b], rh, "f32", f"h of sequence {b}")
            bo.check(y[at:at + m], bo.short_conv(c["x"][at:at + m], c["w"], c["bias"], c["tail0"][b])[0], "f32")
        at += m
    assert (o[at:] == 7).all() and (y[at:] == 7).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_scan_backward_of_the_most_channels(io):
    """65536 channels x 64 states with more segments than a thread folds.  Only a few channels have a gradient: the
    others add nothing to dB and dC, so that the few make up all of both."""
    N, D, n = 300, 65536, 64
    keep = [0, 1, 31, 4096, 33333, 65528, 65535]
    p = scan_inputs(io, N, D, n, 1)
    do, dh = torch.zeros((1, N, D), dtype=TYPES[io], device="cuda"), torch.zeros(1, D, n, device="cuda")
    do[..., keep], dh[:, keep] = draw(10, (1, N, len(keep)), io), draw(11, (1, len(keep), n))
    g = scan_backward_call(p, do, 1, N, dh_final=dh)
    few = {k: v if k in ("B", "C") else v[:, keep] if k in ROWS + ("h0",) else v[keep] for k, v in p.items()}
    g = {k: v if k in ("dB", "dC") else v[..., keep, :] if k in ("dA", "dh0") else v[..., keep] for k, v in g.items()}
    check_scan_backward(io, few, do[..., keep], dh[:, keep], g, 1, N)


# A that keeps nothing of the tokens before: any step of more than 1e-3 decays to zero in 32 bits and in 64, so the
# oracle takes a finite number in their place.
NOTHING = (float("-inf"), -3.4e38, -3e38, -1e30)


def keep_nothing(p):
    p["dt_bias"].zero_()
    for i, a in enumerate(NOTHING):
        p["A"][2 * i] = a                        # a channel of them
        p["A"][2 * i + 1, 1::3] = a              # and a channel with some
    return dict(p, A=p["A"].clamp(min=-1e6))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
@pytest.mark.parametrize("B,N", [(2, 1), (1, 17), (2, 63), (2, 1203)])
def test_scan_that_keeps_nothing(io, n, B, N):
    D = 24
    p = scan_inputs(io, B * N, D, n, B)
    ref = keep_nothing(p)
    o, h = scan_call(p, B, N)
    cu = torch.arange(0, B * N + 1, N, dtype=torch.int32, device="cuda")
    o2, h2 = gret.selective_scan_varlen(**p, cu_seqlens=cu, max_seqlen=N)
    for b in range(B):
        ro, rh = bo.selective_scan(**scan_rows(ref, b * N, (b + 1) * N, b))
        bo.check(o[b], ro, io, f"o of sequence {b}")
        bo.check(h[b], rh, "f32", f"h of sequence {b}")
        bo.check(o2[b * N:(b + 1) * N], ro, io, f"o of packed sequence {b}")
        bo.check(h2[b], rh, "f32", f"h of packed sequence {b}")
    if N == 1:
        h0 = p.pop("h0")
        o, h = gret.selective_step(**p, h=h0.clone())
        for b in range(B):
            ro, rh = bo.selective_scan(**scan_rows(ref, b, b + 1, b))
            bo.check(o[b:b + 1], ro, io)
            bo.check(h[b], rh, "f32")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
@pytest.mark.parametrize("B,N", [(2, 1), (2, 17), (2, 601)])
def test_scan_backward_that_keeps_nothing(io, n, B, N):
    D = 24
    p = scan_inputs(io, B * N, D, n, B)
    ref = keep_nothing(p)
    do, dh = draw(10, (B, N, D), io), draw(11, (B, D, n))
    check_scan_backward(io, ref, do, dh, scan_backward_call(p, do, B, N, dh_final=dh), B, N)


def check_norm(io, stream, T, D):
    p = norm_inputs(io, stream, T, D)
    r, n = gret.residual_norm(**p)
    rr, rn = bo.residual_norm(**p)
    bo.check(r, rr, stream, "r")
    bo.check(n, rn, io, "n")
    dr, dn = draw(8, (T, D), stream), draw(9, (T, D), io)
    g = gret.residual_norm_backward(**p, dr=dr, dn=dn)
    for k, v in bo.residual_norm(**p, dr=dr, dn=dn).items():
        bo.check(g[k], v, stream if k == "dx" else io if k in ("dy", "dgate") else "f32", k)
    again = gret.residual_norm_backward(**p, dr=dr, dn=dn)
    assert all(torch.equal(g[k], again[k]) for k in g)


@pytest.mark.parametrize("io,stream", KINDS)
@pytest.mark.parametrize("D", [8, 72, 256])
def test_norm_blocks_of_one_warp_with_many_rows(io, stream, D):
    # 16 blocks an SM, each of one warp, whose rows in shared memory are replaced while it walks seven or eight rows
    check_norm(io, stream, 16 * torch.cuda.get_device_properties(0).multi_processor_count * 7 + 5, D)


# ------------------------------------------------- cut sequences of every segment length and join
PERIOD = 24                                      # channels that a wide tensor repeats: no warp's or block's share of them
WARP = {8: 32, 16: 16, 32: 16, 64: 8}            # the scan's channels a warp


def wide(t, D, dim=-1):
    """24 channels, along `dim`, repeated up to D."""
    return t.repeat([D // PERIOD if i == dim % t.dim() else 1 for i in range(t.dim())])


def repeated(p, D):
    """The scan's inputs of 24 channels, repeated up to D."""
    at = {"A": 0, "h0": 1}
    return {k: v if k in ("B", "C") or v is None else wide(v, D, at.get(k, -1)) for k, v in p.items()}


def check_repeated(got, want, io, dim, what):
    """The 24 channels' result, and the same bits in every repetition along `dim`."""
    parts = got.split(PERIOD, dim)
    bo.check(parts[0], want, io, what)
    for i, part in enumerate(parts):
        assert torch.equal(part, parts[0]), f"{what}, repetition {i}"


TYPE_IDS = {"bf16": gret.Dtype.BF16, "f32": gret.Dtype.F32}
# sequences, tokens of each, warps of channels -> tokens of a segment and segments of a sequence (on 148 SMs)
CUTS = [(5, 500, 16, 32, 16), (2, 1500, 16, 32, 47), (6, 500, 21, 64, 8), (3, 1021, 21, 64, 16), (3, 1040, 21, 64, 17),
        (2, 1700, 21, 64, 27), (4, 1200, 64, 80, 15), (2, 2500, 64, 80, 32)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
@pytest.mark.parametrize("B,N,warps,seg,segs", CUTS)
def test_scan_cut_into_segments_of_many_tiles(io, n, B, N, warps, seg, segs):
    """Segments of two, four and five tiles; up to 16 of them joined by the second launch, more by a fold."""
    D = WARP[n] * warps // PERIOD * PERIOD
    need = gret.gret_selective_scan_workspace_size(B, N, D, n, TYPE_IDS[io])
    assert need // (D * (n + 1) * 4) == B * segs and -(-N // seg) == segs and -(-N // (seg + 16)) < segs
    p = scan_inputs(io, B * N, PERIOD, n, B)
    o, h = scan_call(repeated(p, D), B, N)
    for b in range(B):
        ro, rh = bo.selective_scan(**scan_rows(p, b * N, (b + 1) * N, b))
        check_repeated(o[b], ro, io, 1, f"o of sequence {b}")
        check_repeated(h[b], rh, "f32", 0, f"h of sequence {b}")


# sequences in all, the long ones among them, warps of channels -> tokens of a segment; the longest has up to 16 segments
# or more, and the batch up to 64 sequences (the rests by length), up to 256 (in the batch's order) or more (unranked)
PACKED_CUTS = [(12, (1500, 100, 900), 40, 64), (12, (1000, 700), 40, 64), (40, (2000, 1100), 6, 16),
               (70, (2000, 1100), 6, 16), (70, (2600, 64, 1100), 40, 64), (70, (950, 800), 40, 64),
               (300, (2000, 1500), 6, 32), (300, (2500, 1700, 900), 30, 80), (300, (1000, 900), 30, 64)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
@pytest.mark.parametrize("S,longest,warps,seg", PACKED_CUTS)
def test_scan_packed_and_cut_in_every_order(io, n, S, longest, warps, seg):
    lens = list(longest) + [(37 * i) % 40 for i in range(S - len(longest))]
    lens = [lens[i * 11 % S] for i in range(S)]                 # the long ones among the others
    D, T = WARP[n] * warps // PERIOD * PERIOD, sum(lens) + 3
    assert sorted(lens)[-len(longest):] == sorted(longest)
    need = gret.gret_selective_scan_varlen_workspace_size(S, T, max(lens), D, n, TYPE_IDS[io])
    slots = need // (D * (n + 1) * 4) - S
    assert slots == T // seg and slots != T // (seg + 16) and (seg == 16 or slots != T // (seg - 16))
    p = scan_inputs(io, T, PERIOD, n, S)
    o = torch.full((T, D), 7.0, dtype=TYPES[io], device="cuda")
    _, h = gret.selective_scan_varlen(**repeated(p, D), cu_seqlens=offsets(lens), max_seqlen=max(lens), o=o)
    at = 0
    for b, m in enumerate(lens):
        if m:
            ro, rh = bo.selective_scan(**scan_rows(p, at, at + m, b))
            check_repeated(o[at:at + m], ro, io, 1, f"o of sequence {b}")
            check_repeated(h[b], rh, "f32", 0, f"h of sequence {b}")
        else:
            assert torch.equal(h[b], wide(p["h0"][b], D, 0))
        at += m
    assert (o[at:] == 7).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
def test_scan_backward_of_several_sequences_of_many_segments(io, n):
    # 22 segments or more each: folded in eight parts
    B, N, D = 3, 700, 40
    p = scan_inputs(io, B * N, D, n, B)
    do, dh = draw(10, (B, N, D), io), draw(11, (B, D, n))
    check_scan_backward(io, p, do, dh, scan_backward_call(p, do, B, N, dh_final=dh), B, N)


# --------------------------------------------------- the convolution's long segments
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 4])
def test_conv_segments_of_64_tokens(io, K):
    """Enough rows and channels that a thread walks 64 tokens, whose copies go around their buffers."""
    B, N, D, lens = 2, 4737, 171 * PERIOD, [5000, 0, 1, 3, 4001, 63, 65, 300, 38]
    T = B * N
    assert T // 64 * (D // 4) >= 148 * 1024 and sum(lens) == T - 3
    small = conv_inputs(io, T, PERIOD, K, len(lens))
    p = {k: wide(v, D, 0 if k == "w" else -1) for k, v in small.items()}
    y, tail = gret.short_conv(p["x"].view(B, N, D), p["w"], p["bias"], tail0=p["tail0"][:B])
    for b in range(B):
        ry, rt = bo.short_conv(small["x"][b * N:(b + 1) * N], small["w"], small["bias"], small["tail0"][b])
        check_repeated(y[b], ry, io, 1, f"y of sequence {b}")
        check_repeated(tail[b], rt, io, 1, f"tail of sequence {b}")
    y = torch.full((T, D), 7.0, dtype=TYPES[io], device="cuda")
    _, tail = gret.short_conv_varlen(p["x"], p["w"], p["bias"], offsets(lens), max(lens), tail0=p["tail0"], y=y)
    at = 0
    for b, m in enumerate(lens):
        ry, rt = bo.short_conv(small["x"][at:at + m], small["w"], small["bias"], small["tail0"][b])
        check_repeated(y[at:at + m], ry, io, 1, f"y of packed sequence {b}")
        check_repeated(tail[b], rt, io, 1, f"tail of packed sequence {b}")
        at += m
    assert (y[at:] == 7).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("K", [3, 4])
def test_conv_backward_segments_of_128_tokens(io, K):
    B, N, D = 2, 4737, 342 * PERIOD
    slots = -(-N // 128) * B
    assert gret.gret_short_conv_backward_workspace_size(B, N, D, K, TYPE_IDS[io]) // ((K + 1) * D * 4) == -(-slots // 4)
    small = conv_inputs(io, B * N, PERIOD, K, B)
    p = {k: wide(v, D, 0 if k == "w" else -1) for k, v in small.items()}
    dy, dtail = draw(5, (B, N, PERIOD), io), draw(6, (B, K - 1, PERIOD), io)
    g = gret.short_conv_backward(p["x"].view(B, N, D), p["w"], p["bias"], wide(dy, D), tail0=p["tail0"],
                                 dtail=wide(dtail, D))
    total = None
    for b in range(B):
        want = bo.short_conv(small["x"][b * N:(b + 1) * N], small["w"], small["bias"], small["tail0"][b], dy=dy[b],
                             dtail=dtail[b])
        check_repeated(g["dx"][b], want["dx"], io, 1, f"dx of sequence {b}")
        check_repeated(g["dtail0"][b], want["dtail0"], io, 1, f"dtail0 of sequence {b}")
        total = {k: want[k] if total is None else total[k] + want[k] for k in ("dw", "dbias")}
    for k, v in total.items():
        check_repeated(g[k], v, "f32", 0, k)


# ------------------------------------------------------- the norm's blocks with many rows
# Rows that go at least twice around a block's rows in shared memory, on 148 SMs: 2672 rows of 2048 channels (forward six
# or seven rows a block, one vector a thread; gradients nine or ten), 1337 rows of up to 4096 (gradients nine or ten, one
# vector a thread), 745 rows of more (five or six, two vectors); all parts and vectors that fill the rows at 2048, 4096
# and 8192 channels
@pytest.mark.parametrize("io,stream", KINDS)
@pytest.mark.parametrize("T,D", [(2672, 2048), (1337, 2056), (1337, 4096), (745, 4104), (745, 8192)])
def test_norm_blocks_with_many_rows(io, stream, T, D):
    check_norm(io, stream, T, D)


# ------------------------------------------------------------------ large batches
def sample(p, rows, seqs, keep):
    """Some rows, sequences and channels of a scan's inputs."""
    q = {k: v[rows] if k in ROWS else v for k, v in p.items()}
    q["h0"] = None if q["h0"] is None else q["h0"][seqs]
    at = {"A": 0, "h0": 0}
    return {k: v if k in ("B", "C") or v is None else v[..., keep, :] if k in at else v[..., keep] for k, v in q.items()}


def random_scan(io, rows, D, n, seqs):
    """Inputs drawn on the GPU, for sizes that the host would take long for."""
    gen = torch.Generator("cuda").manual_seed(5)
    normal = lambda *s, to="f32": torch.randn(s, generator=gen, device="cuda", dtype=TYPES[to])  # noqa: E731
    return dict(u=normal(rows, D, to=io), dt=normal(rows, D, to=io), A=-torch.exp(normal(D, n)), B=normal(rows, n, to=io),
                C=normal(rows, n, to=io), skip=normal(D), z=normal(rows, D, to=io), dt_bias=normal(D) - 3,
                h0=normal(seqs, D, n)), normal


def check_large(io, B, N, D, n, keep, seqs):
    """All calls at a size of many rows, at some sequences and channels."""
    p, normal = random_scan(io, B * N, D, n, B)
    do = normal(B, N, D, to=io)
    o, h = scan_call(p, B, N)
    g = scan_backward_call(p, do, B, N)
    w, bias = normal(D, 4), normal(D)
    y, tail = gret.short_conv(p["u"].view(B, N, D), w, bias)
    c = gret.short_conv_backward(p["u"].view(B, N, D), w, bias, do)
    norm = dict(x=p["u"], y=p["dt"], gate=p["z"], scale=normal(D), w_post=normal(D), w_next=normal(D))
    r, v = gret.residual_norm(**norm)
    m = gret.residual_norm_backward(**norm, dr=do.view(B * N, D), dn=do.view(B * N, D))
    for b in seqs:
        rows = slice(b * N, (b + 1) * N)
        q, up = sample(p, rows, b, keep), do[b][:, keep]
        ro, rh = bo.selective_scan(**q)
        bo.check(o[b][:, keep], ro, io, f"o of sequence {b}")
        bo.check(h[b][keep], rh, "f32", f"h of sequence {b}")
        want = bo.selective_scan(**q, do=up)
        for k in ("du", "ddt", "dz"):
            bo.check(g[k][b][:, keep], want[k], io, f"{k} of sequence {b}")
        bo.check(g["dh0"][b][keep], want["dh0"], "f32", f"dh0 of sequence {b}")
        ry, rt = bo.short_conv(q["u"], w[keep], bias[keep])
        bo.check(y[b][:, keep], ry, io, f"y of sequence {b}")
        bo.check(tail[b][:, keep], rt, io, f"tail of sequence {b}")
        bo.check(c["dx"][b][:, keep], bo.short_conv(q["u"], w[keep], bias[keep], dy=up)["dx"], io, f"dx of sequence {b}")
        whole = {k: t[rows] if t.dim() == 2 else t for k, t in norm.items()}
        rr, rn = bo.residual_norm(**whole)
        bo.check(r[rows], rr, io, f"r of sequence {b}")
        bo.check(v[rows], rn, io, f"n of sequence {b}")
        want = bo.residual_norm(**whole, dr=do[b], dn=do[b])
        for k in ("dx", "dy", "dgate"):
            bo.check(m[k][rows], want[k], io, f"norm's {k} of sequence {b}")


def test_outputs_past_31_bits():
    """Dense tensors of more than 2^31 entries, each side of that and at the end."""
    B, N, D = 5300, 100, 4096
    cross = 2 ** 31 // (N * D)
    assert B * N * D > 2 ** 31
    check_large("bf16", B, N, D, 16, [0, 31, 2047, 4095], [0, cross, B - 1])
    torch.cuda.empty_cache()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 2, 40])
def test_more_sequences_than_a_grids_second_dimension(io, N):
    B = 70001
    check_large(io, B, N, 16, 8, list(range(16)), [0, 1, 65535, 65536, B - 1])
    p, normal = random_scan(io, B, 16, 8, B)
    h0, p["h0"] = p["h0"], None
    lens = torch.arange(B, device="cuda") % 3
    lens[-1] += B - lens.sum()                   # the last sequence takes the rows that are left
    cu = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32)
    longest, x = int(lens.max()), p["u"]
    o, h = gret.selective_scan_varlen(**dict(p, h0=h0), cu_seqlens=cu, max_seqlen=longest)
    w, tail = normal(16, 4), normal(B, 3, 16, to=io)
    y, t = gret.short_conv_varlen(x, w, None, cu, longest, tail0=tail)
    q = {k: v for k, v in p.items() if k != "h0"}
    o1, h1 = gret.selective_step(**q, h=h0, h_out=torch.empty_like(h0))
    y1, t1 = gret.short_conv_step(x, w, None, tail, tail_out=torch.empty_like(tail))
    for b in (0, 1, 2, 65534, 65535, 65536, B - 2):
        at, end = int(cu[b]), int(cu[b + 1])
        ro, rh = bo.selective_scan(**scan_rows(dict(p, h0=h0), at, end, b)) if end > at else (None, bo.f64(h0[b]))
        if end > at:
            bo.check(o[at:end], ro, io, f"o of packed sequence {b}")
            bo.check(y[at:end], bo.short_conv(x[at:end], w, None, tail[b])[0], io, f"y of packed sequence {b}")
        bo.check(h[b], rh, "f32", f"h of packed sequence {b}")
        ro, rh = bo.selective_scan(**scan_rows(dict(p, h0=h0), b, b + 1, b))
        bo.check(o1[b:b + 1], ro, io)
        bo.check(h1[b], rh, "f32")
        ry, rt = bo.short_conv(x[b:b + 1], w, None, tail[b])
        bo.check(y1[b:b + 1], ry, io)
        assert (t1[b].double().cpu().numpy() == rt.v).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
@pytest.mark.parametrize("N,at", [(61, 22), (1203, 700)])
def test_a_value_that_is_no_number_stays_in_its_channel_and_behind_its_token(io, n, N, at):
    """Whole and cut sequences: what comes before the token, and every other channel, keeps its bits."""
    B, D, bad = 2, 40, 13
    p = scan_inputs(io, B * N, D, n, B)
    others = [d for d in range(D) if d != bad]
    do = draw(10, (B, N, D), io)
    o, h = scan_call(p, B, N)
    g = scan_backward_call(p, do, B, N)
    c = conv_inputs(io, B * N, D, 4, B)
    x = c["x"].view(B, N, D)
    y, tail = gret.short_conv(x, c["w"], c["bias"], tail0=c["tail0"])
    dx = gret.short_conv_backward(x, c["w"], c["bias"], do, tail0=c["tail0"])
    for k in ("u", "dt", "z", "do"):
        for value in (float("nan"), float("inf")):
            up = do.clone()
            q = dict(p, **{k: p[k].clone()}) if k != "do" else p
            (up if k == "do" else q[k].view(B, N, D))[1, at, bad] = value
            o2, h2 = scan_call(q, B, N)
            g2 = scan_backward_call(q, up, B, N)
            assert torch.equal(o2[0], o[0]) and torch.equal(o2[1, :at], o[1, :at]) and torch.equal(h2[0], h[0]), (k, value)
            assert torch.equal(o2[..., others], o[..., others]) and torch.equal(h2[:, others], h[:, others]), (k, value)
            for w in ("du", "ddt", "dz"):
                assert torch.equal(g2[w][0], g[w][0]) and torch.equal(g2[w][..., others], g[w][..., others]), (k, w, value)
            for w in ("dA", "dskip", "ddt_bias"):
                assert torch.equal(g2[w][others], g[w][others]), (k, w, value)
            # a gradient goes back no further than to the tokens it comes from
            assert k != "do" or all(torch.equal(g2[w][1, at + 1:], g[w][1, at + 1:]) for w in ("du", "ddt", "dz")), value
    for value in (float("nan"), float("inf")):
        x2 = x.clone()
        x2[1, at, bad] = value
        y2, t2 = gret.short_conv(x2, c["w"], c["bias"], tail0=c["tail0"])
        assert torch.equal(y2[0], y[0]) and torch.equal(y2[1, :at], y[1, :at]) and torch.equal(y2[1, at + 4:], y[1, at + 4:])
        assert torch.equal(y2[..., others], y[..., others]) and torch.equal(t2, tail)
        dx2 = gret.short_conv_backward(x2, c["w"], c["bias"], do, tail0=c["tail0"])
        assert torch.equal(dx2["dx"][..., others], dx["dx"][..., others]) and torch.equal(dx2["dx"][0], dx["dx"][0])
        assert torch.equal(dx2["dx"][1, :at - 3], dx["dx"][1, :at - 3])
        assert torch.equal(dx2["dx"][1, at + 4:], dx["dx"][1, at + 4:])
        assert torch.equal(dx2["dw"][others], dx["dw"][others]) and torch.equal(dx2["dbias"][others], dx["dbias"][others])


@pytest.mark.parametrize("io,stream", KINDS)
def test_a_row_that_is_no_number_stays_in_its_row(io, stream):
    T, D, bad = 3000, 264, 1444
    p = norm_inputs(io, stream, T, D)
    dr, dn = draw(8, (T, D), stream), draw(9, (T, D), io)
    r, n = gret.residual_norm(**p)
    g = gret.residual_norm_backward(**p, dr=dr, dn=dn)
    rest = [t for t in range(T) if t != bad]
    for k in ("x", "y", "gate"):
        for value in (float("nan"), float("inf")):
            q = dict(p, **{k: p[k].clone()})
            q[k][bad, 77] = value
            r2, n2 = gret.residual_norm(**q)
            g2 = gret.residual_norm_backward(**q, dr=dr, dn=dn)
            gret.check_device_status()
            for a, b in [(r, r2), (n, n2)] + [(g[w], g2[w]) for w in ("dx", "dy", "dgate")]:
                assert torch.equal(a[rest], b[rest]), (k, value)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n", [8, 16, 32, 64])
def test_scan_of_states_that_grow(io, n):
    """A positive A, by less over the whole sequence than fp32 holds: cut sequences and their gradients."""
    B, N, D = 2, 1203, 24
    p = scan_inputs(io, B * N, D, n, B)
    p["A"] = p["A"].abs().clamp(max=2.0) * 0.02
    o, h = scan_call(p, B, N)
    do, dh = draw(10, (B, N, D), io), draw(11, (B, D, n))
    g = scan_backward_call(p, do, B, N, dh_final=dh)
    for b in range(B):
        ro, rh = bo.selective_scan(**scan_rows(p, b * N, (b + 1) * N, b))
        bo.check(o[b], ro, io, f"o of sequence {b}")
        bo.check(h[b], rh, "f32", f"h of sequence {b}")
    check_scan_backward(io, p, do, dh, g, B, N)
