"""The 64-bit oracle of the selective state space block, checked against what its formulas fix."""
import numpy as np
import pytest

from oracle import block_oracle as bo

RNG = np.random.default_rng


def _scan_inputs(seed, N, D, n):
    r = RNG(seed)
    return dict(u=r.standard_normal((N, D)), dt=r.standard_normal((N, D)), A=-np.exp(r.standard_normal((D, n))),
                B=r.standard_normal((N, n)), C=r.standard_normal((N, n)), skip=r.standard_normal(D),
                z=r.standard_normal((N, D)), dt_bias=r.standard_normal(D), h0=r.standard_normal((D, n)))


def test_conv_is_numpy_convolution():
    r = RNG(1)
    x, w = r.standard_normal((9, 3)), r.standard_normal((3, 4))
    y, tail = bo.short_conv(x, w, swish=False)
    for d in range(3):
        np.testing.assert_allclose(y.v[:, d], np.convolve(x[:, d], w[d, ::-1])[:9], rtol=1e-12, atol=1e-13)
    np.testing.assert_array_equal(tail.v, x[-3:])


def test_conv_and_scan_in_pieces():
    r = RNG(2)
    x, w, b = r.standard_normal((11, 2)), r.standard_normal((2, 4)), r.standard_normal(2)
    whole, tail = bo.short_conv(x, w, b)
    y1, t1 = bo.short_conv(x[:2], w, b)
    y2, t2 = bo.short_conv(x[2:], w, b, tail0=t1)
    np.testing.assert_allclose(np.concatenate([y1.v, y2.v]), whole.v, rtol=1e-13)
    np.testing.assert_array_equal(t2.v, tail.v)
    p = _scan_inputs(3, 9, 2, 8)
    o, h = bo.selective_scan(**p)
    cut = lambda a, b: {k: (v[a:b] if k in ("u", "dt", "B", "C", "z") else v) for k, v in p.items()}  # noqa: E731
    o1, h1 = bo.selective_scan(**cut(0, 4))
    o2, h2 = bo.selective_scan(**dict(cut(4, 9), h0=h1.v))
    np.testing.assert_allclose(np.concatenate([o1.v, o2.v]), o.v, rtol=1e-12)
    np.testing.assert_allclose(h2.v, h.v, rtol=1e-12)


def test_scan_closed_form():
    # constant decay and input: a geometric sum
    N, D, n = 6, 1, 8
    A = np.full((D, n), -1.0)
    raw = np.log(np.expm1(0.5))
    o, h = bo.selective_scan(np.ones((N, D)), np.full((N, D), raw), A, np.ones((N, n)), np.ones((N, n)) / n)
    a = np.exp(-0.5)
    np.testing.assert_allclose(o.v[:, 0], 0.5 * (1 - a ** np.arange(1, N + 1)) / (1 - a), rtol=1e-12)


def test_norm_rows():
    r = RNG(4)
    x, y = r.standard_normal((3, 16)), r.standard_normal((3, 16))
    s, n = bo.residual_norm(x, y, w_next=np.ones(16), eps=0.0)
    np.testing.assert_allclose(s.v, x + y, rtol=1e-14)
    np.testing.assert_allclose((n.v ** 2).mean(-1), 1, rtol=1e-12)


def _differences(f, args, name, seed):
    """Directional derivative of the scalar f along a random direction of args[name]."""
    d = RNG(seed).standard_normal(np.shape(args[name]))
    h = 1e-6
    up, down = (f(**{**args, name: np.asarray(args[name]) + s * h * d}) for s in (1, -1))
    return d, (up - down) / (2 * h)


@pytest.mark.parametrize("name", ["u", "dt", "A", "B", "C", "skip", "z", "dt_bias", "h0"])
def test_scan_gradients_are_differences(name):
    p = _scan_inputs(5, 7, 3, 8)
    r = RNG(6)
    do, dh = r.standard_normal((7, 3)), r.standard_normal((3, 8))

    def f(**a):
        o, h = bo.selective_scan(**a)
        return (o.v * do).sum() + (h.v * dh).sum()

    d, slope = _differences(f, p, name, 7)
    g = bo.selective_scan(**p, do=do, dh_final=dh)["d" + name]
    np.testing.assert_allclose((g.v * d).sum(), slope, rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("name", ["x", "w", "bias", "tail0"])
@pytest.mark.parametrize("N", [1, 2, 9])
def test_conv_gradients_are_differences(name, N):
    r = RNG(8)
    p = dict(x=r.standard_normal((N, 3)), w=r.standard_normal((3, 4)), bias=r.standard_normal(3),
             tail0=r.standard_normal((3, 3)))
    dy, dt = r.standard_normal((N, 3)), r.standard_normal((3, 3))

    def f(**a):
        y, t = bo.short_conv(**a)
        return (y.v * dy).sum() + (t.v * dt).sum()

    d, slope = _differences(f, p, name, 9)
    g = bo.short_conv(**p, dy=dy, dtail=dt)["d" + name]
    np.testing.assert_allclose((g.v * d).sum(), slope, rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("name", ["x", "y", "gate", "scale", "w_post", "w_next"])
def test_norm_gradients_are_differences(name):
    r = RNG(10)
    p = {k: r.standard_normal((4, 16)) for k in ("x", "y", "gate")}
    p.update({k: r.standard_normal(16) for k in ("scale", "w_post", "w_next")})
    dr, dn = r.standard_normal((4, 16)), r.standard_normal((4, 16))

    def f(**a):
        s, n = bo.residual_norm(**a)
        return (s.v * dr).sum() + (n.v * dn).sum()

    d, slope = _differences(f, p, name, 11)
    g = bo.residual_norm(**p, dr=dr, dn=dn)["d" + name]
    np.testing.assert_allclose((g.v * d).sum(), slope, rtol=1e-6, atol=1e-7)


def test_bounds_hold_in_fp32():
    # the same recurrence in numpy's fp32 stays inside the carried bound
    p = {k: np.asarray(v, np.float32) for k, v in _scan_inputs(12, 40, 3, 8).items()}
    o, h = bo.selective_scan(**p)
    s = p["h0"].copy()
    for t in range(40):
        d = np.log1p(np.exp(p["dt"][t] + p["dt_bias"])).astype(np.float32)
        s = np.exp(d[:, None] * p["A"]) * s + (d * p["u"][t])[:, None] * p["B"][t]
    assert (np.abs(s - h.v) <= h.e).all()


def test_softplus_polynomial_keeps_its_stated_error():
    """The polynomial that the kernels take for log1p(e) / e, read from their source, against log1p in 64 bits."""
    import os
    import re

    path = os.path.join(os.path.dirname(__file__), "..", "gated_retention_sequence_b200", "csrc", "gret_block.cuh")
    with open(path) as f:
        body = f.read().split("float2 softplus2(float2 x) {")[1].split("\n}")[0]
    coefficients = [np.float32(c) for c in re.findall(r"both\((-?[0-9.]+)f\)", body)]
    assert len(coefficients) == 10
    e = np.unique(np.concatenate([np.linspace(0, 1, 500001)[1:], np.logspace(-30, 0, 100001)]).astype(np.float32))
    x, want = e.astype(np.float64), np.log1p(e.astype(np.float64))
    exact, single = np.zeros_like(x), np.zeros_like(e)
    for c in coefficients:
        exact = exact * x + np.float64(c)
        # a fused multiply-add: the product of two fp32 is exact in 64 bits, the sum is rounded to 32
        single = (single.astype(np.float64) * x + np.float64(c)).astype(np.float32)
    single = (single.astype(np.float64) * x).astype(np.float32).astype(np.float64)
    unit = 2.0 ** -24
    assert np.abs(exact * x / want - 1).max() <= 0.56 * unit
    assert np.abs(single / want - 1).max() <= 2.6 * unit
