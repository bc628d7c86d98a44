"""The selective state space block's operators in 64 bits, with bounds on what fp32 arithmetic may be off.

Every value is a pair: the fp64 result and a bound on the error of the same formula evaluated in fp32, carried along
operation by operation (a running error analysis).  ``ULP`` is fp32's unit roundoff 2^-24; each rule adds the operation's
own rounding to what its operands bring in:

* a + b: |a| + |b| units, which covers a sum whose terms are joined in another order;
* a b:   one unit of the result;
* a sum of k terms: k units of the sum of magnitudes (any order);
* exp(x): 4 + 3|x| units (an exponential of 2 units, taken as 2^(x log2 e) with two roundings of the argument);
* sigmoid, softplus, 1/sqrt: 8 + 2|x|, 8 and 4 units.

``check`` holds a result to four times the bound (a recurrence cut into segments joins partial results that may be
larger than the whole) and half a step of the type it is stored in.
"""
from __future__ import annotations

import numpy as np

ULP = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SLACK = 4.0


class Val:
    """A value in 64 bits and a bound on its error in 32."""

    def __init__(self, v, e=None):
        self.v = np.asarray(v, dtype=np.float64)
        self.e = np.zeros_like(self.v) if e is None else np.asarray(e, dtype=np.float64)

    def __getitem__(self, i):
        return Val(self.v[i], self.e[i])

    def __add__(self, o):
        o = _val(o)
        return Val(self.v + o.v, self.e + o.e + (np.abs(self.v) + np.abs(o.v)) * ULP)

    def __sub__(self, o):
        o = _val(o)
        return self + Val(-o.v, o.e)

    def __mul__(self, o):
        o = _val(o)
        v = self.v * o.v
        return Val(v, np.abs(self.v) * o.e + np.abs(o.v) * self.e + self.e * o.e + np.abs(v) * ULP)

    __radd__, __rmul__ = __add__, __mul__

    def sum(self, axis, keepdims=False):
        k = self.v.shape[axis]
        return Val(self.v.sum(axis, keepdims=keepdims), self.e.sum(axis, keepdims=keepdims)
                   + k * np.abs(self.v).sum(axis, keepdims=keepdims) * ULP)


def _val(x):
    return x if isinstance(x, Val) else Val(x)


def _exp(x):
    v = np.exp(x.v)
    return Val(v, v * (np.expm1(x.e) + (4 + 3 * np.abs(x.v)) * ULP))


def _sigmoid(x):
    v = 1 / (1 + np.exp(-x.v))
    return Val(v, v * (1 - v) * x.e + v * (8 + 2 * np.abs(x.v)) * ULP)


def _softplus(x):
    v = np.logaddexp(0, x.v)
    return Val(v, x.e / (1 + np.exp(-x.v)) + 8 * v * ULP)


def _rsqrt(x):
    v = 1 / np.sqrt(x.v)
    return Val(v, 0.5 * v ** 3 * x.e + 4 * v * ULP)


def _swish(x):
    return x * _sigmoid(x)


def _swish_slope(x):
    s = _sigmoid(x)
    return s * (Val(1.0) + x * (Val(1.0) - s))


def _stack(items, axis=0):
    return Val(np.stack([i.v for i in items], axis), np.stack([i.e for i in items], axis))


def f64(t):
    return t if isinstance(t, Val) else Val(t.detach().to("cpu").double().numpy() if hasattr(t, "detach") else t)


def check(got, want, io, what=""):
    """|got - want| <= 4 bound + half a step of the storage type, element by element."""
    got = got.detach().to("cpu").double().numpy()
    assert got.shape == want.v.shape, (what, got.shape, want.v.shape)
    assert np.isfinite(got).all(), f"{what}: not finite"
    allowed = SLACK * want.e + HALF_STEP[io] * (np.abs(want.v) + SLACK * want.e) + 1e-37
    off = np.abs(got - want.v) / allowed
    assert off.size == 0 or off.max() <= 1, f"{what}: {off.max():.3g} times the bound at {np.unravel_index(off.argmax(), off.shape)}"


# ---- one sequence each: rows [N, ...]
def short_conv(x, w, bias=None, tail0=None, swish=True, dy=None, dtail=None):
    """Returns (y, tail), or the gradients of <y, dy> + <tail, dtail>: dx, dw, dbias, dtail0."""
    x, w = f64(x), f64(w)
    N, D = x.v.shape
    K = w.v.shape[1]
    past = Val(np.zeros((K - 1, D))) if tail0 is None else f64(tail0)
    line = np.concatenate([past.v, x.v])
    s = Val(np.zeros((N, D)) if bias is None else np.broadcast_to(f64(bias).v, (N, D)))
    for k in range(K):
        s = s + Val(line[k:k + N]) * w[:, k]
    if dy is None:
        return (_swish(s) if swish else s), Val(line[N:])
    ds = f64(dy) * (_swish_slope(s) if swish else Val(np.ones((N, D))))
    dline = Val(np.zeros((N + K - 1, D)))
    for k in range(K):
        pad = lambda a: np.concatenate([np.zeros((k, D)), a, np.zeros((K - 1 - k, D))])  # noqa: E731
        term = ds * w[:, k]
        dline = dline + Val(pad(term.v), pad(term.e))
    if dtail is not None:
        dline = dline + Val(np.concatenate([np.zeros((N, D)), f64(dtail).v]))
    dw = [(ds * Val(line[k:k + N])).sum(0) for k in range(K)]
    return {"dx": dline[K - 1:], "dtail0": dline[:K - 1], "dw": _stack(dw, 1), "dbias": ds.sum(0)}


def selective_scan(u, dt, A, B, C, skip=None, z=None, dt_bias=None, h0=None, do=None, dh_final=None):
    """Returns (o, h_final), or the gradients of <o, do> + <h_final, dh_final>."""
    u, dt, A, B, C = map(f64, (u, dt, A, B, C))
    N, D = u.v.shape
    n = A.v.shape[1]
    raw = dt if dt_bias is None else dt + f64(dt_bias)
    delta = _softplus(raw)
    h = Val(np.zeros((D, n))) if h0 is None else f64(h0)
    before, decays, states, ys = [], [], [], []
    for t in range(N):
        before.append(h)
        a = _exp(delta[t][:, None] * A)
        h = a * h + (delta[t] * u[t])[:, None] * B[t][None, :]
        decays.append(a)
        states.append(h)
        ys.append((h * C[t][None, :]).sum(1))
    y = _stack(ys) if N else Val(np.zeros((0, D)))
    if skip is not None:
        y = y + u * f64(skip)
    gate = None if z is None else _swish(f64(z))
    if do is None:
        return (y if gate is None else y * gate), h
    do = f64(do)
    dy = do if gate is None else do * gate
    out = {"dz": None if z is None else do * y * _swish_slope(f64(z))}
    g = Val(np.zeros((D, n))) if dh_final is None else f64(dh_final)
    du, ddelta, dB, dC = [], [], [], []
    dA = Val(np.zeros((D, n)))
    for t in reversed(range(N)):
        g = g + dy[t][:, None] * C[t][None, :]
        dC.append((states[t] * dy[t][:, None]).sum(0))
        dB.append((g * (delta[t] * u[t])[:, None]).sum(0))
        gb = (g * B[t][None, :]).sum(1)
        g = g * decays[t]
        slope = g * before[t]
        du.append(delta[t] * gb)
        ddelta.append((slope * A).sum(1) + u[t] * gb)
        dA = dA + slope * delta[t][:, None]
    du = _stack(du[::-1])
    out["du"] = du if skip is None else du + dy * f64(skip)
    ddt = _stack(ddelta[::-1]) * _sigmoid(raw)
    out.update(ddt=ddt, dA=dA, dB=_stack(dB[::-1]), dC=_stack(dC[::-1]), dh0=g, dskip=(dy * u).sum(0),
               ddt_bias=ddt.sum(0))
    return out


def residual_norm(x, y=None, gate=None, scale=None, w_post=None, w_next=None, eps=1e-5, dr=None, dn=None):
    """Returns (r, n), or with dr or dn the gradients of <r, dr> + <n, dn>."""
    x = f64(x)
    D = x.v.shape[-1]
    one = Val(np.ones(D))
    rms = lambda v: _rsqrt((v * v).sum(-1, True) * Val(1.0 / D) + Val(eps))  # noqa: E731
    w_post_, w_next_, scale_ = (one if w is None else f64(w) for w in (w_post, w_next, scale))
    r, yn, ky, q, sw = x, None, None, None, None
    if y is not None:
        yn = f64(y)
        if w_post is not None:
            ky = rms(yn)
            yn = yn * ky
        q = yn * w_post_
        sw = one if gate is None else _swish(f64(gate))
        r = x + q * sw * scale_
    kr = rms(r)
    rn = r * kr
    if dr is None and dn is None:
        return r, (None if w_next is None else rn * w_next_)
    out = {}
    total = Val(np.zeros_like(x.v)) if dr is None else f64(dr)
    if w_next is not None:
        t = f64(dn) * w_next_
        total = total + kr * (t - rn * ((t * rn).sum(-1, True) * Val(1.0 / D)))
        out["dw_next"] = (f64(dn) * rn).sum(0)
    out["dx"] = total
    if y is not None:
        dp = total * scale_
        dq = dp * sw
        out["dscale"] = (total * (q * sw)).sum(0)
        out["dw_post"] = (dq * yn).sum(0)
        if gate is not None:
            out["dgate"] = dp * q * _swish_slope(f64(gate))
        e = dq * w_post_
        out["dy"] = e if w_post is None else ky * (e - yn * ((e * yn).sum(-1, True) * Val(1.0 / D)))
    return out
