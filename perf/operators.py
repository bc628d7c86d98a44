"""Cases of the selective state space block's operators: the short causal convolution, the selective scan and the
residual norm, each for prompts, for single tokens and for training.

``listed`` and ``draw`` name cases, ``prepare`` makes their inputs on the GPU, ``run`` makes one pass and ``exact``
gives the same outputs in 64 bits.  With ``own`` false a pass is made of elementary torch operations in 32 bits; with
``own`` true it calls the library.

Formulas (t a token, d a channel, n a state; sigma the logistic function, swish(v) = v sigma(v)):

* short convolution   y[t,d] = act(bias[d] + sum_k w[d,k] x[t-K+1+k,d]), x before the first token from the tail of
  the tokens before (zero where there are none); the new tail is the last K-1 inputs.
* selective scan      delta[t,d] = softplus(dt[t,d] + dt_bias[d])
                      h[t,d,n] = exp(delta[t,d] A[d,n]) h[t-1,d,n] + delta[t,d] u[t,d] B[t,n]
                      o[t,d] = (sum_n C[t,n] h[t,d,n] + skip[d] u[t,d]) swish(z[t,d])
* residual norm       r = x + scale (.) rms(y) (.) w_post (.) swish(gate);  n = rms(r) (.) w_next,
                      rms(v) = v / sqrt(mean(v^2) + eps) over the row
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-5
MAX_WORK = 16384 * 2048          # tokens x channels a drawn case may have


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a prompt batch as a server packs it: 38 prompts of very different lengths, one of them empty and one of a
        # single token, each continued from an earlier piece
        {"name": "conv_prompt_packed", "op": "conv", "form": "packed", "tokens": 16384, "seqs": 38, "channels": 4096,
         "taps": 4, "type": "bf16"},
        # one decode step of a full serving batch
        {"name": "conv_step_256", "op": "conv", "form": "step", "tokens": 256, "seqs": 256, "channels": 4096, "taps": 4,
         "type": "bf16"},
        # the gradients of one layer of a training batch of 4 x 4096 tokens
        {"name": "conv_backward", "op": "conv", "form": "backward", "tokens": 16384, "seqs": 4, "channels": 4096,
         "taps": 4, "type": "bf16"},
        # the same packed prompts through the scan
        {"name": "scan_prompt_packed", "op": "scan", "form": "packed", "tokens": 16384, "seqs": 38, "channels": 4096,
         "states": 16, "type": "bf16"},
        # one long document and few channels, as a rank holds when the channels are split over several GPUs: the
        # only parallelism left is along the tokens
        {"name": "scan_prompt_long", "op": "scan", "form": "uniform", "tokens": 65536, "seqs": 1, "channels": 512,
         "states": 16, "type": "bf16"},
        # a check in full precision: odd lengths, a channel count that fills no block
        {"name": "scan_prompt_f32", "op": "scan", "form": "uniform", "tokens": 3 * 1021, "seqs": 3, "channels": 328,
         "states": 32, "type": "f32"},
        # one decode step of a full serving batch: the states are all there is to read
        {"name": "scan_step_256", "op": "scan", "form": "step", "tokens": 256, "seqs": 256, "channels": 4096,
         "states": 16, "type": "bf16"},
        # one decode step of a single user: latency
        {"name": "scan_step_1", "op": "scan", "form": "step", "tokens": 1, "seqs": 1, "channels": 2048, "states": 16,
         "type": "bf16"},
        # the gradients of one layer of a training batch of 4 x 4096 tokens
        {"name": "scan_backward", "op": "scan", "form": "backward", "tokens": 16384, "seqs": 4, "channels": 2048,
         "states": 16, "type": "bf16"},
        # after the block and before the next one, over a batch of prompts
        {"name": "norm_prompt", "op": "norm", "form": "forward", "tokens": 16384, "channels": 4096, "type": "bf16",
         "stream": "bf16"},
        # the same for the 8 tokens of a small decode batch: latency
        {"name": "norm_step_8", "op": "norm", "form": "forward", "tokens": 8, "channels": 2048, "type": "bf16",
         "stream": "bf16"},
        # its gradients in training, where the residual stream is kept in 32 bits
        {"name": "norm_backward", "op": "norm", "form": "backward", "tokens": 16384, "channels": 4096, "type": "bf16",
         "stream": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "norm"])
    channels = 8 * _log(rng, 8, 512)                       # 64 .. 4096
    c = {"op": op, "type": rng.choice(["bf16", "bf16", "f32"])}
    form = rng.choice({"conv": ["uniform", "packed", "step", "backward"],
                       "scan": ["uniform", "packed", "step", "backward"], "norm": ["forward", "backward"]}[op])
    most = max(1, MAX_WORK // channels)
    if form == "step":
        tokens = seqs = _log(rng, 1, 300)
    elif op == "norm":
        tokens, seqs = _log(rng, 1, min(16384, most)), 0
    elif form == "packed":
        tokens = _log(rng, 64, min(16384, most))
        seqs = _log(rng, 2, max(2, min(64, tokens // 8)))
    else:
        seqs = _log(rng, 1, 8)
        tokens = seqs * _log(rng, 1, max(1, min(16384, most) // seqs))
    c.update(form=form, tokens=tokens, channels=channels)
    if op == "norm":
        c["stream"] = "f32" if c["type"] == "f32" else rng.choice(["bf16", "f32"])
    else:
        c["seqs"] = seqs
    if op == "conv":
        c["taps"] = rng.choice([2, 3, 4, 4])
    if op == "scan":
        c["states"] = rng.choice([8, 16, 16, 32, 64])
        if form != "step":                                 # the plain form holds several values for each state
            keep = max(1, min(tokens, MAX_WORK * 16 // (channels * c["states"])))
            c["tokens"] = keep if form == "packed" else max(1, keep // seqs) * seqs
    return c


def _lengths(case):
    """Sequence lengths: equal ones, or for a packed batch a spread with an empty one and one of a single token."""
    T, S = case["tokens"], case["seqs"]
    if case["form"] != "packed":
        return [T // S] * S
    rng = random.Random("%d/%d" % (T, S))
    share = [math.exp(rng.uniform(0.0, 7.0)) for _ in range(S)]
    if S > 3:
        share[rng.randrange(S)] = 0.0
    whole = sum(share)
    lens = [int(T * s / whole) for s in share]
    if S > 4 and T > 100:
        lens[lens.index(min(v for v in lens if v > 0))] = 1
    lens[lens.index(max(lens))] += T - sum(lens)
    return lens


# ------------------------------------------------------------------ inputs
def _type(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    io, T, D, form = _type(case["type"]), case["tokens"], case["channels"], case["form"]

    def normal(*shape, std=1.0, mean=0.0, to=torch.float32):
        return (torch.randn(shape, generator=gen, device=dev) * std + mean).to(to)

    st = {"op": case["op"], "form": form, "io": io}
    if case["op"] == "norm":
        stream = _type(case["stream"])
        st.update(x=normal(T, D, std=3.0, to=stream), y=normal(T, D, to=io), gate=normal(T, D, to=io),
                  w_post=normal(D, std=0.1, mean=1.0), w_next=normal(D, std=0.1, mean=1.0),
                  scale=normal(D, std=0.1, mean=0.5))
        if form == "backward":
            st.update(dr=normal(T, D, to=stream), dn=normal(T, D, to=io))
        return st

    S, K = case["seqs"], case.get("taps", 0)
    lens = _lengths(case)
    cu = [0]
    for v in lens:
        cu.append(cu[-1] + v)
    st.update(S=S, N=T // S, longest=max(lens), lens=lens, cu=torch.tensor(cu, dtype=torch.int32, device=dev))
    starts = torch.zeros(T, dtype=torch.bool, device=dev)
    starts[[a for a, v in zip(cu, lens) if v]] = True
    st["starts"] = starts
    st["of"] = torch.repeat_interleave(torch.arange(S, device=dev), torch.tensor(lens, device=dev), output_size=T)
    st["pos"] = torch.arange(T, device=dev) - st["cu"].long()[st["of"]]
    if case["op"] == "conv":
        # x is the left half of the projection that also makes the gate z
        st["x"] = normal(T, 2 * D, to=io)[:, :D]
        st["w"] = (torch.rand(D, K, generator=gen, device=dev) * 2 - 1) / math.sqrt(K)
        st["bias"] = normal(D, std=0.1)
        st["tail"] = normal(S, K - 1, D, to=io)
        if form == "step":
            st["tail_out"] = torch.empty_like(st["tail"])
        if form == "backward":
            st["dy"] = normal(T, D, to=io)
            st["tail"] = None
        return st
    n = case["states"]
    pre = normal(T, D)
    st["u"] = (pre * torch.sigmoid(pre)).to(io)
    st["dt"] = normal(T, D, std=0.5, to=io)
    # step sizes spread over 0.001 .. 0.1, decays -1 .. -n: memories of one token to a thousand
    step = torch.exp(torch.rand(D, generator=gen, device=dev) * math.log(100.0) + math.log(0.001))
    st["dt_bias"] = torch.log(torch.expm1(step))
    st["A"] = -torch.arange(1, n + 1, device=dev, dtype=torch.float32) * torch.exp(normal(D, n, std=0.1))
    # B and C are columns of one projection, next to the low-rank input of dt
    bc = normal(T, 64 + 2 * n, to=io)
    st["B"], st["C"] = bc[:, 64:64 + n], bc[:, 64 + n:]
    st["z"] = normal(T, 2 * D, to=io)[:, D:]
    st["skip"] = normal(D, std=0.1, mean=1.0)
    st["h"] = None if form in ("uniform", "backward") else normal(S, D, n, std=0.1)
    if form == "step":
        st["h_out"] = torch.empty_like(st["h"])
    if form == "backward":
        st["do"] = normal(T, D, to=io)
        st["dh"] = normal(S, D, n, std=0.1)
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    if own:
        return _own(st)
    if st["op"] == "norm":
        return _norm_backward(st) if st["form"] == "backward" else _norm(st)
    if st["op"] == "conv":
        if st["form"] == "step":
            return _conv_step(st)
        return _conv_backward(st) if st["form"] == "backward" else _conv(st)
    if st["form"] == "step":
        return _scan_step(st)
    return _scan_backward(st) if st["form"] == "backward" else _scan(st)


def _own(st):
    import gated_retention_sequence_b200 as gret
    form = st["form"]
    if st["op"] == "norm":
        if form == "backward":
            return gret.residual_norm_backward(st["x"], st["y"], st["dr"], st["dn"], gate=st["gate"], scale=st["scale"],
                                               w_post=st["w_post"], w_next=st["w_next"], eps=EPS)
        r, n = gret.residual_norm(st["x"], st["y"], gate=st["gate"], scale=st["scale"], w_post=st["w_post"],
                                  w_next=st["w_next"], eps=EPS)
        return {"r": r, "n": n}
    S, N = st["S"], st["N"]

    def rows(t):
        return t.view(S, N, t.shape[-1]) if t.is_contiguous() else t.unflatten(0, (S, N))

    if st["op"] == "conv":
        if form == "step":
            y, tail = gret.short_conv_step(st["x"], st["w"], st["bias"], st["tail"], tail_out=st["tail_out"])
        elif form == "packed":
            y, tail = gret.short_conv_varlen(st["x"], st["w"], st["bias"], st["cu"], st["longest"], tail0=st["tail"])
        elif form == "uniform":
            y, tail = gret.short_conv(rows(st["x"]), st["w"], st["bias"], tail0=st["tail"])
            y = y.view(S * N, -1)
        else:
            g = gret.short_conv_backward(rows(st["x"]), st["w"], st["bias"], rows(st["dy"]))
            return {"dx": g["dx"].view(S * N, -1), "dw": g["dw"], "dbias": g["dbias"]}
        return {"y": y, "tail": tail}
    par = dict(skip=st["skip"], dt_bias=st["dt_bias"])
    if form == "step":
        o, h = gret.selective_step(st["u"], st["dt"], st["A"], st["B"], st["C"], st["h"], z=st["z"], h_out=st["h_out"],
                                   **par)
    elif form == "packed":
        o, h = gret.selective_scan_varlen(st["u"], st["dt"], st["A"], st["B"], st["C"], st["cu"], st["longest"],
                                          z=st["z"], h0=st["h"], **par)
    elif form == "uniform":
        o, h = gret.selective_scan(rows(st["u"]), rows(st["dt"]), st["A"], rows(st["B"]), rows(st["C"]),
                                   z=rows(st["z"]), **par)
        o = o.view(S * N, -1)
    else:
        g = gret.selective_scan_backward(rows(st["u"]), rows(st["dt"]), st["A"], rows(st["B"]), rows(st["C"]),
                                         rows(st["do"]), z=rows(st["z"]), dh_final=st["dh"], **par)
        return {k: g[k].view(S * N, -1) if k in ("du", "ddt", "dB", "dC", "dz") else g[k]
                for k in ("du", "ddt", "dA", "dB", "dC", "dz", "dskip", "ddt_bias")}
    return {"o": o, "h": h}


# ---- plain forms, in 32 bits
def _swish(v):
    return v * torch.sigmoid(v)


def _swish_slope(v):
    s = torch.sigmoid(v)
    return s * (1 + v * (1 - s))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _shifted(x, tail, st, by):
    """Row t of the result is row t - by of x; rows from before the first token come from the tail, or are zero."""
    if by == 0:
        return x
    T = x.shape[0]
    back = torch.clamp(torch.arange(T, device=x.device) - by, min=0)
    inside = (st["pos"] >= by)[:, None]
    if tail is None:
        return torch.where(inside, x[back], torch.zeros((), device=x.device))
    slot = torch.clamp(tail.shape[1] + st["pos"] - by, min=0, max=tail.shape[1] - 1)
    return torch.where(inside, x[back], tail[st["of"], slot])


def _conv(st):
    x, w, K = st["x"].float(), st["w"], st["w"].shape[1]
    tail = None if st["tail"] is None else st["tail"].float()
    s = st["bias"] + sum(w[:, k] * _shifted(x, tail, st, K - 1 - k) for k in range(K))
    # the last K-1 inputs of each sequence, from the old tail where it is shorter than that
    cu, R = st["cu"].long(), K - 1
    j = torch.arange(R, device=x.device)
    length = cu[1:] - cu[:-1]
    at = cu[1:, None] - R + j
    old = torch.clamp(length[:, None] + j, max=R - 1)
    inside = (length[:, None] - R + j >= 0)[..., None]
    before = torch.zeros((), device=x.device) if tail is None else tail[torch.arange(len(length), device=x.device)[:, None], old]
    new = torch.where(inside, x[torch.clamp(at, min=0, max=x.shape[0] - 1)], before)
    return {"y": _swish(s).to(st["io"]), "tail": new.to(st["io"])}


def _conv_step(st):
    window = torch.cat([st["tail"], st["x"][:, None]], 1)
    s = st["bias"] + (window.float() * st["w"].t()).sum(1)
    st["tail_out"].copy_(window[:, 1:])
    return {"y": _swish(s).to(st["io"]), "tail": st["tail_out"]}


def _conv_backward(st):
    x, w, dy, K, T = st["x"].float(), st["w"], st["dy"].float(), st["w"].shape[1], st["x"].shape[0]
    past = [_shifted(x, None, st, K - 1 - k) for k in range(K)]
    ds = dy * _swish_slope(st["bias"] + sum(w[:, k] * past[k] for k in range(K)))
    left = st["N"] - 1 - st["pos"]

    def ahead(by):
        at = torch.clamp(torch.arange(T, device=x.device) + by, max=T - 1)
        return torch.where((left >= by)[:, None], ds[at], torch.zeros((), device=x.device))

    dx = sum(w[:, k] * ahead(K - 1 - k) for k in range(K))
    return {"dx": dx.to(st["io"]), "dw": torch.stack([(ds * p).sum(0) for p in past], 1), "dbias": ds.sum(0)}


def _prefix(a, b, longest):
    """h_t = a_t h_(t-1) + b_t along the first axis, by doubling: after each pass (a, b) covers twice as many tokens.
    Overwrites a and b; a is zero where a sequence starts."""
    reach = 1
    while reach < longest:
        b[reach:] += a[reach:] * b[:-reach]
        a[reach:] = a[reach:] * a[:-reach]
        reach *= 2
    return b


def _states(st):
    """u, delta, the decays, the increments and the states, all in 32 bits."""
    u = st["u"].float()
    logits = st["dt"].float() + st["dt_bias"]
    delta = _softplus(logits)
    decay = torch.exp(delta[..., None] * st["A"])
    b = (delta * u)[..., None] * st["B"].float()[:, None, :]
    first = torch.nonzero(st["starts"])[:, 0]
    if st["h"] is not None:
        b[first] += decay[first] * st["h"][st["of"][first]]
    a = decay.clone()
    a[first] = 0
    return u, logits, delta, decay, _prefix(a, b, st["longest"])


def _scan(st):
    u, _, _, _, h = _states(st)
    y = (h * st["C"].float()[:, None, :]).sum(-1) + st["skip"] * u
    cu = st["cu"].long()
    last = h[torch.clamp(cu[1:] - 1, min=0)]
    none = torch.zeros_like(last) if st["h"] is None else st["h"]
    last = torch.where((cu[1:] > cu[:-1])[:, None, None], last, none)
    return {"o": (y * _swish(st["z"].float())).to(st["io"]), "h": last}


def _scan_step(st):
    u, delta = st["u"].float(), _softplus(st["dt"].float() + st["dt_bias"])
    h = torch.exp(delta[..., None] * st["A"]) * st["h"] + (delta * u)[..., None] * st["B"].float()[:, None, :]
    y = (h * st["C"].float()[:, None, :]).sum(-1) + st["skip"] * u
    st["h_out"].copy_(h)
    return {"o": (y * _swish(st["z"].float())).to(st["io"]), "h": st["h_out"]}


def _scan_backward(st):
    u, logits, delta, decay, h = _states(st)
    z, B, C, A, do = st["z"].float(), st["B"].float(), st["C"].float(), st["A"], st["do"].float()
    y = (h * C[:, None, :]).sum(-1) + st["skip"] * u
    dz = do * y * _swish_slope(z)
    dy = do * _swish(z)
    # the states' gradients run backwards: g_t = C_t dy_t + a_(t+1) g_(t+1), with dh_final at each last token
    T, N = u.shape[0], st["N"]
    last = torch.arange(N - 1, T, N, device=u.device)
    g = dy[..., None] * C[:, None, :]
    g[last] += st["dh"]
    a = torch.zeros_like(decay)
    a[:-1] = decay[1:]
    a[last] = 0
    g = _prefix(a.flip(0), g.flip(0), st["longest"]).flip(0)
    before = torch.zeros_like(h)
    before[1:] = h[:-1]
    before[st["starts"]] = 0
    through = g * before * decay                             # d / d(delta A)
    s = (g * B[:, None, :]).sum(-1)
    ddelta = (through * A).sum(-1) + u * s
    ddt = ddelta * torch.sigmoid(logits)
    io = st["io"]
    return {"du": (st["skip"] * dy + delta * s).to(io), "ddt": ddt.to(io), "dA": (through * delta[..., None]).sum(0),
            "dB": (g * (delta * u)[..., None]).sum(1).to(io), "dC": (h * dy[..., None]).sum(1).to(io),
            "dz": dz.to(io), "dskip": (dy * u).sum(0), "ddt_bias": ddt.sum(0)}


def _rms(v):
    return torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _norm(st):
    y = st["y"].float()
    r = st["x"].float() + st["scale"] * (y * _rms(y) * st["w_post"] * _swish(st["gate"].float()))
    return {"r": r.to(st["x"].dtype), "n": (r * _rms(r) * st["w_next"]).to(st["io"])}


def _norm_backward(st):
    x, y, gate, dn = st["x"].float(), st["y"].float(), st["gate"].float(), st["dn"].float()
    ky = _rms(y)
    yn = y * ky
    q, sw = yn * st["w_post"], _swish(gate)
    r = x + st["scale"] * (q * sw)
    kr = _rms(r)
    rn = r * kr
    t = dn * st["w_next"]
    dr = st["dr"].float() + kr * (t - rn * (t * rn).mean(-1, keepdim=True))
    dp = dr * st["scale"]
    dq = dp * sw
    e = dq * st["w_post"]
    dy = ky * (e - yn * (e * yn).mean(-1, keepdim=True))
    io = st["io"]
    return {"dx": dr.to(st["x"].dtype), "dy": dy.to(io), "dgate": (dp * q * _swish_slope(gate)).to(io),
            "dscale": (dr * q * sw).sum(0), "dw_post": (dq * yn).sum(0), "dw_next": (dn * rn).sum(0)}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    T, D = case["tokens"], case["channels"]
    e = {"bf16": 2, "f32": 4}[case["type"]]
    form, op = case["form"], case["op"]
    if op == "norm":
        s = {"bf16": 2, "f32": 4}[case["stream"]]
        if form == "backward":                            # x, dr, dx; y, gate, dn, dy, dgate; three weights and gradients
            return {"bytes": T * D * (3 * s + 5 * e) + 24 * D, "flops": 40 * T * D}
        return {"bytes": T * D * (2 * s + 3 * e) + 12 * D, "flops": 16 * T * D}
    S = case["seqs"]
    if op == "conv":
        K = case["taps"]
        tail = S * (K - 1) * D * e
        if form == "backward":                            # x, dy, dx; w, bias and their gradients
            return {"bytes": 3 * T * D * e + 8 * D * (K + 1), "flops": T * D * (6 * K + 10)}
        return {"bytes": 2 * T * D * e + 2 * tail + 4 * D * (K + 1),
                "flops": T * D * (2 * K + 6)}
    n = case["states"]
    par = 4 * D * (n + 2)                                 # A, skip, dt_bias
    if form == "backward":                                # u, dt, z, do, du, ddt, dz; B, C, dB, dC; dh_final
        return {"bytes": T * (7 * D + 4 * n) * e + 2 * par + 4 * S * D * n, "flops": T * D * (22 * n + 30)}
    state = 4 * S * D * n * (1 if form == "uniform" else 2)
    return {"bytes": T * (4 * D + 2 * n) * e + par + state, "flops": T * D * (7 * n + 12)}


# ------------------------------------------------------------------ the same in 64 bits, token by token
def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "norm":
        return _norm64(st)
    wide = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in st.items()}
    lens = st["lens"] if st["form"] != "step" else [1] * st["S"]
    return (_conv64 if st["op"] == "conv" else _scan64)(wide, lens)


def _grid(lens, dev):
    """For each token of the longest sequence: how many sequences have it, longest first, and its rows there."""
    lens = np.asarray(lens)
    first = np.cumsum(lens) - lens
    order = np.argsort(-lens, kind="stable")
    rows = torch.as_tensor(first[order], device=dev)
    count = [int((lens > t).sum()) for t in range(int(lens.max()))] if len(lens) > 1 else [1] * int(lens[0])
    return torch.as_tensor(order, device=dev), [(c, rows[:c] + t) for t, c in enumerate(count)]


def _conv64(st, lens):
    x, w, bias, K = st["x"], st["w"], st["bias"], st["w"].shape[1]
    tails = torch.zeros(len(lens), K - 1, x.shape[1], dtype=x.dtype, device=x.device) if st["tail"] is None else st["tail"]
    y, new, at = torch.empty_like(x), [], 0
    grads = st["form"] == "backward"
    dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(bias)
    for s, length in enumerate(lens):
        line = torch.cat([tails[s], x[at:at + length]])
        new.append(line[line.shape[0] - (K - 1):])
        if length:
            pieces = line.unfold(0, K, 1)                  # [length, D, K]
            s64 = torch.einsum("tdk,dk->td", pieces, w) + bias
            y[at:at + length] = s64 / (1 + torch.exp(-s64))
            if grads:
                sig = 1 / (1 + torch.exp(-s64))
                ds = st["dy"][at:at + length] * (sig + s64 * sig * (1 - sig))
                dw += torch.einsum("td,tdk->dk", ds, pieces)
                db += ds.sum(0)
                for k in range(K):
                    keep = length - (K - 1 - k)
                    if keep > 0:
                        dx[at:at + keep] += ds[K - 1 - k:] * w[:, k]
        at += length
    if grads:
        return {"dx": dx, "dw": dw, "dbias": db}
    return {"y": y, "tail": torch.stack(new)}


def _scan64(st, lens):
    u, A, B, C, z = st["u"], st["A"], st["B"], st["C"], st["z"]
    S, D, n, dev = len(lens), u.shape[1], A.shape[1], u.device
    raw = st["dt"] + st["dt_bias"]
    delta = torch.where(raw > 30, raw, torch.log1p(torch.exp(torch.clamp(raw, max=30))))
    grads = st["form"] == "backward"
    order, steps = _grid(lens, dev)
    h = torch.zeros(S, D, n, dtype=torch.float64, device=dev) if st["h"] is None else st["h"][order]
    y, kept = torch.empty_like(u), []
    for live, row in steps:
        if grads:
            kept.append(h.clone())
        h[:live] = torch.exp(delta[row, :, None] * A) * h[:live] + (delta[row] * u[row])[..., None] * B[row, None, :]
        y[row] = torch.einsum("sdn,sn->sd", h[:live], C[row])
    y = y + st["skip"] * u
    sig = 1 / (1 + torch.exp(-z))
    if not grads:
        back = torch.empty_like(h)
        back[order] = h
        return {"o": y * z * sig, "h": back}
    dy = st["do"] * z * sig
    dz = st["do"] * y * (sig + z * sig * (1 - sig))
    g = st["dh"].clone()
    du, dd, dA = st["skip"] * dy, torch.zeros_like(u), torch.zeros_like(A)
    dB, dC = torch.zeros_like(B), torch.zeros_like(C)
    for (_, row), old in zip(reversed(steps), reversed(kept)):   # every sequence has every token here
        dl, uu = delta[row], u[row]
        a = torch.exp(dl[..., None] * A)
        now = a * old + (dl * uu)[..., None] * B[row, None, :]
        g = g + dy[row][..., None] * C[row, None, :]
        dC[row] = torch.einsum("sdn,sd->sn", now, dy[row])
        dB[row] = torch.einsum("sdn,sd->sn", g, dl * uu)
        gb = torch.einsum("sdn,sn->sd", g, B[row])
        du[row] += dl * gb
        slope = g * a * old
        dd[row] = (slope * A).sum(-1) + uu * gb
        dA += (slope * dl[..., None]).sum(0)
        g = g * a
    ddt = dd / (1 + torch.exp(-raw))
    return {"du": du, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "dz": dz, "dskip": (dy * u).sum(0),
            "ddt_bias": ddt.sum(0)}


def _norm64(st):
    grads = st["form"] == "backward"
    names = ("x", "y", "gate", "scale", "w_post", "w_next")
    v = {k: st[k].double().requires_grad_(grads) for k in names}
    T = v["x"].shape[1]
    rms = lambda m: torch.sqrt(torch.einsum("td,td->t", m, m) / T + EPS)[:, None]  # noqa: E731
    r = v["x"] + v["scale"] * v["w_post"] * v["y"] / rms(v["y"]) * v["gate"] / (1 + torch.exp(-v["gate"]))
    n = v["w_next"] * r / rms(r)
    if not grads:
        return {"r": r, "n": n}
    g = torch.autograd.grad([r, n], [v[k] for k in names], [st["dr"].double(), st["dn"].double()])
    return {"d" + k: t for k, t in zip(names, g)}
