"""Cases and plain forms of the operators around the recurrence: root-mean-square
norm, short causal convolution and selective state space scan.

``listed()`` names the cases, ``draw`` makes more of the same ranges,
``prepare`` makes a case's inputs, ``run`` makes one pass through the operator
(its plain form in elementary torch operations, or, where ``own`` is true, the
library's call), ``work`` counts what a pass cannot do without and ``exact``
computes the same outputs from the definition in 64 bits.

rms norm       s = x (+ residual);  y = s / sqrt(mean(s^2) + eps) * weight, or
               y / scale in e4m3 with scale = max(amax |y|, 1e-10) / 448 over
               each group of columns
short conv     y_t = silu(bias + sum_j w[:, j] x_{t - W + 1 + j}), per channel
selective scan h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,
               y_t = (C_t . h_t + D x_t) silu(z_t),
               delta_t = softplus(dt_t + dt_bias)
"""
import math

import torch

own = False

EPS = 1e-6
FP8_MAX = 448.0
SCALE_FLOOR = 1e-10
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 256 sequences: the residual stream enters a layer (latency)
        dict(name="norm_step", op="norm", way="fwd", dtype="bf16", rows=256, dim=4096, residual=True, group=-1),
        # the recurrence's output of a batch, normalised per head and handed to an 8-bit projection
        dict(name="norm_heads_fp8", op="norm", way="fwd", dtype="bf16", rows=524288, dim=128, residual=False,
             group=128),
        # odd sizes, 32-bit residual stream, one scale a row
        dict(name="norm_odd_fp8", op="norm", way="fwd", dtype="f32", rows=3001, dim=1153, residual=True, group=0),
        # training: the gradient through the norm, joined with the residual stream's own gradient
        dict(name="norm_backward", op="norm", way="bwd", dtype="bf16", rows=16384, dim=4096, residual=True, group=-1),
        # prompts packed along one token axis, x one half of a joint projection
        dict(name="conv_packed", op="conv", way="fwd", dtype="bf16", tokens=65536, seqs=16, packed=True, dim=4096,
             width=4, bias=False, strided=True),
        # training: q, k, v's convolution; the gradient arrives in 32 bits from the recurrence
        dict(name="conv_backward", op="conv", way="bwd", dtype="bf16", tokens=16384, seqs=4, packed=False, dim=4096,
             width=4, bias=True, strided=False),
        # one decode step of 256 sequences over q, k and v of 32 heads of 128
        dict(name="conv_step", op="conv", way="step", dtype="bf16", tokens=256, seqs=256, packed=False, dim=12288,
             width=4, bias=False, strided=False),
        # a batch of prompts
        dict(name="scan_batch", op="scan", way="fwd", dtype="bf16", tokens=32768, seqs=8, packed=False, dim=4096,
             state=16, groups=1, gate=True),
        # one long document with few channels: too few rows to fill the card
        dict(name="scan_long", op="scan", way="fwd", dtype="bf16", tokens=65536, seqs=1, packed=False, dim=1024,
             state=16, groups=1, gate=True),
        # packed prompts of odd lengths, odd width, a wide state in groups, 32-bit activations
        dict(name="scan_odd", op="scan", way="fwd", dtype="f32", tokens=7919, seqs=7, packed=True, dim=1030, state=64,
             groups=2, gate=False),
        # training
        dict(name="scan_backward", op="scan", way="bwd", dtype="bf16", tokens=8192, seqs=4, packed=False, dim=4096,
             state=16, groups=1, gate=True),
        # one decode step of 256 sequences
        dict(name="scan_step", op="scan", way="step", dtype="bf16", tokens=256, seqs=256, packed=False, dim=4096,
             state=16, groups=1, gate=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, evenly over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "conv", "scan"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        way = rng.choice(["fwd", "fwd", "bwd"])
        dim = rng.choice([64, 128, 256, 1000, 1024, 2048, 4096, 7168, _spread(rng, 17, 8192)])
        rows = _spread(rng, 1, max(1, (1 << 24) // dim))
        groups = [-1, -1, 0] + ([128] if dim % 128 == 0 else []) + ([32] if dim % 32 == 0 else [])
        return dict(op=op, way=way, dtype=dtype, rows=rows, dim=dim, residual=rng.random() < 0.5,
                    group=-1 if way == "bwd" else rng.choice(groups))
    way = rng.choice(["fwd", "fwd", "bwd", "step"])
    seqs = _spread(rng, 1, 256) if way == "step" else _spread(rng, 1, 16)
    if op == "conv":
        dim = rng.choice([256, 1024, 4096, _spread(rng, 33, 8192)])
        tokens = seqs if way == "step" else seqs * _spread(rng, 1, max(1, (1 << 25) // (dim * seqs)))
        return dict(op=op, way=way, dtype=dtype, tokens=tokens, seqs=seqs, packed=way != "step" and rng.random() < 0.5,
                    dim=dim, width=rng.choice([2, 3, 4, 4]), bias=rng.random() < 0.5,
                    strided=way == "fwd" and rng.random() < 0.5)
    state = rng.choice([8, 16, 16, 32, 64])
    groups = rng.choice([1, 1, 2])
    dim = groups * rng.choice([128, 512, 1024, _spread(rng, 33, 2048)])
    tokens = seqs
    if way != "step":
        most = min((1 << 28) // (dim * state), 4096 if way == "bwd" else 16384)
        tokens = seqs * _spread(rng, 1, max(1, most // seqs))
    return dict(op=op, way=way, dtype=dtype, tokens=tokens, seqs=seqs, packed=way != "step" and rng.random() < 0.5,
                dim=dim, state=state, groups=groups, gate=rng.random() < 0.7)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _lengths(case, gen):
    """Lengths of the packed sequences (sum = tokens), uneven and from 1 token up."""
    n, total = case["seqs"], case["tokens"]
    share = torch.rand(n, generator=gen, dtype=torch.float64) + 0.05
    at = (share.cumsum(0) / share.sum() * (total - n)).round().long()
    at[-1] = total - n
    return [int(b) - int(a) + 1 for a, b in zip([0] + at[:-1].tolist(), at.tolist())]


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev) * std + mean).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=gen, device=dev) * (hi - lo) + lo

    st = dict(case)
    if case["op"] == "norm":
        r, d = case["rows"], case["dim"]
        st["weight"] = normal(d, std=0.1, mean=1.0)
        if case["way"] == "bwd":
            st["s"] = normal(r, d, std=1.5)
            st["dy"] = normal(r, d)
            st["ds"] = normal(r, d) if case["residual"] else None
        else:
            st["x"] = normal(r, d)
            st["residual_in"] = normal(r, d, std=2.0) if case["residual"] else None
        return st

    n, t, d = case["seqs"], case["tokens"], case["dim"]
    st["lens"], st["cu"] = [t // n] * n, None
    shape = (n, t // n)
    if case["way"] == "step":
        shape = (n,)
    elif case["packed"]:
        st["lens"] = _lengths(case, host)
        edges = [0]
        for x in st["lens"]:
            edges.append(edges[-1] + x)
        st["cu"] = torch.tensor(edges, dtype=torch.int32, device=dev)
        shape = (1, t)

    if case["op"] == "conv":
        w = case["width"]
        st["x"] = normal(*shape, 2 * d)[..., :d] if case["strided"] else normal(*shape, d)
        st["weight"] = uniform(d, w, lo=-1.0, hi=1.0).mul_(w ** -0.5).to(dt)
        st["b"] = normal(d, std=0.1) if case["bias"] else None
        st["state"] = normal(n, w - 1, d)
        if case["way"] == "step":
            st["state_out"] = torch.empty_like(st["state"])
        if case["way"] == "bwd":
            st["dy"] = normal(*shape, d, dtype=torch.float32)
            st["dstate"] = normal(n, w - 1, d, dtype=torch.float32)
        return st

    s, g = case["state"], case["groups"]
    st["x"] = normal(*shape, d)
    st["dt"] = normal(*shape, d, std=0.5)
    st["A"] = -(torch.arange(1, s + 1, device=dev, dtype=torch.float32) * torch.exp(normal(d, s, std=0.1, dtype=torch.float32)))
    st["B"] = normal(*shape, g, s)
    st["C"] = normal(*shape, g, s)
    st["D"] = normal(d, std=0.2, mean=1.0, dtype=torch.float32)
    st["z"] = normal(*shape, 2 * d)[..., d:] if case["gate"] else None
    first = torch.exp(uniform(d, lo=math.log(1e-3), hi=math.log(1e-1)))  # time steps of 0.001 to 0.1
    st["dt_bias"] = torch.log(torch.expm1(first))
    st["S0"] = normal(n, d, s, std=0.1, dtype=torch.float32)
    if case["way"] == "bwd":
        st["dy"] = normal(*shape, d)
        st["dS"] = normal(n, d, s, std=0.1, dtype=torch.float32)
    if case["way"] == "step":
        st["S_out"] = torch.empty_like(st["S0"])  # the next state beside the old one, as speculative decoding keeps it
    return st


# ---------------------------------------------------------------------------
# Plain forms (32 bits)
# ---------------------------------------------------------------------------
def _norm_plain(st):
    dt = DT[st["dtype"]]
    w = st["weight"].float()
    if st["way"] == "bwd":
        s, dy = st["s"].float(), st["dy"].float()
        r = torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS)
        wdy = dy * w
        dx = wdy * r - s * (r * r * r) * (wdy * s).mean(-1, keepdim=True)
        if st["ds"] is not None:
            dx = dx + st["ds"].float()
        return dx.to(dt), (dy * s * r).sum(0)
    s = st["x"].float()
    if st["residual_in"] is not None:
        s = s + st["residual_in"].float()
    y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS) * w
    out = s.to(dt) if st["residual_in"] is not None else None
    if st["group"] < 0:
        return (y.to(dt),) + ((out,) if out is not None else ())
    rows, d = y.shape
    yg = y.view(rows, -1, st["group"] or d)
    scale = yg.abs().amax(-1).clamp_min(SCALE_FLOOR) / FP8_MAX
    q = (yg / scale[..., None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(rows, d)
    return (q, scale) + ((out,) if out is not None else ())


def _conv_rows(st, x, state, kind):
    """Every sequence's rows, the kept inputs before the first among them: [n tokens + width - 1, dim]."""
    flat = x.reshape(-1, st["dim"]).to(kind)
    at, rows = 0, []
    for i, n in enumerate(st["lens"]):
        rows.append(torch.cat([state[i].to(kind), flat[at:at + n]], 0))
        at += n
    return rows


def _conv_plain(st):
    dt, w, wd = DT[st["dtype"]], st["width"], st["weight"].float()
    b = st["b"].float() if st["b"] is not None else 0.0
    if st["way"] == "step":
        rows = torch.cat([st["state"].float(), st["x"].float()[:, None]], 1)
        p = (rows * wd.t()[None]).sum(1) + b
        return (p * torch.sigmoid(p)).to(dt), rows[:, 1:].to(dt)
    rows = _conv_rows(st, st["x"], st["state"], torch.float32)
    if st["way"] == "fwd":
        ys = []
        for r in rows:
            n = r.shape[0] - w + 1
            p = sum(r[j:j + n] * wd[:, j] for j in range(w)) + b
            ys.append(p * torch.sigmoid(p))
        y = torch.cat(ys, 0).to(dt).view(st["x"].shape)
        return y, torch.stack([r[r.shape[0] - w + 1:] for r in rows]).to(dt)
    dy = st["dy"].reshape(-1, st["dim"])
    at, dxs, dinit = 0, [], []
    dw, db = torch.zeros_like(wd), torch.zeros(st["dim"], device=wd.device)
    for i, r in enumerate(rows):
        n = r.shape[0] - w + 1
        p = sum(r[j:j + n] * wd[:, j] for j in range(w)) + b
        sg = torch.sigmoid(p)
        dp = dy[at:at + n] * sg * (1 + p * (1 - sg))
        dr = torch.zeros_like(r)
        for j in range(w):
            dr[j:j + n] += dp * wd[:, j]
            dw[:, j] += (dp * r[j:j + n]).sum(0)
        db += dp.sum(0)
        dr[n:] += st["dstate"][i]
        dinit.append(dr[:w - 1])
        dxs.append(dr[w - 1:])
        at += n
    out = (torch.cat(dxs, 0).to(dt).view(st["x"].shape), dw, torch.stack(dinit))
    return out + ((db,) if st["b"] is not None else ())


def _softplus(v):
    return v.clamp_min(0) + torch.log1p(torch.exp(-v.abs()))


def _scan_pieces(st, piece):
    """Token indices [pieces, piece] of every sequence cut into pieces (-1 past
    its end), and the pieces of each sequence in order, [seqs, most] (-1: none)."""
    index, of, at = [], [], 0
    for n in st["lens"]:
        k = -(-n // piece)
        idx = torch.arange(k * piece)
        idx = torch.where(idx < n, idx + at, torch.full_like(idx, -1))
        of.append(list(range(sum(map(len, of)), sum(map(len, of)) + k)))
        index.append(idx.view(k, piece))
        at += n
    most = max(map(len, of))
    table = torch.tensor([o + [-1] * (most - len(o)) for o in of])
    dev = st["x"].device
    return torch.cat(index).to(dev), table.to(dev)


def _scan_inputs(st, index):
    """Inputs cut into pieces, in 32 bits; a place past a sequence's end gets
    delta = 0, which leaves the state as it is."""
    d, s, g = st["dim"], st["state"], st["groups"]
    live = (index >= 0)[..., None]
    at = index.clamp_min(0)

    def cut(v, *shape):
        return v.reshape(-1, *shape)[at].float()

    raw = cut(st["dt"], d) + st["dt_bias"]
    delta = torch.where(live, _softplus(raw), torch.zeros_like(raw))
    x = torch.where(live, cut(st["x"], d), torch.zeros_like(raw))
    each = d // g
    # B and C of a group, spread over its channels
    bm = cut(st["B"], g, s)
    cm = torch.where(live[..., None], cut(st["C"], g, s), torch.zeros_like(bm))
    return raw, delta, x, bm, cm, each


def _per_channel(v, each):
    return v.repeat_interleave(each, dim=1) if v.shape[1] > 1 else v


def _piece_length(case):
    return max(8, min(128, round(math.sqrt(max(case["lens"]) / 2))))


def _scan_entries(st, delta, x, bm, table, each):
    """The state before every piece: local states, then the pieces in order."""
    A = st["A"]
    n, d, s = st["seqs"], st["dim"], st["state"]
    local = torch.zeros(delta.shape[0], d, s, device=A.device)
    for t in range(delta.shape[1]):
        dl = delta[:, t, :, None]
        local = torch.exp(dl * A) * local + dl * x[:, t, :, None] * _per_channel(bm[:, t], each)
    total = torch.exp(delta.double().sum(1)[..., None] * A.double()).float()
    entry = torch.zeros_like(local)
    h = st["S0"].clone()
    for k in range(table.shape[1]):
        at, live = table[:, k].clamp_min(0), (table[:, k] >= 0)[:, None, None]
        entry[at[table[:, k] >= 0]] = h[table[:, k] >= 0]
        h = torch.where(live, total[at] * h + local[at], h)
    return entry, h, total


def _uncut(v, index, like):
    flat = torch.empty((int((index >= 0).sum()),) + v.shape[2:], device=v.device)
    flat[index[index >= 0]] = v[index >= 0]
    return flat.view(like)


def _scan_plain(st):
    dt, A = DT[st["dtype"]], st["A"]
    d, s, g = st["dim"], st["state"], st["groups"]
    if st["way"] == "step":
        delta = _softplus(st["dt"].float() + st["dt_bias"])
        x = st["x"].float()
        each = d // g
        h = torch.exp(delta[..., None] * A) * st["S0"] + (delta * x)[..., None] * _per_channel(st["B"].float(), each)
        y = (h * _per_channel(st["C"].float(), each)).sum(-1) + st["D"] * x
        if st["z"] is not None:
            z = st["z"].float()
            y = y * z * torch.sigmoid(z)
        return y.to(dt), h
    index, table = _scan_pieces(st, _piece_length(st))
    raw, delta, x, bm, cm, each = _scan_inputs(st, index)
    entry, last, total = _scan_entries(st, delta, x, bm, table, each)
    length = index.shape[1]
    at = index.clamp_min(0)
    z = st["z"].reshape(-1, d)[at].float() if st["z"] is not None else None
    h, yy, kept = entry, torch.empty_like(x), []
    for t in range(length):
        dl = delta[:, t, :, None]
        if st["way"] == "bwd":
            kept.append(h)
        h = torch.exp(dl * A) * h + dl * x[:, t, :, None] * _per_channel(bm[:, t], each)
        yy[:, t] = (h * _per_channel(cm[:, t], each)).sum(-1)
    yy = yy + st["D"] * x
    if st["way"] == "fwd":
        y = yy if z is None else yy * z * torch.sigmoid(z)
        return _uncut(y, index, st["x"].shape).to(dt), last

    dyo = torch.where((index >= 0)[..., None], st["dy"].reshape(-1, d)[at].float(), torch.zeros_like(x))
    dyy, dz = dyo, None
    if z is not None:
        sg = torch.sigmoid(z)
        dyy = dyo * z * sg
        dz = dyo * yy * sg * (1 + z * (1 - sg))
    # the gradient that enters every piece from its right: local ones, then the pieces from the last to the first
    r = torch.zeros_like(entry)
    for t in reversed(range(length)):
        r = torch.exp(delta[:, t, :, None] * A) * (dyy[:, t, :, None] * _per_channel(cm[:, t], each) + r)
    right = torch.zeros_like(entry)
    carry = st["dS"].clone()
    for k in reversed(range(table.shape[1])):
        on, live = table[:, k].clamp_min(0), (table[:, k] >= 0)[:, None, None]
        right[on[table[:, k] >= 0]] = carry[table[:, k] >= 0]
        carry = torch.where(live, total[on] * carry + r[on], carry)
    dS0 = carry
    ddelta, dx = torch.empty_like(x), torch.empty_like(x)
    dB = torch.empty_like(bm)
    dC = torch.empty_like(cm)
    dA = torch.zeros_like(A)
    r, h = right, h
    for t in reversed(range(length)):
        dl, xt = delta[:, t, :, None], x[:, t, :, None]
        b, c = _per_channel(bm[:, t], each), _per_channel(cm[:, t], each)
        gr = dyy[:, t, :, None] * c + r
        dC[:, t] = (dyy[:, t, :, None] * h).view(-1, g, each, s).sum(2)
        before = kept[t]
        r = torch.exp(dl * A) * gr
        ra = r * before
        dA += (dl * ra).sum(0)
        gb = (gr * b).sum(-1)
        ddelta[:, t] = (ra * A).sum(-1) + gb * x[:, t]
        dx[:, t] = gb * delta[:, t]
        dB[:, t] = (gr * (dl * xt)).view(-1, g, each, s).sum(2)
        h = before
    dx = dx + dyy * st["D"]
    ddt = ddelta * torch.sigmoid(raw)
    ddt = torch.where((index >= 0)[..., None], ddt, torch.zeros_like(ddt))
    shape = st["x"].shape
    out = (_uncut(dx, index, shape).to(dt), _uncut(ddt, index, shape).to(dt), dA,
           _uncut(dB, index, st["B"].shape), _uncut(dC, index, st["C"].shape), (dyy * x).sum((0, 1)),
           ddt.sum((0, 1)), dS0)
    return out + ((_uncut(dz, index, shape).to(dt),) if dz is not None else ())


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def _own_run(st):
    import kimi_delta_attention_31_b200 as kda
    op, way = st["op"], st["way"]
    if op == "norm":
        if way == "bwd":
            g = kda.rms_norm_bwd(st["dy"], st["s"], st["weight"], ds=st["ds"], eps=EPS)
            return g["dx"], g["dweight"]
        if st["group"] < 0:
            y, s = kda.rms_norm_fwd(st["x"], st["weight"], st["residual_in"], eps=EPS)
            return (y,) + ((s,) if s is not None else ())
        q, scale, s = kda.rms_norm_quant_fwd(st["x"], st["weight"], st["residual_in"], eps=EPS, group=st["group"])
        return (q, scale) + ((s,) if s is not None else ())
    if op == "conv":
        if way == "step":
            y = kda.short_conv_step(st["x"], st["weight"], st["state"], st["b"], state_out=st["state_out"])
            return y, st["state_out"]
        if way == "fwd":
            return kda.short_conv_fwd(st["x"], st["weight"], st["b"], st["state"], st["cu"])
        g = kda.short_conv_bwd(st["x"], st["weight"], st["dy"], st["b"], st["state"], st["dstate"], st["cu"])
        return (g["dx"], g["dweight"], g["dinit"]) + ((g["dbias"],) if st["b"] is not None else ())
    if way == "step":
        y = kda.selective_scan_step(st["x"], st["dt"], st["A"], st["B"], st["C"], st["S0"], st["D"], st["z"],
                                    st["dt_bias"], S_out=st["S_out"])
        return y, st["S_out"]
    if way == "fwd":
        return kda.selective_scan_fwd(st["x"], st["dt"], st["A"], st["B"], st["C"], st["D"], st["z"], st["dt_bias"],
                                      st["S0"], st["cu"])
    g = kda.selective_scan_bwd(st["x"], st["dt"], st["A"], st["B"], st["C"], st["dy"], st["D"], st["z"],
                               st["dt_bias"], st["S0"], st["dS"], st["cu"])
    names = ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dS0") + (("dz",) if st["z"] is not None else ())
    return tuple(g[n] for n in names)


def run(state):
    if own:
        return _own_run(state)
    return {"norm": _norm_plain, "conv": _conv_plain, "scan": _scan_plain}[state["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        r, d = case["rows"], case["dim"]
        n = r * d
        if case["way"] == "bwd":
            return dict(bytes=n * e * (4 if case["residual"] else 3) + d * (e + 4), flops=12.0 * n)
        out = n * e if case["group"] < 0 else n + 4 * r * (d // (case["group"] or d))
        return dict(bytes=n * e * (3 if case["residual"] else 1) + out + d * e, flops=5.0 * n)
    t, d, n = case["tokens"], case["dim"], case["seqs"]
    if case["op"] == "conv":
        w = case["width"]
        keep = n * (w - 1) * d
        par = d * (w + (1 if case["bias"] else 0))
        if case["way"] == "bwd":
            return dict(bytes=t * d * (2 * e + 4) + keep * (e + 8) + par * (e + 4), flops=t * d * (6.0 * w + 10))
        return dict(bytes=2 * t * d * e + 2 * keep * e + par * e, flops=t * d * (2.0 * w + 5))
    s, g = case["state"], case["groups"]
    z = 1 if case["gate"] else 0
    par, keep = d * s * 4 + 8 * d, n * d * s * 4
    if case["way"] == "bwd":
        return dict(bytes=t * d * e * (5 + 2 * z) + t * g * s * (2 * e + 8) + 2 * par + 3 * keep,
                    flops=22.0 * t * d * s)
    return dict(bytes=t * d * e * (3 + z) + 2 * t * g * s * e + par + 2 * keep, flops=7.0 * t * d * s)


# ---------------------------------------------------------------------------
# The same from the definitions, in 64 bits, token by token
# ---------------------------------------------------------------------------
def _exact_norm(st):
    f = torch.float64
    w = st["weight"].to(f)
    if st["way"] == "bwd":
        s, dy = st["s"].to(f), st["dy"].to(f)
        d = s.shape[1]
        q = s.square().sum(1, keepdim=True) / d + EPS
        n = s / q.sqrt()
        dn = dy * w
        dx = (dn - n * (dn * n).sum(1, keepdim=True) / d) / q.sqrt()
        return (dx if st["ds"] is None else dx + st["ds"].to(f)), (dy * n).sum(0)
    s = st["x"].to(f)
    if st["residual_in"] is not None:
        s = s + st["residual_in"].to(f)
    y = s / (s.square().sum(1, keepdim=True) / s.shape[1] + EPS).sqrt() * w
    tail = (s,) if st["residual_in"] is not None else ()
    if st["group"] < 0:
        return (y,) + tail
    width = st["group"] or y.shape[1]
    cols = y.reshape(y.shape[0], y.shape[1] // width, width)
    scale = cols.abs().max(2).values.clamp_min(SCALE_FLOOR) / FP8_MAX
    return ((cols / scale.unsqueeze(2)).reshape(y.shape), scale) + tail


def _exact_conv(st):
    f = torch.float64
    d, w = st["dim"], st["width"]
    wt = st["weight"].to(f)
    bias = st["b"].to(f) if st["b"] is not None else torch.zeros(d, dtype=f, device=wt.device)
    x = st["x"].to(f).reshape(-1, d)
    y, dx = torch.empty_like(x), torch.zeros_like(x)
    dw, db = torch.zeros_like(wt), torch.zeros_like(bias)
    states, dinits = [], []
    start = 0
    for i, n in enumerate(st["lens"]):
        rows = torch.cat([st["state"][i].to(f), x[start:start + n]])
        windows = rows.unfold(0, w, 1)  # [n, d, w]
        p = (windows * wt).sum(2) + bias
        sg = 1 / (1 + torch.exp(-p))
        y[start:start + n] = p * sg
        states.append(rows[n:])
        if st["way"] == "bwd":
            dp = st["dy"].to(f).reshape(-1, d)[start:start + n] * (sg + p * sg * (1 - sg))
            dw += (windows * dp.unsqueeze(2)).sum(0)
            db += dp.sum(0)
            drows = torch.zeros_like(rows)
            drows[n:] = st["dstate"][i].to(f)
            for j in range(w):
                drows[j:j + n] += dp * wt[:, j]
            dinits.append(drows[:w - 1])
            dx[start:start + n] = drows[w - 1:]
        start += n
    if st["way"] == "bwd":
        out = (dx.view(st["x"].shape), dw, torch.stack(dinits))
        return out + ((db,) if st["b"] is not None else ())
    return y.view(st["x"].shape), torch.stack(states)


def _exact_scan(st):
    f = torch.float64
    n, d, s, g = st["seqs"], st["dim"], st["state"], st["groups"]
    dev = st["x"].device
    most = max(st["lens"]) if st["way"] != "step" else 1
    lens = st["lens"] if st["way"] != "step" else [1] * n
    starts = [sum(lens[:i]) for i in range(n)]
    pos = torch.arange(most, device=dev)[None]
    live = pos < torch.tensor(lens, device=dev)[:, None]
    at = torch.where(live, pos + torch.tensor(starts, device=dev)[:, None], torch.zeros_like(pos))
    group = torch.arange(d, device=dev) // (d // g)

    def rows(name, *shape):
        return st[name].reshape(-1, *shape)

    A = st["A"].to(f)

    def token(t):
        i = at[:, t]
        raw = rows("dt", d)[i].to(f) + st["dt_bias"].to(f)
        delta = torch.log1p(torch.exp(-raw.abs())) + raw.clamp_min(0)
        return (i, raw, delta, rows("x", d)[i].to(f), rows("B", g, s)[i].to(f)[:, group],
                rows("C", g, s)[i].to(f)[:, group])

    total = sum(lens)
    h = st["S0"].to(f)
    yy = torch.zeros(total, d, dtype=f, device=dev)
    keep = []
    for t in range(most):
        on = live[:, t]
        i, raw, delta, x, b, c = token(t)
        if st["way"] == "bwd":
            keep.append(h)
        new = torch.exp(delta[..., None] * A) * h + (delta * x)[..., None] * b
        h = torch.where(on[:, None, None], new, h)
        yt = (c * h).sum(2) + st["D"].to(f) * x
        yy[i[on]] = yt[on]
    shape = st["x"].shape
    z = rows("z", d).to(f) if st["z"] is not None else None
    sig = 1 / (1 + torch.exp(-z)) if z is not None else None
    if st["way"] != "bwd":
        return (yy if z is None else yy * z * sig).view(shape), h
    dyo = rows("dy", d).to(f)
    dyy = dyo if z is None else dyo * z * sig
    dx, ddt = torch.zeros_like(yy), torch.zeros_like(yy)
    dB = torch.zeros(total, g, s, dtype=f, device=dev)
    dC = torch.zeros_like(dB)
    dA, dD, dbias = torch.zeros_like(A), torch.zeros(d, dtype=f, device=dev), torch.zeros(d, dtype=f, device=dev)
    gr = st["dS"].to(f)
    for t in reversed(range(most)):
        on = live[:, t, None, None]
        i, raw, delta, x, b, c = token(t)
        dyt = dyy[i]
        a = torch.exp(delta[..., None] * A)
        after = a * keep[t] + (delta * x)[..., None] * b
        full = gr + dyt[..., None] * c
        m = torch.where(on, full, torch.zeros_like(full))
        ddelta = (m * (A * a * keep[t] + b * x[..., None])).sum(2)
        dr = ddelta / (1 + torch.exp(-raw))
        o = live[:, t]
        dx[i[o]] = ((m * b).sum(2) * delta + dyt * st["D"].to(f))[o]
        ddt[i[o]] = dr[o]
        dbias += dr.sum(0)
        dD += (dyt * x)[o].sum(0)
        dA += (m * a * keep[t] * delta[..., None]).sum(0)
        dB[i[o]] = (m * (delta * x)[..., None]).view(n, g, d // g, s).sum(2)[o]
        dC[i[o]] = (dyt[..., None] * after).view(n, g, d // g, s).sum(2)[o]
        gr = torch.where(on, a * full, gr)
    out = (dx.view(shape), ddt.view(shape), dA, dB.view(st["B"].shape), dC.view(st["C"].shape), dD, dbias, gr)
    if z is not None:
        out += ((dyo * yy * sig * (1 + z * (1 - sig))).view(shape),)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "conv": _exact_conv, "scan": _exact_scan}[case["op"]](st)
