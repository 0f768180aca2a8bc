"""GPU: short causal convolution (prefill, step, backward) against the 64-bit
form.  Bounds: p is a sum of W + 1 products in fp32, off by at most 2^-21 of the
sum of their sizes; sigmoid adds 2^-22 (8 + |p|) relative; |d silu| <= 1.1 and
|d (silu')| <= 0.5; a stored value adds half a step."""
import pytest
import torch

import kimi_delta_attention_31_b200 as kda
import layer_ref as R
from layer_ref import F64, U, rel_rms, within

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _inputs(dev, lens, D, W, dtype, seed, bias=True, packed=True, wdtype=None):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=dev)
    N, T = len(lens), sum(lens)
    lead = (1, T) if packed else (N, lens[0])
    wdtype = wdtype or dtype
    d = dict(x=r(*lead, D).to(dtype), weight=(r(D, W) * W ** -0.5).to(wdtype), bias=r(D).to(wdtype) if bias else None,
             state=r(N, W - 1, D).to(dtype))
    d["cu"] = torch.tensor(R.bounds(lens), dtype=torch.int32, device=dev) if packed else None
    return d


def _c(t):
    return None if t is None else t.detach().cpu().to(F64)


def _flat(t):
    return _c(t).reshape(-1, t.shape[-1])


def _p_size(d, lens):
    """sum of the sizes of p's terms, and p."""
    W = d["weight"].shape[1]
    x, w, b, st = _flat(d["x"]), _c(d["weight"]), _c(d["bias"]), _c(d["state"])
    ps, sizes, at = [], [], 0
    for n, length in enumerate(lens):
        rows = torch.cat([st[n], x[at:at + length]])
        at += length
        for t in range(length):
            terms = rows[t:t + W] * w.t()
            ps.append(terms.sum(0) + (0 if b is None else b))
            sizes.append(terms.abs().sum(0) + (0 if b is None else b.abs()))
    return torch.stack(ps), torch.stack(sizes)


CASES = [((1,), 1, 4), ((2,), 33, 4), ((3,), 64, 3), ((5, 5), 128, 2), ((70,), 1024, 4), ((17, 17, 17), 1032, 4),
         ((0, 1, 2, 3, 0, 40, 0), 48, 4), ((0, 130, 1, 1, 1, 65), 100, 3), ((200,), 257, 2), ((0, 0), 16, 4)]


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("lens,D,W", CASES)
def test_conv(cuda_device, lens, D, W, dtype, wdtype):
    dt = DT[dtype]
    packed = len(set(lens)) > 1
    d = _inputs(cuda_device, lens, D, W, dt, sum(lens) + D, D % 3 != 0, packed, DT[wdtype])
    y, so = kda.short_conv_fwd(d["x"], d["weight"], d["bias"], d["state"], d["cu"])
    assert kda.device_error() == 0
    ry, rs = R.conv(_flat(d["x"]), _c(d["weight"]), _c(d["bias"]), _c(d["state"]), lens)
    assert torch.equal(_c(so), rs)
    if sum(lens):
        p, size = _p_size(d, lens)
        within(y.reshape(-1, D), ry, U[dt] * ry.abs() + 1.1 * 2.0 ** -21 * size + 2.0 ** -22 * (8 + p.abs()) * ry.abs())
    # without a state: zeros
    y0, s0 = kda.short_conv_fwd(d["x"], d["weight"], d["bias"], None, d["cu"])
    y1, s1 = kda.short_conv_fwd(d["x"], d["weight"], d["bias"], torch.zeros_like(d["state"]), d["cu"])
    assert torch.equal(y0, y1) and torch.equal(s0, s1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,D,W", [(1, 1, 4), (3, 33, 3), (7, 1024, 4), (2, 4104, 2), (65, 48, 4)])
def test_step_equals_the_prefill_bit_for_bit(cuda_device, N, D, W, dtype):
    dt = DT[dtype]
    d = _inputs(cuda_device, [1] * N, D, W, dt, N + D, True, False)
    y, so = kda.short_conv_fwd(d["x"], d["weight"], d["bias"], d["state"])
    out = torch.empty_like(d["state"])
    kept = d["state"].clone()
    y2 = kda.short_conv_step(d["x"][:, 0], d["weight"], d["state"], d["bias"], state_out=out)
    assert torch.equal(y[:, 0], y2) and torch.equal(so, out) and torch.equal(d["state"], kept)
    y3 = kda.short_conv_step(d["x"][:, 0], d["weight"], d["state"], d["bias"])  # in place
    assert torch.equal(y3, y2) and torch.equal(d["state"], out)


@pytest.mark.parametrize("dtype,dy32", [("bf16", True), ("bf16", False), ("f32", True)])
@pytest.mark.parametrize("lens,D,W", CASES + [((300, 300), 36, 4), ((1, 1, 1, 90, 2, 0, 33), 516, 4)])
def test_conv_backward(cuda_device, lens, D, W, dtype, dy32):
    dt = DT[dtype]
    packed = len(set(lens)) > 1
    d = _inputs(cuda_device, lens, D, W, dt, sum(lens) + 2 * D, D % 3 != 0, packed)
    dy = torch.randn(d["x"].shape, device=cuda_device).to(torch.float32 if dy32 else dt)
    dstate = torch.randn(len(lens), W - 1, D, device=cuda_device) if D % 2 == 0 else None
    out = kda.short_conv_bwd(d["x"], d["weight"], dy, d["bias"], d["state"], dstate, d["cu"])
    assert kda.device_error() == 0
    g = R.grads(lambda x, weight, bias, state: R.conv(x, weight, bias, state, lens),
                dict(x=_flat(d["x"]), weight=_c(d["weight"]), bias=_c(d["bias"]), state=_c(d["state"])),
                [_flat(dy), _c(dstate)])
    assert torch.isfinite(out["dx"].float()).all()
    # every gradient is a sum of at most max(4, tokens) products of fp32 factors good to 2^-19
    assert rel_rms(out["dx"].reshape(-1, D), g["x"]) <= U[dt] + 1e-5
    for name, ref in (("dweight", g["weight"]), ("dbias", g["bias"]), ("dinit", g["state"])):
        if ref is not None:
            assert rel_rms(out[name], ref) <= 1e-5, name
        else:
            assert out[name] is None


def test_gradient_against_differences(cuda_device):
    lens = [4, 0, 9]
    d = _inputs(cuda_device, lens, 20, 4, torch.float32, 11)
    dy = torch.randn(d["x"].shape, device=cuda_device)
    out = kda.short_conv_bwd(d["x"], d["weight"], dy, d["bias"], d["state"], None, d["cu"])
    v = {k: torch.randn(t.shape, dtype=F64) for k, t in (("x", d["x"][0]), ("weight", d["weight"]), ("bias", d["bias"]),
                                                         ("state", d["state"]))}
    h = 1e-5

    def loss(k):
        a = {n: (_flat(d[n]) if n == "x" else _c(d[n])) + k * h * v[n] for n in v}
        return float((R.conv(a["x"], a["weight"], a["bias"], a["state"], lens)[0] * _flat(dy)).sum())

    slope = (loss(1) - loss(-1)) / (2 * h)
    got = sum(float((_c(out[n]).reshape(v[m].shape) * v[m]).sum())
              for n, m in (("dx", "x"), ("dweight", "weight"), ("dbias", "bias"), ("dinit", "state")))
    assert abs(got - slope) <= 1e-4 * abs(slope) + 1e-3


def test_slices_and_odd_addresses(cuda_device):
    for dt in (torch.bfloat16, torch.float32):
        wide = torch.randn(2, 50, 700, device=cuda_device).to(dt)
        w, st = torch.randn(64, 4, device=cuda_device).to(dt), torch.randn(2, 3, 64, device=cuda_device).to(dt)
        dy = torch.randn(2, 50, 64, device=cuda_device)
        for lo in (0, 64, 65, 131):
            x = wide[..., lo:lo + 64]
            y, s = kda.short_conv_fwd(x, w, None, st)
            y2, s2 = kda.short_conv_fwd(x.contiguous(), w, None, st)
            assert torch.equal(y, y2) and torch.equal(s, s2)
            a, b = kda.short_conv_bwd(x, w, dy, None, st), kda.short_conv_bwd(x.contiguous(), w, dy, None, st)
            assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dinit"], b["dinit"])
            assert rel_rms(a["dweight"], b["dweight"].cpu()) <= 1e-6


def test_special_values_stay_in_their_window(cuda_device):
    x = torch.randn(1, 40, 32, device=cuda_device)
    w = torch.randn(32, 4, device=cuda_device)
    cu = torch.tensor([0, 22, 40], dtype=torch.int32, device=cuda_device)
    ref, _ = kda.short_conv_fwd(x, w, None, None, cu)
    x[0, 20] = float("nan")                  # seen by tokens 20, 21 of its own sequence only
    y, _ = kda.short_conv_fwd(x, w, None, None, cu)
    keep = torch.ones(40, dtype=torch.bool, device=cuda_device)
    keep[20:22] = False
    assert torch.equal(y[0, keep], ref[0, keep]) and bool(torch.isnan(y[0, ~keep]).all())
    big = torch.full((1, 8, 32), 1e30, device=cuda_device)
    y, _ = kda.short_conv_fwd(big, -w.abs(), None, torch.full((1, 3, 32), 1e30, device=cuda_device))
    assert torch.count_nonzero(y) == 0       # silu of a huge negative number is 0


@pytest.mark.parametrize("table", [[0, 30, 10, 60], [0, 20, 40, 50], [5, 20, 40, 60], [0, 70, 80, 60], [-9, 3, 5, 60]])
def test_malformed_table_is_reported(cuda_device, table):
    """The values stay where a missed check could not leave the buffers either."""
    x, w = torch.randn(1, 60, 32, device=cuda_device), torch.randn(32, 4, device=cuda_device)
    st = torch.randn(3, 3, 32, device=cuda_device)
    cu = torch.tensor(table, dtype=torch.int32, device=cuda_device)
    assert kda.device_error() == 0
    kda.short_conv_fwd(x, w, None, st, cu)
    assert kda.device_error() == 1
    kda.short_conv_bwd(x, w, x, None, st, st, cu)
    assert kda.device_error() == 1
    good = torch.tensor([0, 20, 40, 60], dtype=torch.int32, device=cuda_device)
    kda.short_conv_fwd(x, w, None, st, good)
    assert kda.device_error() == 0


def test_more_than_2_to_the_31_elements(cuda_device):
    D, T = 8192, (1 << 18) + 40
    x = torch.zeros(1, T, D, dtype=torch.bfloat16, device=cuda_device)
    tail = torch.randn(1, 37, D, device=cuda_device).to(torch.bfloat16)
    x[:, -37:] = tail
    w = torch.randn(D, 4, device=cuda_device).to(torch.bfloat16)
    y, s = kda.short_conv_fwd(x, w)
    y2, s2 = kda.short_conv_fwd(tail, w)
    assert torch.equal(y[:, -37:], y2) and torch.equal(s, s2) and torch.count_nonzero(y[:, :-37].view(-1)[::4099]) == 0
    a, b = kda.short_conv_bwd(x, w, x), kda.short_conv_bwd(tail, w, tail)
    assert torch.equal(a["dx"][:, -37:], b["dx"]) and rel_rms(a["dweight"], b["dweight"].cpu()) <= 1e-6


@pytest.mark.parametrize("D,W,dtype", [(8, 4, "bf16"), (20, 3, "f32"), (33, 4, "bf16")])
def test_long_runs(cuda_device, D, W, dtype):
    """Runs of many groups of tokens, sequences that end anywhere in them (the
    64-bit form on the device, by shifted products)."""
    dt = DT[dtype]
    g = torch.Generator().manual_seed(D)
    lens = [int(n) for n in torch.randint(0, 900, (70,), generator=g)] + [40000]
    d = _inputs(cuda_device, lens, D, W, dt, 5, True, True)
    dy = torch.randn(d["x"].shape, device=cuda_device)
    dstate = torch.randn(len(lens), W - 1, D, device=cuda_device)
    y, so = kda.short_conv_fwd(d["x"], d["weight"], d["bias"], d["state"], d["cu"])
    out = kda.short_conv_bwd(d["x"], d["weight"], dy, d["bias"], d["state"], dstate, d["cu"])
    assert kda.device_error() == 0
    x, st = d["x"][0].to(F64).requires_grad_(True), d["state"].to(F64).requires_grad_(True)
    w, b = d["weight"].to(F64).requires_grad_(True), d["bias"].to(F64).requires_grad_(True)
    ys, ss, at = [], [], 0
    for n, length in enumerate(lens):
        rows = torch.cat([st[n], x[at:at + length]])
        at += length
        ys.append(R.silu(sum(rows[j:j + length] * w[:, j] for j in range(W)) + b))
        ss.append(rows[length:])
    ry, rs = torch.cat(ys), torch.stack(ss)
    ((ry * dy[0].to(F64)).sum() + (rs * dstate.to(F64)).sum()).backward()
    assert torch.equal(so.to(F64), rs.detach())
    # |p| is at most 16 here or so: 2^-21 of the sum of sizes and 2^-22 (8 + |p|) of y stay under 2^-17 (1 + |y|)
    assert bool(((y[0].to(F64) - ry).abs() <= U[dt] * ry.abs() + 2.0 ** -17 * (1 + ry.abs())).all())
    assert rel_rms(out["dx"][0], x.grad.cpu()) <= U[dt] + 1e-5
    for name, t in (("dweight", w), ("dbias", b), ("dinit", st)):
        assert rel_rms(out[name], t.grad.cpu()) <= 2e-5, name


def test_many_short_sequences(cuda_device):
    g = torch.Generator().manual_seed(3)
    lens = [int(n) for n in torch.randint(0, 6, (700,), generator=g)] + [0, 0, 90, 0]
    d = _inputs(cuda_device, lens, 24, 4, torch.float32, 17)
    dy, dstate = torch.randn(d["x"].shape, device=cuda_device), torch.randn(len(lens), 3, 24, device=cuda_device)
    y, so = kda.short_conv_fwd(d["x"], d["weight"], d["bias"], d["state"], d["cu"])
    out = kda.short_conv_bwd(d["x"], d["weight"], dy, d["bias"], d["state"], dstate, d["cu"])
    assert kda.device_error() == 0
    ry, rs = R.conv(_flat(d["x"]), _c(d["weight"]), _c(d["bias"]), _c(d["state"]), lens)
    assert torch.equal(_c(so), rs)
    p, size = _p_size(d, lens)
    within(y[0], ry, U[torch.float32] * ry.abs() + 1.1 * 2.0 ** -21 * size + 2.0 ** -22 * (8 + p.abs()) * ry.abs())
    gr = R.grads(lambda x, weight, bias, state: R.conv(x, weight, bias, state, lens),
                 dict(x=_flat(d["x"]), weight=_c(d["weight"]), bias=_c(d["bias"]), state=_c(d["state"])),
                 [_flat(dy), _c(dstate)])
    for name, key in (("dx", "x"), ("dweight", "weight"), ("dbias", "bias"), ("dinit", "state")):
        assert rel_rms(out[name].reshape(gr[key].shape), gr[key]) <= 1e-5, name
