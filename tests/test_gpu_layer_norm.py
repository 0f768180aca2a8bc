"""GPU: root-mean-square norm (plain, e4m3, backward) against the 64-bit form.

Bounds: r = rsqrt(mean s^2 + eps) in fp32 is good to 2^-17 relative (a sum of
squares whose longest chain is 128 additions, half of that in the root, and the
approximate rsqrt), s and the products add units of 2^-24; the stored value adds
half a step."""
import pytest
import torch

import kimi_delta_attention_31_b200 as kda
import layer_ref as R
from layer_ref import F64, U, rel_rms, within

pytestmark = pytest.mark.gpu

K = 2.0 ** -16
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _inputs(dev, rows, D, dtype, seed, residual, wdtype=None):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=dev)
    x = r(rows, D).to(dtype)
    w = (1 + 0.1 * r(D)).to(wdtype or dtype)
    res = (2 * r(rows, D)).to(dtype) if residual else None
    return x, w, res


def _ref(x, w, res, eps=1e-6):
    c = lambda t: None if t is None else t.detach().cpu().to(F64)
    return R.norm(c(x), c(w), c(res), eps)


SHAPES = [(1, 1), (3, 17), (5, 64), (7, 128), (9, 250), (2, 256), (3, 512), (4, 1000), (2, 1153), (3, 2048), (2, 4096),
          (2, 7168), (1, 8191), (3, 16384), (1, 16383), (300, 96)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", SHAPES)
def test_norm(cuda_device, rows, D, dtype, residual):
    dt = DT[dtype]
    x, w, res = _inputs(cuda_device, rows, D, dt, rows + D, residual, torch.float32 if D % 3 else dt)
    y, s = kda.rms_norm_fwd(x, w, res)
    ry, rs = _ref(x, w, res)
    within(y, ry, (U[dt] + K) * ry.abs(), "y")
    if residual:
        within(s, rs, (U[dt] * (1 + 2.0 ** -20) + 2.0 ** -24) * rs.abs(), "s")
    else:
        assert s is None
    assert kda.device_error() == 0


def _check_quant(q, scale, ry, group):
    rows, D = ry.shape
    yg = ry.view(rows, -1, group or D)
    rscale = yg.abs().amax(-1).clamp_min(1e-10) / 448
    within(scale, rscale, 2 * K * rscale, "scale")
    # half a step of e4m3: 2^-4 relative, 2^-10 below the smallest normal value (2^-6)
    v = yg / rscale[..., None]
    bound = torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10)) + 4 * K * v.abs()
    within(q.float().view(yg.shape), v, bound, "q")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D,group", [(5, 128, 128), (1, 32, 32), (33, 96, 32), (3, 1024, 64), (2, 4096, 128),
                                          (4, 192, 64), (3, 17, 0), (2, 1153, 0), (7, 128, 0), (2, 7168, 128),
                                          (1, 16384, 32), (2, 16384, 0)])
def test_norm_quant(cuda_device, rows, D, group, dtype):
    x, w, res = _inputs(cuda_device, rows, D, DT[dtype], rows * D, True)
    q, scale, s = kda.rms_norm_quant_fwd(x, w, res, group=group)
    assert q.dtype == torch.float8_e4m3fn and tuple(scale.shape) == (rows, D // group if group else 1)
    ry, rs = _ref(x, w, res)
    _check_quant(q, scale, ry, group)
    within(s, rs, (U[DT[dtype]] * (1 + 2.0 ** -20) + 2.0 ** -24) * rs.abs(), "s")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", SHAPES + [(2000, 128), (700, 1000), (1500, 4096)])
def test_norm_backward(cuda_device, rows, D, dtype):
    dt = DT[dtype]
    s, w, dy = _inputs(cuda_device, rows, D, dt, 5 * rows + D, True)
    ds = torch.randn(rows, D, device=cuda_device).to(dt) if rows % 2 else None
    out = kda.rms_norm_bwd(dy, s, w, ds)
    c = lambda t: t.cpu().to(F64)
    g = R.grads(lambda x, weight: (R.norm(x, weight)[0],), dict(x=c(s), weight=c(w)), [c(dy)])
    want = g["x"] + (c(ds) if ds is not None else 0)
    # dx is a difference of terms of this size, each good to 3K
    r = 1 / (c(s).square().mean(-1, keepdim=True) + 1e-6).sqrt()
    size = (r * c(w) * c(dy)).abs() + c(s).abs() * r ** 3 * (c(w) * c(dy) * c(s)).abs().mean(-1, keepdim=True)
    within(out["dx"], want, U[dt] * want.abs() + 4 * K * size, "dx")
    dsize = (c(dy) * c(s) * r).abs().sum(0)
    within(out["dweight"], g["weight"], 2 * K * dsize, "dweight")


def test_gradient_against_differences(cuda_device):
    """<gradient, v> is the slope of the 64-bit loss along v."""
    s, w, dy = _inputs(cuda_device, 6, 200, torch.float32, 9, True)
    out = kda.rms_norm_bwd(dy, s, w)
    c = lambda t: t.cpu().to(F64)
    vs, vw, h = torch.randn(6, 200, dtype=F64), torch.randn(200, dtype=F64), 1e-5
    loss = lambda k: float((R.norm(c(s) + k * h * vs, c(w) + k * h * vw)[0] * c(dy)).sum())
    slope = (loss(1) - loss(-1)) / (2 * h)
    got = float((c(out["dx"]) * vs).sum() + (c(out["dweight"]) * vw).sum())
    assert abs(got - slope) <= 1e-4 * abs(slope) + 1e-3


def test_slices_in_place_and_odd_addresses(cuda_device):
    """A slice of a joint projection, a base address off the vector, outputs in
    place and heads: the same numbers as the packed call."""
    g = torch.Generator(device=cuda_device).manual_seed(3)
    for dt in (torch.bfloat16, torch.float32):
        wide = torch.randn(6, 3, 512, generator=g, device=cuda_device).to(dt)
        w = torch.randn(128, generator=g, device=cuda_device).to(dt)
        for lo in (0, 128, 129, 255):
            x = wide[..., lo:lo + 128]
            y, _ = kda.rms_norm_fwd(x, w)
            y2, _ = kda.rms_norm_fwd(x.contiguous(), w)
            assert rel_rms(y.float(), y2.float().cpu()) <= 2 * U[dt]
        x, res = wide[..., :128].contiguous(), wide[..., 128:256].contiguous()
        y, s = kda.rms_norm_fwd(x, w, res)
        x2, r2 = x.clone(), res.clone()
        kda.rms_norm_fwd(x2, w, r2, y=x2, s=r2)
        assert torch.equal(x2, y) and torch.equal(r2, s)
        dy = torch.randn(6, 3, 128, generator=g, device=cuda_device).to(dt)
        ref = kda.rms_norm_bwd(dy, s, w, ds=y)
        d2 = dy.clone()
        out = kda.rms_norm_bwd(d2, s, w, ds=y, dx=d2)
        assert torch.equal(out["dx"], ref["dx"]) and out["dx"] is d2
        assert torch.equal(out["dweight"], ref["dweight"])
        with pytest.raises(kda.KDAError):  # group scales need aligned rows
            kda.rms_norm_quant_fwd(wide[..., 1:129], w, group=32)


def test_special_values_stay_in_their_rows(cuda_device):
    x = torch.randn(6, 256, device=cuda_device)
    x[1] = 0
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    w = torch.ones(256, device=cuda_device)
    y, _ = kda.rms_norm_fwd(x, w)
    ry, _ = _ref(x, w, None)
    for r in (0, 1, 4, 5):
        within(y[r], ry[r], (U[torch.float32] + K) * ry[r].abs(), str(r))
    assert torch.count_nonzero(y[1]) == 0 and bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3, 9]))
    for group in (0, 32):
        q, scale, _ = kda.rms_norm_quant_fwd(x, w, group=group)
        assert bool(torch.isnan(scale[2]).all()) and bool(torch.isnan(q[2].float()).all())
        assert torch.count_nonzero(q[1].float()) == 0 and bool((scale[1] == 1e-10 / 448).all())
        ok = [0, 4, 5]
        _check_quant(q[ok], scale[ok], ry[ok], group)


def test_no_rows_and_a_second_call(cuda_device):
    w = torch.ones(64, device=cuda_device)
    x = torch.zeros(0, 64, device=cuda_device)
    assert kda.rms_norm_fwd(x, w)[0].shape == (0, 64)
    assert kda.rms_norm_quant_fwd(x, w)[0].shape == (0, 64)
    out = kda.rms_norm_bwd(x, x, w)
    assert torch.count_nonzero(out["dweight"]) == 0
    s, wt, dy = _inputs(cuda_device, 3000, 256, torch.bfloat16, 1, True)
    a, b = kda.rms_norm_bwd(dy, s, wt), kda.rms_norm_bwd(dy, s, wt)
    assert torch.equal(a["dweight"], b["dweight"]) and torch.equal(a["dx"], b["dx"])


def test_more_than_2_to_the_31_elements(cuda_device):
    rows, D = (1 << 31) // 4096 + 3, 4096
    x = torch.empty(rows, D, dtype=torch.bfloat16, device=cuda_device)
    g = torch.Generator(device=cuda_device).manual_seed(4)
    tail = torch.randn(5, D, generator=g, device=cuda_device).to(torch.bfloat16)
    x.fill_(1.0)
    x[-5:] = tail
    w = torch.ones(D, dtype=torch.bfloat16, device=cuda_device)
    y, _ = kda.rms_norm_fwd(x, w)
    y2, _ = kda.rms_norm_fwd(tail, w)
    assert torch.equal(y[-5:], y2) and bool((y[:-5].view(-1)[::4099] == 1.0).all())
    q, scale, _ = kda.rms_norm_quant_fwd(x, w, group=128)
    q2, scale2, _ = kda.rms_norm_quant_fwd(tail, w, group=128)
    assert torch.equal(q[-5:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(scale[-5:], scale2)


@pytest.mark.parametrize("rows,D,dtype", [(300001, 72, "bf16"), (299999, 50, "bf16"), (160003, 128, "f32"),
                                          (400000, 17, "f32"), (40001, 500, "bf16")])
def test_many_rows(cuda_device, rows, D, dtype):
    """Rows that a thread takes in turns, and the backward's rows over every CTA
    (the 64-bit form on the device: only its own arithmetic is used)."""
    dt = DT[dtype]
    x, w, res = _inputs(cuda_device, rows, D, dt, D, True)
    y, s = kda.rms_norm_fwd(x, w, res)
    ry, rs = R.norm(x.to(F64), w.to(F64), res.to(F64))
    assert bool(((y.to(F64) - ry).abs() <= (U[dt] + K) * ry.abs()).all())
    assert bool(((s.to(F64) - rs).abs() <= (U[dt] * (1 + 2.0 ** -20) + 2.0 ** -24) * rs.abs()).all())
    q, scale, _ = kda.rms_norm_quant_fwd(x, w, res)
    rscale = ry.abs().amax(-1, keepdim=True) / 448
    assert bool(((scale.to(F64) - rscale).abs() <= 2 * K * rscale).all())
    v = ry / rscale
    bound = torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10)) + 4 * K * v.abs()
    assert bool(((q.to(F64) - v).abs() <= bound).all())
    if D % 32 == 0:
        q, scale, _ = kda.rms_norm_quant_fwd(x, w, res, group=32)
        rg = ry.view(rows, -1, 32)
        rscale = rg.abs().amax(-1) / 448
        assert bool(((scale.to(F64) - rscale).abs() <= 2 * K * rscale).all())
    out = kda.rms_norm_bwd(y, s, w, x)
    sd, g = s.to(F64), y.to(F64)
    r = 1 / (sd.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    gw = g * w.to(F64)
    want = r * gw - sd * r ** 3 * (gw * sd).mean(-1, keepdim=True) + x.to(F64)
    size = (r * gw).abs() + sd.abs() * r ** 3 * (gw * sd).abs().mean(-1, keepdim=True)
    # dx adds three terms in fp32: its two additions round partial sums that are at most |ds| + size, by half a step
    # (2^-24) each, whatever is left of them in dx
    adds = 2 * 2.0 ** -24 * (x.to(F64).abs() + size)
    assert bool(((out["dx"].to(F64) - want).abs() <= U[dt] * want.abs() + 4 * K * size + adds).all())
    terms = g * sd * r
    # a column's sum in fp32: chains of up to rows / 148 additions, each off by 2^-24 of what it holds
    assert bool(((out["dweight"].to(F64) - terms.sum(0)).abs() <= (2 * K + rows / 148 * 2.0 ** -24) * terms.abs().sum(0)).all())


@pytest.mark.parametrize("rows,D,group", [(5000, 128, 128), (4096, 128, 32), (900, 1153, 0), (300, 4096, 128), (700, 2048, 0),
                                          (3000, 17, 0), (64, 16384, 64)])
def test_quantised_values_are_the_quotients_rounded_once(cuda_device, rows, D, group):
    """q is e4m3(y / scale) to the bit: y as the fp32 norm gives it (the same rows in the same threads), scale as
    returned, the quotient rounded to fp32 and then to e4m3.  Without the rounding of a division, quotients next to a
    border between two e4m3 values land on the wrong side of it."""
    x, w, res = _inputs(cuda_device, rows, D, torch.float32, rows + D, True)
    x, res, w = x.to(torch.bfloat16).float(), res.to(torch.bfloat16).float(), w.to(torch.bfloat16).float()
    y, _ = kda.rms_norm_fwd(x, w, res)
    q, scale, _ = kda.rms_norm_quant_fwd(x, w, res, group=group)
    yg = y.view(rows, -1, group or D)
    want = (yg / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(rows, D)
    assert int((q.view(torch.uint8) != want.view(torch.uint8)).sum()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,group", [(128, 128), (128, 0), (96, 32), (33, 0), (4096, 64)])
def test_quotients_half_way_go_to_the_even_value(cuda_device, D, group, dtype):
    """Rows of +-4 and weights that are whole numbers of at most 8 bits over 64: y = s / 4 * w = +-w, the largest one
    7 = 448 / 64, the scale 1 / 64 exactly, y / scale whole numbers, many of them half way between two e4m3 values."""
    dt = DT[dtype]
    g = torch.Generator(device=cuda_device).manual_seed(D)
    k = torch.randint(0, 225, (D,), generator=g, device=cuda_device)
    k[:: group or D] = 224  # every group's largest
    w = (k.float() / 32).to(dt)
    x = torch.where(torch.rand(50, D, generator=g, device=cuda_device) < 0.5, -4.0, 4.0).to(dt)
    q, scale, _ = kda.rms_norm_quant_fwd(x, w, eps=0.0, group=group)
    assert bool((scale == 1 / 64).all())
    v = (2 * k.float() * x.float().sign())
    assert torch.equal(q.view(torch.uint8), v.to(torch.float8_e4m3fn).view(torch.uint8))


def test_infinite_scales(cuda_device):
    """A weight so large that y is infinite: the group's scale is infinite, its finite values 0, the infinite one NaN."""
    x = torch.ones(3, 128, device=cuda_device)
    w = torch.ones(128, device=cuda_device)
    x[1, 5], w[5] = 8.0, 3e38
    for group in (0, 32):
        q, scale, _ = kda.rms_norm_quant_fwd(x, w, eps=0.0, group=group)
        y, _ = kda.rms_norm_fwd(x, w, eps=0.0)
        assert bool(torch.isinf(y[1, 5])) and bool(torch.isinf(scale[1, 0])) and bool(torch.isfinite(scale[[0, 2]]).all())
        assert bool(torch.isnan(q[1, 5].float())) and torch.count_nonzero(q[1, :5].float()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale,eps", [(1e15, 1e-6), (1e17, 1e-6), (1e-13, 0.0), (1e-17, 0.0)])
@pytest.mark.parametrize("rows,D", [(5, 128), (3, 1001), (4, 4096), (2, 16384)])
def test_backward_of_rows_far_from_one(cuda_device, rows, D, scale, eps, dtype):
    """dx is 1 / scale of the unit rows' while mean(s^2) is inside fp32's range (1e-34 to 1e34 here)."""
    dt = DT[dtype]
    s, w, dy = _inputs(cuda_device, rows, D, dt, 7 * rows + D, True)
    s = (s.float() * scale).to(dt)
    out = kda.rms_norm_bwd(dy, s, w, eps=eps)
    c = lambda t: t.cpu().to(F64)
    g = R.grads(lambda x, weight: (R.norm(x, weight, eps=eps)[0],), dict(x=c(s), weight=c(w)), [c(dy)])
    r = 1 / (c(s).square().mean(-1, keepdim=True) + eps).sqrt()
    size = (r * c(w) * c(dy)).abs() + c(s).abs() * r ** 3 * (c(w) * c(dy) * c(s)).abs().mean(-1, keepdim=True)
    # mean(s^2) of 1e-34 is 1e4 times fp32's smallest normal value: the bounds of unit rows hold
    within(out["dx"], g["x"], U[dt] * g["x"].abs() + 4 * K * size, "dx")
    within(out["dweight"], g["weight"], 2 * K * (c(dy) * c(s) * r).abs().sum(0), "dweight")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [33, 127, 129, 257, 385, 511, 513, 641, 769, 1023, 1025, 1281, 1535, 1537, 2047, 2049, 4097, 8193])
def test_rows_at_odd_places_of_every_length(cuda_device, D, dtype):
    """Rows read element by element: just below and above the lengths at which a thread takes another number of them."""
    dt = DT[dtype]
    x, w, res = _inputs(cuda_device, 5, D, dt, D, True)
    y, s = kda.rms_norm_fwd(x, w, res)
    q, scale, s2 = kda.rms_norm_quant_fwd(x, w, res)
    ry, rs = _ref(x, w, res)
    within(y, ry, (U[dt] + K) * ry.abs(), "y")
    within(s, rs, (U[dt] * (1 + 2.0 ** -20) + 2.0 ** -24) * rs.abs(), "s")
    assert torch.equal(s, s2)
    _check_quant(q, scale, ry, 0)
