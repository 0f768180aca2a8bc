"""GPU: selective scan (prefill, step, backward) against the 64-bit form.
Forward bounds are carried along the recurrence (layer_ref.scan_error).  A
gradient in fp32 is a sum over up to 300 tokens of products whose factors
(states, carried gradients) are each good to 300 x 2^-21 at worst: 1e-4 of its
root mean square, plus half a step where it is stored in bf16."""
import pytest
import torch

import kimi_delta_attention_31_b200 as kda
import layer_ref as R
from layer_ref import F64, U, rel_rms, within

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "S0")


def _inputs(dev, lens, d, S, groups, dtype, seed, packed, gate=True, skip=True, bias=True, s0=True):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=dev)
    N, T = len(lens), sum(lens)
    lead = (1, T) if packed else (N, lens[0])
    return dict(x=r(*lead, d).to(dtype), dt=(0.5 * r(*lead, d) - (0 if bias else 3)).to(dtype),
                A=-(torch.arange(1, S + 1, device=dev) * torch.exp(0.1 * r(d, S))), B=r(*lead, groups, S).to(dtype),
                C=r(*lead, groups, S).to(dtype), D=r(d) if skip else None, z=r(*lead, d).to(dtype) if gate else None,
                dt_bias=r(d) - 3 if bias else None, S0=r(N, d, S) if s0 else None,
                cu=torch.tensor(R.bounds(lens), dtype=torch.int32, device=dev) if packed else None)


def _c(t):
    return None if t is None else t.detach().cpu().to(F64)


def _ref_args(v, lens):
    d, S = v["A"].shape
    row = lambda t: None if t is None else _c(t).reshape(sum(lens), *t.shape[2:])
    S0 = _c(v["S0"]) if v["S0"] is not None else torch.zeros(len(lens), d, S, dtype=F64)
    return dict(x=row(v["x"]), dt=row(v["dt"]), A=_c(v["A"]), B=row(v["B"]), C=row(v["C"]), D=_c(v["D"]), z=row(v["z"]),
                dt_bias=_c(v["dt_bias"]), state=S0)


def _fwd(v, **kw):
    return kda.selective_scan_fwd(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"], v["dt_bias"], v["S0"],
                                  v["cu"], **kw)


def _bwd(v, dy, dS, **kw):
    return kda.selective_scan_bwd(v["x"], v["dt"], v["A"], v["B"], v["C"], dy, v["D"], v["z"], v["dt_bias"], v["S0"],
                                  dS, v["cu"], **kw)


def _check_fwd(v, lens, y, So):
    dt = v["x"].dtype
    args = _ref_args(v, lens)
    ry, rS = R.scan(*args.values(), lens)
    ey, eS = R.scan_error(*args.values(), lens, dt)
    within(y.reshape(ry.shape), ry, U[dt] * ry.abs() + ey, "y")
    within(So, rS, eS + 2.0 ** -23 * rS.abs(), "S_out")


CASES = [((1,), 1, 16, 1), ((2, 2, 2), 33, 16, 1), ((7,), 130, 8, 1), ((9, 9), 64, 32, 2), ((40,), 36, 64, 2),
         ((130,), 10, 16, 2), ((129, 129), 256, 16, 1), ((300,), 34, 8, 2), ((0, 1, 2, 0, 140, 63, 64, 1, 0), 48, 16, 1),
         ((1, 1, 1, 90, 33, 0, 150), 20, 64, 2), ((64, 128, 64), 70, 32, 1), ((65, 0, 0, 127), 260, 8, 2), ((0, 0), 8, 16, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,d,S,groups", CASES)
def test_scan(cuda_device, lens, d, S, groups, dtype):
    packed = len(set(lens)) > 1
    v = _inputs(cuda_device, lens, d, S, groups, DT[dtype], sum(lens) + d, packed)
    y, So = _fwd(v)
    assert kda.device_error() == 0
    _check_fwd(v, lens, y, So)


@pytest.mark.parametrize("gate,skip,bias,s0", [(False, True, True, True), (True, False, True, False),
                                              (True, True, False, True), (False, False, False, False)])
def test_scan_optional_inputs(cuda_device, gate, skip, bias, s0):
    for lens in ((50, 50), (80, 0, 200, 3)):
        v = _inputs(cuda_device, lens, 40, 16, 1, torch.float32, 5, lens[0] != lens[1], gate, skip, bias, s0)
        y, So = _fwd(v)
        _check_fwd(v, lens, y, So)
        y2, none = _fwd(v, output_final_state=False)
        assert none is None and torch.equal(y, y2)
        dy, dS = torch.randn_like(v["x"]), torch.randn(len(lens), 40, 16, device=cuda_device)
        out = _bwd(v, dy, dS)
        _check_bwd(v, lens, out, dy, dS)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,d,S,groups", [(1, 1, 16, 1), (3, 33, 8, 1), (5, 130, 64, 2), (17, 256, 32, 2), (64, 100, 16, 1)])
def test_step(cuda_device, N, d, S, groups, dtype):
    dt = DT[dtype]
    v = _inputs(cuda_device, [1] * N, d, S, groups, dt, N + d, False)
    row = {k: (t[:, 0] if k in ("x", "dt", "z", "B", "C") else t) for k, t in v.items()}
    out, kept = torch.empty_like(v["S0"]), v["S0"].clone()
    y = kda.selective_scan_step(row["x"], row["dt"], v["A"], row["B"], row["C"], v["S0"], v["D"], row["z"], v["dt_bias"],
                                S_out=out)
    assert torch.equal(kept, v["S0"])
    _check_fwd(v, [1] * N, y, out)
    y2 = kda.selective_scan_step(row["x"], row["dt"], v["A"], row["B"], row["C"], v["S0"], v["D"], row["z"],
                                 v["dt_bias"])
    assert torch.equal(y, y2) and torch.equal(v["S0"], out)  # in place


def _check_bwd(v, lens, out, dy, dS):
    dt = v["x"].dtype
    args = _ref_args(v, lens)
    g = R.grads(lambda **a: R.scan(*a.values(), lens), args, [_c(dy).reshape(args["x"].shape), _c(dS)])
    for name, key, bf in (("dx", "x", True), ("ddt", "dt", True), ("dz", "z", True), ("dA", "A", False),
                          ("dB", "B", False), ("dC", "C", False), ("dD", "D", False), ("ddt_bias", "dt_bias", False),
                          ("dS0", "state", False)):
        ref, got = g[key], out[name]
        if ref is None:
            assert got is None, name
            continue
        assert torch.isfinite(got.float()).all(), name
        err = rel_rms(got.reshape(ref.shape), ref)
        assert err <= 1e-4 + (U[dt] if bf else 0), f"{name}: {err:.3e}"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,d,S,groups", CASES)
def test_scan_backward(cuda_device, lens, d, S, groups, dtype):
    packed = len(set(lens)) > 1
    v = _inputs(cuda_device, lens, d, S, groups, DT[dtype], sum(lens) + 3 * d, packed, gate=d % 3 != 0)
    dy = torch.randn_like(v["x"])
    dS = torch.randn(len(lens), d, S, device=cuda_device) if d % 4 else None
    out = _bwd(v, dy, dS)
    assert kda.device_error() == 0
    _check_bwd(v, lens, out, dy, dS)
    again = _bwd(v, dy, dS)
    for name, t in out.items():
        assert t is None or torch.equal(t, again[name]), name


def test_gradient_against_differences(cuda_device):
    lens = [70, 0, 13]
    v = _inputs(cuda_device, lens, 6, 8, 1, torch.float32, 21, True)
    dy, dS = torch.randn_like(v["x"]), torch.randn(3, 6, 8, device=cuda_device)
    out = _bwd(v, dy, dS)
    args = _ref_args(v, lens)
    dirs = {k: torch.randn_like(t) for k, t in args.items()}
    h = 1e-6

    def loss(k):
        y, S = R.scan(*[t + k * h * dirs[n] for n, t in args.items()], lens)
        return float((y * _c(dy)[0]).sum() + (S * _c(dS)).sum())

    slope = (loss(1) - loss(-1)) / (2 * h)
    key = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", D="dD", z="dz", dt_bias="ddt_bias", state="dS0")
    got = sum(float((_c(out[key[n]]).reshape(t.shape) * t).sum()) for n, t in dirs.items())
    assert abs(got - slope) <= 2e-4 * abs(slope) + 1e-2


@pytest.mark.parametrize("value", [-60.0, 30.0])
def test_extreme_time_steps(cuda_device, value):
    """Steps of 0 (the state stays) and huge ones (it is forgotten)."""
    lens = (20, 20)
    v = _inputs(cuda_device, lens, 24, 16, 1, torch.float32, 8, False)
    v["dt_bias"].fill_(0.0)
    v["dt"][:, 5:11] = value
    y, So = _fwd(v)
    _check_fwd(v, lens, y, So)
    dy = torch.randn_like(v["x"])
    _check_bwd(v, lens, _bwd(v, dy, None), dy, torch.zeros_like(v["S0"]))


def test_nan_stays_in_its_sequence_and_channel(cuda_device):
    lens = (90, 150, 60)
    v = _inputs(cuda_device, lens, 40, 16, 1, torch.float32, 9, True)
    ref, rS = _fwd(v)
    v["x"][0, 120, 7] = float("nan")
    y, So = _fwd(v)
    keep = torch.ones(300, 40, dtype=torch.bool, device=cuda_device)
    keep[120:240, 7] = False
    assert torch.equal(y[0][keep], ref[0][keep]) and bool(torch.isnan(y[0][~keep]).all())
    keepS = torch.ones(3, 40, dtype=torch.bool, device=cuda_device)
    keepS[1, 7] = False
    assert torch.equal(So[keepS], rS[keepS])


def test_slices_of_a_joint_projection(cuda_device):
    for dt in (torch.bfloat16, torch.float32):
        v = _inputs(cuda_device, (140, 140), 36, 16, 2, dt, 12, False)
        ref, rS = _fwd(v)
        dy = torch.randn_like(v["x"])
        gref = _bwd(v, dy, None)
        wide = torch.randn(2, 140, 1 + 3 * 36 + 2 * 32 + 2, device=cuda_device).to(dt)
        at, s = 1, dict(v)
        for n in ("x", "dt", "z"):
            s[n] = wide[..., at:at + 36].copy_(v[n])
            at += 36
        for n in ("B", "C"):
            s[n] = wide[..., at:at + 32].copy_(v[n].flatten(2)).unflatten(-1, (2, 16))
            at += 32
        y, So = _fwd(s)
        assert torch.equal(y, ref) and torch.equal(So, rS)
        g = _bwd(s, dy, None)
        for n, t in gref.items():
            assert torch.equal(t, g[n]), n


@pytest.mark.parametrize("table", [[0, 150, 60, 300], [0, 100, 200, 250], [17, 100, 200, 300], [0, 350, 400, 300],
                                   [-40, 100, 200, 300]])
def test_malformed_table_is_reported(cuda_device, table):
    """Token indices come from the grid and sequence indices from a search over
    the table's own entries, so no table leads out of the buffers."""
    v = _inputs(cuda_device, (100, 100, 100), 20, 16, 1, torch.float32, 13, True)
    good, v["cu"] = v["cu"], torch.tensor(table, dtype=torch.int32, device=cuda_device)
    assert kda.device_error() == 0
    _fwd(v)
    assert kda.device_error() == 1
    _bwd(v, v["x"], v["S0"])
    assert kda.device_error() == 1
    v["cu"] = good
    y, So = _fwd(v)
    assert kda.device_error() == 0
    _check_fwd(v, (100, 100, 100), y, So)


def test_more_than_2_to_the_31_elements(cuda_device):
    """A long packed batch whose last sequence starts past 2^31 elements."""
    d, tail = 8192, 70
    T = (1 << 18) + 30 + tail
    v = _inputs(cuda_device, (tail,), d, 8, 1, torch.bfloat16, 14, False, gate=False)
    big = dict(v)
    for n in ("x", "dt", "B", "C"):
        big[n] = torch.zeros(1, T, *v[n].shape[2:], dtype=torch.bfloat16, device=cuda_device)
        big[n][:, -tail:] = v[n]
    big["S0"] = torch.cat([torch.zeros_like(v["S0"]), v["S0"]])
    big["cu"] = torch.tensor([0, T - tail, T], dtype=torch.int32, device=cuda_device)
    y, So = _fwd(big)
    ref, rS = _fwd(v)
    assert kda.device_error() == 0
    assert torch.count_nonzero(y[:, :T - tail].view(-1)[::4099]) == 0
    # the chunks fall elsewhere: equal up to fp32 rounding, which bf16 outputs mostly hide
    assert rel_rms(y[:, -tail:].float(), ref.float().cpu()) <= 2.0 ** -9
    assert rel_rms(So[1], rS[0].cpu()) <= 1e-5


def test_tokens_behind_the_last_sequence_are_refused(cuda_device):
    v = _inputs(cuda_device, (30, 30), 16, 16, 1, torch.float32, 15, True)
    v["cu"] = torch.tensor([0, 20, 40], dtype=torch.int32, device=cuda_device)  # 60 tokens given
    _fwd(v)
    assert kda.device_error() == 1


@pytest.mark.parametrize("lens,dtype", [((9000,), "f32"), ((2500, 2500, 2500), "bf16"), ((3000, 0, 5000, 700, 1), "f32")])
def test_long_sequences(cuda_device, lens, dtype):
    """Chunks of many tiles.  Decays of up to a few thousand tokens' memory
    (steps of 0.001 to 0.1, A from -1): errors add up over the memory, so the
    forward's bound is the recurrence's own; the gradients, which sum as many
    terms, 3e-4 of their root mean square."""
    packed = len(set(lens)) > 1
    v = _inputs(cuda_device, lens, 16, 8, 2, DT[dtype], 31, packed)
    v["dt_bias"] -= 1.5
    y, So = _fwd(v)
    assert kda.device_error() == 0
    _check_fwd(v, lens, y, So)
    dy, dS = torch.randn_like(v["x"]), torch.randn(len(lens), 16, 8, device=cuda_device)
    out = _bwd(v, dy, dS)
    args = _ref_args(v, lens)
    g = R.grads(lambda **a: R.scan(*a.values(), lens), args, [_c(dy).reshape(args["x"].shape), _c(dS)])
    for name, key, bf in (("dx", "x", True), ("ddt", "dt", True), ("dz", "z", True), ("dA", "A", False),
                          ("dB", "B", False), ("dC", "C", False), ("dD", "D", False), ("ddt_bias", "dt_bias", False),
                          ("dS0", "state", False)):
        err = rel_rms(out[name].reshape(g[key].shape), g[key])
        assert err <= 3e-4 + (U[DT[dtype]] if bf else 0), f"{name}: {err:.3e}"


def test_nan_in_the_backward_stays_with_its_sequence(cuda_device):
    """A NaN input of one sequence and channel reaches that sequence's dB, dC and
    that channel's sums, and nothing of the other sequences."""
    lens = (70, 90, 60)
    v = _inputs(cuda_device, lens, 37, 16, 1, torch.float32, 33, True)
    dy = torch.randn_like(v["x"])
    ref = _bwd(v, dy, None)
    v["x"][0, 100, 36] = float("nan")
    out = _bwd(v, dy, None)
    other = torch.ones(220, dtype=torch.bool, device=cuda_device)
    other[70:160] = False
    for name in ("dx", "ddt", "dz", "dB", "dC"):
        assert torch.equal(out[name][0][other], ref[name][0][other]), name
    assert torch.equal(out["dA"][:36], ref["dA"][:36]) and torch.equal(out["dD"][:36], ref["dD"][:36])
    assert torch.equal(out["dS0"][[0, 2]], ref["dS0"][[0, 2]]) and torch.equal(out["dx"][..., :36], ref["dx"][..., :36])


def test_many_short_sequences_and_more_than_a_grid_dimension_of_steps(cuda_device):
    g = torch.Generator().manual_seed(3)
    lens = [int(n) for n in torch.randint(0, 6, (500,), generator=g)] + [0, 0, 40, 0]
    v = _inputs(cuda_device, lens, 12, 8, 1, torch.float32, 41, True)
    y, So = _fwd(v)
    assert kda.device_error() == 0
    _check_fwd(v, lens, y, So)
    dy, dS = torch.randn_like(v["x"]), torch.randn(len(lens), 12, 8, device=cuda_device)
    _check_bwd(v, lens, _bwd(v, dy, dS), dy, dS)
    N = 65536 + 5  # the step's sequences lie along a grid dimension of 65535
    w = _inputs(cuda_device, [1] * N, 2, 8, 1, torch.float32, 42, False)
    row = {k: (t[:, 0] if k in ("x", "dt", "z", "B", "C") else t) for k, t in w.items()}
    keep = w["S0"].clone()
    y = kda.selective_scan_step(row["x"], row["dt"], w["A"], row["B"], row["C"], w["S0"], w["D"], row["z"], w["dt_bias"])
    at = [0, 1, 65534, 65535, 65536, N - 1]
    sub = {k: (t[at] if k in ("x", "dt", "z", "B", "C") else t) for k, t in w.items()}
    sub["S0"] = keep[at]
    _check_fwd(sub, [1] * len(at), y[at], w["S0"][at])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["dy", "z", "C", "B", "dt", "x", "dS", "S0"])
@pytest.mark.parametrize("lens,d,S,groups", [((200, 70, 90, 150), 37, 16, 1), ((128, 128, 128), 33, 16, 1),
                                             ((300, 300), 36, 64, 2), ((64, 0, 1, 64, 191, 3), 20, 8, 2)])
def test_non_finite_values_stay_with_their_sequence(cuda_device, lens, d, S, groups, name, value):
    """A NaN or infinity that enters one sequence, forward or backward: every output of the others is what it was, to
    the bit.  Starts inside a tile of tokens and on its border, in the middle of eight tokens and on theirs, sequences of
    several tiles before it, packed and in rows."""
    packed = len(set(lens)) > 1
    v = _inputs(cuda_device, lens, d, S, groups, torch.float32, 51, packed)
    dy, dS = torch.randn_like(v["x"]), torch.randn(len(lens), d, S, device=cuda_device)
    ry, rS = _fwd(v)
    ref = _bwd(v, dy, dS)
    at, total = R.bounds(lens), sum(lens)
    rows = lambda t: t.reshape(total, *t.shape[2:])
    for n in range(len(lens)):
        for back in sorted({0, lens[n] // 2, max(lens[n] - 1, 0)}):
            if name not in ("dS", "S0") and back >= lens[n]:
                continue
            w, gy, gS = {k: None if t is None else t.clone() for k, t in v.items()}, dy.clone(), dS.clone()
            if name in ("dS", "S0"):
                (gS if name == "dS" else w["S0"])[n, d // 2, S // 2] = value
            else:
                t = rows(gy if name == "dy" else w[name])[at[n] + back]
                t.view(-1)[t.numel() // 2] = value
            y, So = _fwd(w)
            out = _bwd(w, gy, gS)
            others = torch.ones(total, dtype=torch.bool, device=cuda_device)
            others[at[n]:at[n + 1]] = False
            seqs = [i for i in range(len(lens)) if i != n]
            for what, a, b in [("y", y, ry)] + [(k, out[k], ref[k]) for k in ("dx", "ddt", "dz", "dB", "dC")]:
                assert torch.equal(rows(a)[others], rows(b)[others]), (what, n, back)
            assert torch.equal(So[seqs], rS[seqs]) and torch.equal(out["dS0"][seqs], ref["dS0"][seqs]), (n, back)
    assert kda.device_error() == 0


def test_backward_of_an_empty_batch_through_the_c_abi(cuda_device):
    """No rows, every output given: the sums over tokens are zeros, as the convolution's and the norm's are."""
    d, S = 24, 16
    f = lambda *s: torch.full(s, 7.0, device=cuda_device)
    p = lambda t: t.data_ptr()
    x, B, A, v, kept = f(8, d), f(8, S), f(d, S), f(d), f(2, d, S)
    out = dict(dx=f(8, d), ddt=f(8, d), dA=f(d, S), dB=f(8, S), dC=f(8, S), dD=f(d), dz=f(8, d), db=f(d), dS0=f(2, d, S))
    for nb, T in ((0, 4), (0, 0)):
        for t in out.values():
            t.fill_(7.0)
        st = kda.load_library().kda_selective_scan_bwd(
            p(x), d, p(x), d, p(A), p(B), S, p(B), S, p(v), p(x), d, p(v), p(kept), p(x), p(kept), p(out["dx"]),
            p(out["ddt"]), p(out["dA"]), p(out["dB"]), p(out["dC"]), p(out["dD"]), p(out["dz"]), p(out["db"]),
            p(out["dS0"]), None, 0, nb, T, d, S, 1, kda.KDA_F32, None, 0, torch.cuda.current_stream().cuda_stream)
        assert st == 0, kda.last_error()
        for name in ("dA", "dD", "db"):
            assert torch.count_nonzero(out[name]) == 0, name
        for name in ("dx", "ddt", "dB", "dC", "dz", "dS0"):
            assert bool((out[name] == 7.0).all()), name


@pytest.mark.parametrize("dtype,d,S", [("f32", 4800, 64), ("bf16", 9500, 16)])
def test_packed_sequences_wide_enough_for_one_walk(cuda_device, dtype, d, S):
    """Channels that fill the card: packed sequences run unsplit too, as a batch does, and take no workspace."""
    lens = (40, 0, 90, 1, 7)
    size = kda.load_library().kda_selective_scan_fwd_workspace_size
    assert size(1, sum(lens), d, S, 1, len(lens)) == 0 and size(1, sum(lens), d // 2, S, 1, len(lens)) > 0
    assert size(16, 128, d // 16, S, 1, 0) == 0  # as many channels in rows
    v = _inputs(cuda_device, lens, d, S, 1, DT[dtype], 61, True)
    y, So = _fwd(v)
    assert kda.device_error() == 0
    _check_fwd(v, lens, y, So)
