"""Refusals of the operators around the recurrence, on the CPU: the C ABI
rejects bad arguments before any launch, and the binding rejects wrong types,
shapes and layouts before it reaches the C ABI."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import kimi_delta_attention_31_b200 as kda

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4
BF, F32 = kda.KDA_BF16, kda.KDA_F32


def P(i, off=0):
    return ctypes.c_void_p(0x100000 * (i + 1) + off)


NULL = ctypes.c_void_p(0)


def _norm(**kw):
    a = dict(x=P(1), xs=256, res=P(2), w=P(3), wt=BF, y=P(4), s=P(5), rows=4, D=256, eps=1e-6, dt=BF)
    a.update(kw)
    return kda.load_library().kda_rms_norm_fwd(a["x"], a["xs"], a["res"], a["w"], a["wt"], a["y"], a["s"], a["rows"],
                                               a["D"], a["eps"], a["dt"], None)


def _quant(**kw):
    a = dict(x=P(1), xs=256, w=P(3), y=P(4), sc=P(6), s=None, rows=4, D=256, group=128, dt=BF)
    a.update(kw)
    return kda.load_library().kda_rms_norm_quant_fwd(a["x"], a["xs"], None, a["w"], BF, a["y"], a["sc"], a["s"],
                                                     a["rows"], a["D"], a["group"], 1e-6, a["dt"], None)


def test_norm_refusals():
    assert _norm(rows=0) == 0
    assert _norm(dt=5) == UNSUPPORTED and "dtype" in kda.last_error()
    assert _norm(wt=5) == UNSUPPORTED
    assert _norm(rows=-1) == INVALID and _norm(D=0) == INVALID
    assert _norm(xs=255) == INVALID
    assert _norm(D=16385, xs=16385) == UNSUPPORTED
    assert _norm(eps=-1.0) == INVALID and _norm(eps=float("nan")) == INVALID
    for name in ("x", "w", "y"):
        assert _norm(**{name: NULL}) == INVALID, name
    assert _norm(x=P(1, 1)) == ALIGNMENT and _norm(w=P(3, 2), wt=F32) == ALIGNMENT
    assert _norm(s=P(4)) == INVALID and _norm(y=P(2)) == INVALID and _norm(y=P(3)) == INVALID
    assert _norm(y=P(1), xs=512) == INVALID       # in place needs packed rows
    assert _quant(group=48) == UNSUPPORTED and _quant(D=200, xs=200, group=64) == UNSUPPORTED
    assert _quant(sc=NULL) == INVALID
    assert _quant(x=P(1, 2)) == ALIGNMENT         # group scales need 16-byte rows
    assert _quant(xs=260) == ALIGNMENT
    assert "kda_rms_norm_quant_fwd" in kda.last_error()
    lib = kda.load_library()
    need = lib.kda_rms_norm_bwd_workspace_size(100, 256)
    assert need > 0 and need % (256 * 4) == 0
    bwd = lambda dy=P(1), s=P(2), dx=P(5), dw=P(6), ws=P(7), n=need, rows=100: lib.kda_rms_norm_bwd(
        dy, s, P(3), BF, None, dx, dw, rows, 256, 1e-6, BF, ws, n, None)
    assert bwd(n=need - 1) == WORKSPACE and bwd(ws=NULL) == WORKSPACE
    assert bwd(dy=NULL) == INVALID and bwd(dw=NULL) == INVALID and bwd(dx=P(2)) == INVALID
    assert bwd(dw=P(1)) == INVALID and bwd(dw=P(6, 2)) == ALIGNMENT


def _conv(**kw):
    a = dict(x=P(1), xs=64, w=P(2), b=P(3), wt=BF, st=P(4), y=P(5), so=P(6), cu=None, ns=0, B=2, T=8, D=64, W=4, dt=BF)
    a.update(kw)
    return kda.load_library().kda_short_conv_fwd(a["x"], a["xs"], a["w"], a["b"], a["wt"], a["st"], a["y"], a["so"],
                                                 a["cu"], a["ns"], a["B"], a["T"], a["D"], a["W"], a["dt"], None)


def test_conv_refusals():
    assert _conv(B=0) == 0
    assert _conv(W=1) == UNSUPPORTED and _conv(W=5) == UNSUPPORTED and _conv(dt=9) == UNSUPPORTED
    assert _conv(xs=63) == INVALID and _conv(D=0, xs=1) == INVALID and _conv(T=-1) == INVALID
    assert _conv(cu=P(8), ns=2) == INVALID and _conv(cu=P(8), ns=0, B=1) == INVALID and _conv(ns=1) == INVALID
    assert _conv(cu=P(8, 2), ns=2, B=1) == ALIGNMENT
    for name in ("x", "w", "y"):
        assert _conv(**{name: NULL}) == INVALID, name
    assert _conv(so=P(4)) == INVALID and "alias" in kda.last_error()
    assert _conv(y=P(1)) == INVALID and _conv(so=P(5)) == INVALID
    assert _conv(x=P(1, 1)) == ALIGNMENT and _conv(b=P(3, 2), wt=F32) == ALIGNMENT
    lib = kda.load_library()
    step = lambda st=P(4), so=P(4), y=P(5), N=3: lib.kda_short_conv_step(P(1), 64, P(2), None, BF, st, y, so, N, 64, 4,
                                                                        BF, None)
    assert step(N=0) == 0 and step(N=-1) == INVALID
    assert step(st=NULL) == INVALID and step(y=P(4)) == INVALID
    need = lib.kda_short_conv_bwd_workspace_size(2, 8, 64, 4)
    bwd = lambda ws=P(9), n=need, dyt=F32, dx=P(10), dw=P(11): lib.kda_short_conv_bwd(
        P(1), 64, P(2), None, BF, None, P(5), dyt, None, dx, dw, None, None, None, 0, 2, 8, 64, 4, BF, ws, n, None)
    assert need > 0 and bwd(n=need - 1) == WORKSPACE and bwd(ws=NULL) == WORKSPACE
    assert bwd(dyt=7) == UNSUPPORTED and bwd(dx=P(1)) == INVALID and bwd(dw=P(10)) == INVALID
    assert lib.kda_short_conv_bwd_workspace_size(2, 8, 64, 5) == 0


def _scan(fn="fwd", **kw):
    a = dict(x=P(1), xs=64, dt_=P(2), dts=64, A=P(3), B=P(4), bs=32, C=P(5), cs=32, D=P(6), z=P(7), zs=64, bias=P(8),
             S0=P(9), y=P(10), So=P(11), cu=None, ns=0, nb=2, T=8, d=64, S=16, g=2, t=BF, ws=P(12), n=1 << 30)
    a.update(kw)
    lib = kda.load_library()
    head = (a["x"], a["xs"], a["dt_"], a["dts"], a["A"], a["B"], a["bs"], a["C"], a["cs"], a["D"], a["z"], a["zs"],
            a["bias"], a["S0"])
    if fn == "fwd":
        return lib.kda_selective_scan_fwd(*head, a["y"], a["So"], a["cu"], a["ns"], a["nb"], a["T"], a["d"], a["S"],
                                          a["g"], a["t"], a["ws"], a["n"], None)
    if fn == "step":
        return lib.kda_selective_scan_step(*head, a["y"], a["So"], a["nb"], a["d"], a["S"], a["g"], a["t"], None)
    o = dict(dy=P(13), dS=P(14), dx=P(15), ddt=P(16), dA=P(17), dB=P(18), dC=P(19), dD=P(20), dz=P(21), db=P(22),
             dS0=P(23))
    o.update({k: v for k, v in kw.items() if k in o})
    return lib.kda_selective_scan_bwd(*head, o["dy"], o["dS"], o["dx"], o["ddt"], o["dA"], o["dB"], o["dC"], o["dD"],
                                      o["dz"], o["db"], o["dS0"], a["cu"], a["ns"], a["nb"], a["T"], a["d"], a["S"],
                                      a["g"], a["t"], a["ws"], a["n"], None)


@pytest.mark.parametrize("fn", ["fwd", "step", "bwd"])
def test_scan_refusals(fn):
    call = lambda **kw: _scan(fn, **kw)
    for S in (0, 1, 4, 12, 24, 128):
        assert call(S=S) == UNSUPPORTED, S
    assert call(t=3) == UNSUPPORTED
    assert call(g=3) == INVALID and call(g=0) == INVALID and call(d=0) == INVALID and call(nb=-1) == INVALID
    for name in ("xs", "dts", "zs", "bs", "cs"):
        assert call(**{name: 31}) == INVALID, name
    for name in ("x", "dt_", "A", "B", "C"):
        assert call(**{name: NULL}) == INVALID, name
    assert call(x=P(1, 1)) == ALIGNMENT and call(A=P(3, 4)) == ALIGNMENT and call(S0=P(9, 8)) == ALIGNMENT
    assert call(D=P(6, 2)) == ALIGNMENT
    if fn != "bwd":
        assert call(nb=0) == 0
        assert call(y=NULL) == INVALID and call(y=P(1)) == INVALID and call(So=P(10)) == INVALID
    if fn == "fwd":
        assert call(So=P(9)) == INVALID      # chunks read S0 while another writes S_out
    if fn != "step":
        assert call(cu=P(30), ns=2) == INVALID and call(ns=2) == INVALID
        need = (kda.load_library().kda_selective_scan_fwd_workspace_size(1, 4096, 64, 16, 2, 3) if fn == "fwd" else
                kda.load_library().kda_selective_scan_bwd_workspace_size(1, 4096, 64, 16, 2))
        assert need > 0
        assert call(cu=P(30), ns=3, nb=1, T=4096, n=need - 1) == WORKSPACE
        assert call(cu=P(30), ns=3, nb=1, T=4096, ws=NULL) == WORKSPACE
        assert call(cu=P(30), ns=3, nb=1, T=4096, ws=P(12, 8), n=need) == ALIGNMENT
    if fn == "bwd":
        for name in ("dy", "dx", "ddt", "dA", "dB", "dC", "dz"):
            assert call(**{name: NULL}) == INVALID, name
        assert call(dx=P(13)) == INVALID and call(dA=P(18)) == INVALID and call(dS0=P(14)) == INVALID
        assert call(dS0=P(23, 8)) == ALIGNMENT and call(dx=P(15, 1)) == ALIGNMENT


def test_workspace_sizes_of_bad_arguments_are_zero():
    lib = kda.load_library()
    assert lib.kda_rms_norm_bwd_workspace_size(-1, 8) == 0 and lib.kda_rms_norm_bwd_workspace_size(8, 0) == 0
    assert lib.kda_selective_scan_fwd_workspace_size(1, 64, 64, 12, 1, 0) == 0
    assert lib.kda_selective_scan_bwd_workspace_size(1, 64, 64, 16, 3) == 0


def test_binding_refuses_types_shapes_and_layouts():
    bf = torch.bfloat16
    x, w = torch.zeros(2, 8, 16, dtype=bf), torch.zeros(16)
    with pytest.raises(TypeError):
        kda.rms_norm_fwd(x.half(), w)
    with pytest.raises(TypeError):
        kda.rms_norm_fwd(x, w.half())
    with pytest.raises(ValueError):
        kda.rms_norm_fwd(x, w[:8])
    with pytest.raises(TypeError):
        kda.rms_norm_fwd(x, w, residual=x.float())
    with pytest.raises(ValueError):
        kda.rms_norm_quant_fwd(x, w, group=5)
    with pytest.raises(ValueError, match="CUDA"):
        kda.rms_norm_fwd(x, w)                                     # right shapes, host tensors
    with pytest.raises(ValueError, match="evenly"):
        kda.rms_norm_fwd(torch.zeros(2, 9, 16)[:, :8], w)
    with pytest.raises(ValueError, match="adjacent"):
        kda.rms_norm_fwd(torch.zeros(2, 16, 8).transpose(1, 2), torch.zeros(16))
    with pytest.raises(ValueError, match="overlap"):
        kda.rms_norm_fwd(torch.zeros(1, 16).expand(4, 16), w)
    cw = torch.zeros(16, 4)
    with pytest.raises(ValueError):
        kda.short_conv_fwd(x, torch.zeros(16, 5))
    with pytest.raises(TypeError):
        kda.short_conv_fwd(x, cw, bias=torch.zeros(16, dtype=bf))  # not the weight's type
    with pytest.raises(ValueError):
        kda.short_conv_fwd(x, cw, state=torch.zeros(2, 4, 16, dtype=bf))
    with pytest.raises(TypeError):
        kda.short_conv_fwd(x[:1], cw, cu_seqlens=torch.tensor([0, 8]))
    with pytest.raises(ValueError):
        kda.short_conv_fwd(x, cw, cu_seqlens=torch.tensor([0, 8], dtype=torch.int32))
    with pytest.raises(ValueError):
        kda.short_conv_step(x, cw, torch.zeros(2, 3, 16, dtype=bf))
    with pytest.raises(TypeError):
        kda.short_conv_bwd(x, cw, x.half())
    A, B = torch.zeros(16, 8), torch.zeros(2, 8, 2, 8, dtype=bf)
    ok = dict(x=x, dt=x, A=A, B=B, C=B)
    for bad, err in ((dict(dt=x.float()), TypeError), (dict(A=A.to(bf)), TypeError), (dict(B=B[:, :, :, :4]), ValueError),
                     (dict(C=B.float()), TypeError), (dict(z=x[:, :4]), ValueError), (dict(D=torch.zeros(15)), ValueError),
                     (dict(S0=torch.zeros(2, 16, 16)), ValueError), (dict(B=torch.zeros(2, 8, 3, 8, dtype=bf)), ValueError),
                     (dict(), ValueError)):
        with pytest.raises(err):
            kda.selective_scan_fwd(**{**ok, **bad})
    with pytest.raises(TypeError):
        kda.selective_scan_bwd(x, x, A, B, B, x.float())
    with pytest.raises(TypeError):
        kda.selective_scan_step(x[0], x[0], A, B[0], B[0], torch.zeros(8, 16, 8, dtype=bf))


def test_import_on_a_torch_without_cuda():
    """The package imports, and refuses host tensors, where torch lacks the names of its CUDA build."""
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda_')]:\n"
            "    delattr(torch._C, n)\n"
            "import kimi_delta_attention_31_b200 as kda\n"
            "try:\n"
            "    kda.rms_norm_fwd(torch.zeros(2, 16), torch.zeros(16))\n"
            "except ValueError as e:\n"
            "    assert 'CUDA' in str(e)\n"
            "else:\n"
            "    raise SystemExit(1)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert done.returncode == 0, done.stderr


def test_binding_refuses_sizes_past_32_bits():
    """A size that the C ABI's 32-bit integers would be cut to a small one (tensors without memory: nothing is read)."""
    n = (1 << 32) + 16
    e = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="meta")
    calls = [lambda: kda.rms_norm_fwd(e(2, n), e(n)), lambda: kda.rms_norm_quant_fwd(e(2, n), e(n)),
             lambda: kda.rms_norm_bwd(e(2, n), e(2, n), e(n)),
             lambda: kda.short_conv_fwd(e(1, n, 1), e(1, 4)), lambda: kda.short_conv_fwd(e(n, 1, 1), e(1, 4)),
             lambda: kda.short_conv_bwd(e(1, 1, n), e(n, 4), e(1, 1, n)),
             lambda: kda.short_conv_step(e(n, 1), e(1, 4), e(n, 3, 1)),
             lambda: kda.short_conv_fwd(e(1, 1, 1), e(1, 4), cu_seqlens=e(n, dtype=torch.int32))]
    f32 = torch.float32
    for B, T, d, S in ((1, n, 1, 8), (n, 1, 1, 8), (1, 1, n, 8), (1, 1, 1, n)):
        x, A, b = e(B, T, d), e(d, S, dtype=f32), e(B, T, 1, S)
        calls.append(lambda x=x, A=A, b=b: kda.selective_scan_fwd(x, x, A, b, b))
        calls.append(lambda x=x, A=A, b=b: kda.selective_scan_bwd(x, x, A, b, b, x))
    x, b = e(n, 1), e(n, 1, 8)
    calls.append(lambda: kda.selective_scan_step(x, x, e(1, 8, dtype=f32), b, b, e(n, 1, 8, dtype=f32)))
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


@pytest.mark.parametrize("D", [512, 1000, 4096, 7168, 8192, 10240, 12288, 14336, 16384, 40000])
def test_conv_backward_runs_fit_one_wave(D):
    """A line of partial sums per run, as many runs of 512 channels as 148 SMs take at four CTAs each, or fewer."""
    size = kda.load_library().kda_short_conv_bwd_workspace_size
    for tokens in (1, 15, 600, 8192, 16384, 32769, 65536, 1 << 20):
        lines = size(1, tokens, D, 4) // (D * 5 * 4)
        assert 1 <= lines and lines * -(-D // 512) <= 148 * 4, (tokens, lines)


def test_no_symbol_is_shared_between_loaded_copies():
    """Static variables of inline functions (which kernels have been set up on a device) belong to their copy of the
    library: as unique symbols the first copy in a process would own them for all."""
    kda.load_library()
    out = subprocess.run(["nm", "-D", "--defined-only", kda.lib_path()], capture_output=True, text=True, check=True).stdout
    kinds = [line.split()[1] for line in out.splitlines()]
    assert "T" in kinds and "u" not in kinds
