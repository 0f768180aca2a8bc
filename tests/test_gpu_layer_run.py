"""GPU: the operators around the recurrence used together, as a layer uses
them, on other streams, from several threads, captured in graphs, and their
training pass through the layer."""
import threading

import numpy as np
import pytest
import torch

import kimi_delta_attention_31_b200 as kda
import layer_ref as R
import oracle
from layer_ref import F64, U, rel_rms

pytestmark = pytest.mark.gpu


def _layer(dev, lens, H=2, d=32, dtype=torch.float32, seed=1):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=dev)
    T, N, width = sum(lens), len(lens), 3 * H * d
    return dict(qkv=r(1, T, width).to(dtype), w=(0.5 * r(width, 4)).to(dtype), state=r(N, 3, width).to(dtype),
                a=r(1, T, H, d) - 3, b=r(1, T, H), S0=0.1 * r(N, H, d, d), norm=1 + 0.1 * r(d),
                cu=torch.tensor(R.bounds(lens), dtype=torch.int32, device=dev), H=H, d=d)


def _run_layer(v):
    """conv -> recurrence from raw projections -> norm per head, 8 bits out."""
    H, d = v["H"], v["d"]
    y, state = kda.short_conv_fwd(v["qkv"], v["w"], None, v["state"], v["cu"])
    q, k, x = (t.reshape(1, -1, H, d).contiguous() for t in y.split(H * d, -1))
    o, S = kda.chunk_fwd_prep(q, k, x, v["a"], v["b"], v["S0"], v["cu"], 16)
    out, _ = kda.rms_norm_fwd(o, v["norm"].to(o.dtype))
    q8, scale, _ = kda.rms_norm_quant_fwd(o, v["norm"].to(o.dtype), group=32)
    return out, q8, scale, S, state, (q, k, x)


def test_layer_matches_the_oracle_and_its_own_decoding(cuda_device):
    lens = (37, 0, 20)
    v = _layer(cuda_device, lens)
    out, q8, scale, S, state, (q, k, x) = _run_layer(v)
    c = lambda t: t.detach().cpu().to(F64)
    ry, rstate = R.conv(c(v["qkv"])[0], c(v["w"]), None, c(v["state"]), lens)
    assert torch.equal(c(state), rstate)
    n = lambda t: t / t.norm(dim=-1, keepdim=True).clamp_min(1e-12)
    rq, rk, rx = (t.reshape(1, -1, v["H"], v["d"]) for t in ry.split(v["H"] * v["d"], -1))
    ro, rS = oracle.recurrent(n(rq).numpy(), n(rk).numpy(), rx.contiguous().numpy(), -R.softplus(c(v["a"])).numpy(),
                              torch.sigmoid(c(v["b"])).numpy(), c(v["S0"]).numpy(),
                              cu_seqlens=np.array(R.bounds(lens), dtype=np.int64))
    want = R.norm(torch.from_numpy(np.asarray(ro)), c(v["norm"]))[0]
    # the recurrence in fp32 is held to 1e-4; the norm divides by the row's size
    assert rel_rms(out, want) <= 2e-4 and rel_rms(S, torch.from_numpy(np.asarray(rS))) <= 1e-4
    back = q8.float() * scale.repeat_interleave(32, -1)
    assert rel_rms(back, want) <= 2.0 ** -4 + 2e-4

    # one more token of the sequences, step by step, against the prefill of all of it
    tok = _layer(cuda_device, (1, 1, 1), seed=5)
    y = kda.short_conv_step(tok["qkv"][0], v["w"], state)           # state in place
    q1, k1, x1 = (t.reshape(3, v["H"], v["d"]).contiguous() for t in y.split(v["H"] * v["d"], -1))
    o1 = kda.recurrent_step_prep(q1, k1, x1, tok["a"][0], tok["b"][0], S)
    got, _ = kda.rms_norm_fwd(o1, v["norm"])
    whole, at = dict(v), R.bounds(lens)
    whole["cu"] = torch.tensor(R.bounds([m + 1 for m in lens]), dtype=torch.int32, device=cuda_device)
    for name in ("qkv", "a", "b"):
        whole[name] = torch.cat([torch.cat([v[name][:, at[i]:at[i + 1]], tok[name][:, i:i + 1]], 1) for i in range(3)], 1)
    full, *_ = _run_layer(whole)
    last = [b - 1 for b in R.bounds([m + 1 for m in lens])[1:]]
    assert rel_rms(got, full[0, last].cpu()) <= 4e-4


def test_layer_gradients(cuda_device):
    """norm, recurrence and convolution in reverse against autograd through the
    64-bit forms of all three."""
    from oracle.grad import recurrent_prep_grad
    T, H, d = 24, 1, 32
    v = _layer(cuda_device, (T,), H, d)
    out, _, _, _, _, (q, k, x) = _run_layer(v)
    o, _ = kda.chunk_fwd_prep(q, k, x, v["a"], v["b"], v["S0"], v["cu"], 16)
    dout = torch.randn_like(out)
    g1 = kda.rms_norm_bwd(dout, o, v["norm"])
    g2 = kda.chunk_bwd_prep(q, k, x, v["a"], v["b"], g1["dx"], v["S0"], None, v["cu"])
    dqkv = torch.cat([g2[n].flatten(2) for n in ("dq", "dk", "dv")], -1)
    g3 = kda.short_conv_bwd(v["qkv"], v["w"], dqkv, None, v["state"], None, v["cu"])
    c = lambda t: t.detach().cpu().to(F64)
    ro = c(o).requires_grad_(True)
    (R.norm(ro, c(v["norm"]))[0] * c(dout)).sum().backward()
    assert rel_rms(g1["dx"], ro.grad) <= 1e-4
    ref = recurrent_prep_grad(c(q).numpy(), c(k).numpy(), c(x).numpy(), c(v["a"]).numpy(), c(v["b"]).numpy(),
                              c(v["S0"]).numpy(), ro.grad.numpy(), np.zeros((1, H, d, d)))
    dref = torch.cat([torch.from_numpy(np.asarray(ref[n])).flatten(2) for n in ("dq", "dk", "dv")], -1)
    assert rel_rms(dqkv, dref) <= 3e-4
    g = R.grads(lambda x, weight: R.conv(x, weight, None, c(v["state"]), [T]),
                dict(x=c(v["qkv"])[0], weight=c(v["w"])), [dref[0], None])
    assert rel_rms(g3["dx"][0], g["x"]) <= 4e-4 and rel_rms(g3["dweight"], g["weight"]) <= 4e-4


def _block(dev, N, T, d, dtype, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=dev)
    return dict(xz=r(N, T, 2 * d).to(dtype), w=(0.5 * r(d, 4)).to(dtype), dt=(r(N, T, d) - 3).to(dtype),
                A=-torch.exp(r(d, 16)), BC=r(N, T, 1, 32).to(dtype), D=r(d), norm=(1 + 0.1 * r(d)).to(dtype),
                res=r(N, T, d).to(dtype))


def _run_block(v, upto=None):
    """conv -> scan gated by the other half of the projection -> norm with the residual."""
    d, s = v["D"].shape[0], slice(0, upto)
    x, cs = kda.short_conv_fwd(v["xz"][:, s, :d].contiguous(), v["w"])
    y, S = kda.selective_scan_fwd(x, v["dt"][:, s].contiguous(), v["A"], v["BC"][:, s, :, :16].contiguous(),
                                  v["BC"][:, s, :, 16:].contiguous(), v["D"], v["xz"][:, s, d:].contiguous())
    out, r = kda.rms_norm_fwd(y, v["norm"], v["res"][:, s].contiguous())
    return out, r, cs, S


def test_scan_block_decodes_as_it_prefills(cuda_device):
    for dtype in (torch.float32, torch.bfloat16):
        v = _block(cuda_device, 3, 80, 48, dtype, 2)
        full, _, cs_full, S_full = _run_block(v)
        _, _, cs, S = _run_block(v, 76)
        for t in range(76, 80):
            x = kda.short_conv_step(v["xz"][:, t, :48], v["w"], cs)
            y = kda.selective_scan_step(x, v["dt"][:, t], v["A"], v["BC"][:, t, :, :16], v["BC"][:, t, :, 16:], S, v["D"],
                                        v["xz"][:, t, 48:])
            out, _ = kda.rms_norm_fwd(y, v["norm"], v["res"][:, t].contiguous())
            # the same arithmetic in another order of sums: fp32 rounding, a bf16 step at most
            assert rel_rms(out.float(), full[:, t].float().cpu()) <= 1e-5 + (2 * U[dtype] if dtype != torch.float32 else 0)
        assert torch.equal(cs, cs_full) and rel_rms(S, S_full.cpu()) <= 1e-5


def _everything(v, dev):
    """Every new entry point once; a flat list of outputs."""
    outs = list(_run_block(v))
    d = v["D"].shape[0]
    x, z = v["xz"][..., :d], v["xz"][..., d:]
    B, C = v["BC"][..., :16], v["BC"][..., 16:]
    outs += [t for t in kda.selective_scan_bwd(x, v["dt"], v["A"], B, C, v["res"], v["D"], z).values() if t is not None]
    outs += [t for t in kda.short_conv_bwd(x, v["w"], v["res"]).values() if t is not None]
    outs += list(kda.rms_norm_bwd(v["res"], v["dt"], v["norm"]).values())
    q, s, _ = kda.rms_norm_quant_fwd(x, v["norm"])
    cu = torch.zeros(3, dtype=torch.int32, device=dev)
    cu[1], cu[2] = 70, 2 * v["dt"].shape[1]
    flat = lambda t: t.reshape(1, -1, *t.shape[2:])
    outs += list(kda.selective_scan_fwd(flat(x), flat(v["dt"]), v["A"], flat(B), flat(C), v["D"], flat(z), cu_seqlens=cu))
    return outs + [q.view(torch.uint8), s]


def test_streams_threads_and_graphs(cuda_device):
    v = _block(cuda_device, 2, 300, 72, torch.bfloat16, 3)
    ref = [t.clone() for t in _everything(v, cuda_device)]
    torch.cuda.synchronize()
    results, errors = {}, []

    def worker(i):
        try:
            stream = torch.cuda.Stream(cuda_device)
            with torch.cuda.stream(stream):
                for _ in range(3):
                    outs = _everything(v, cuda_device)
                with pytest.raises(ValueError):
                    kda.short_conv_fwd(v["dt"], v["w"][:7])
            stream.synchronize()
            results[i] = outs
        except Exception as e:  # noqa: BLE001  (reported below)
            errors.append(repr(e))

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for outs in results.values():
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))

    # captured, then replayed on other inputs; two graphs share the allocator's pool
    w = {k: t.clone() for k, t in v.items()}
    side = torch.cuda.Stream(cuda_device)
    with torch.cuda.stream(side):
        _everything(w, cuda_device)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0].pool() if graphs else None):
            d = w["D"].shape[0]
            x, cs = kda.short_conv_fwd(w["xz"][..., :d], w["w"])
            y, S = kda.selective_scan_fwd(x, w["dt"], w["A"], w["BC"][..., :16], w["BC"][..., 16:], w["D"],
                                          w["xz"][..., d:])
            grads = kda.selective_scan_bwd(x, w["dt"], w["A"], w["BC"][..., :16], w["BC"][..., 16:], w["res"], w["D"],
                                           w["xz"][..., d:])
            out, r = kda.rms_norm_fwd(y, w["norm"], w["res"])
            nb = kda.rms_norm_bwd(out, r, w["norm"])
            cb = kda.short_conv_bwd(w["xz"][..., :d], w["w"], grads["dx"])
        graphs.append(g)
        outs.append([y, S, out, r, nb["dweight"], cb["dweight"], grads["dA"], grads["dB"]])
    other = _block(cuda_device, 2, 300, 72, torch.bfloat16, 4)
    for src in (other, v):
        for k in w:
            w[k].copy_(src[k])
        d = src["D"].shape[0]
        x, _ = kda.short_conv_fwd(src["xz"][..., :d], src["w"])
        y, S = kda.selective_scan_fwd(x, src["dt"], src["A"], src["BC"][..., :16], src["BC"][..., 16:], src["D"],
                                      src["xz"][..., d:])
        grads = kda.selective_scan_bwd(x, src["dt"], src["A"], src["BC"][..., :16], src["BC"][..., 16:], src["res"],
                                       src["D"], src["xz"][..., d:])
        out, r = kda.rms_norm_fwd(y, src["norm"], src["res"])
        nb = kda.rms_norm_bwd(out, r, src["norm"])
        cb = kda.short_conv_bwd(src["xz"][..., :d], src["w"], grads["dx"])
        want = [y, S, out, r, nb["dweight"], cb["dweight"], grads["dA"], grads["dB"]]
        for g, got in zip(graphs, outs):
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert kda.device_error() == 0
