"""Plain implementations, in 64 bits, of the operators around the recurrence
(norm, short convolution, selective scan): one token at a time, differentiable
by autograd, plus the error bounds the GPU tests hold the kernels to.

U[dtype] is the rounding of a stored value, half a step relative to it."""
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F64 = torch.float64


def silu(v):
    return v * torch.sigmoid(v)


def softplus(v):
    return v.clamp_min(0) + torch.log1p(torch.exp(-v.abs()))


def bounds(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


# ---- norm

def norm(x, weight, residual=None, eps=1e-6):
    s = x if residual is None else x + residual
    return s / (s.square().mean(-1, keepdim=True) + eps).sqrt() * weight, s


# ---- convolution: x [tokens, D], state [N, W-1, D], lens of the sequences

def conv(x, weight, bias, state, lens):
    W = weight.shape[1]
    ys, states, at = [], [], 0
    for n, length in enumerate(lens):
        rows = torch.cat([state[n], x[at:at + length]])
        at += length
        for t in range(length):
            p = (rows[t:t + W] * weight.t()).sum(0)
            ys.append(silu(p if bias is None else p + bias))
        states.append(rows[length:])
    y = torch.stack(ys) if ys else x[:0]
    return y, torch.stack(states)


# ---- scan: x, dt, z [tokens, d], B, C [tokens, groups, S], state [N, d, S]

def scan(x, dt, A, B, C, D, z, dt_bias, state, lens):
    d, groups = x.shape[1], B.shape[1]
    group = torch.arange(d) // (d // groups)
    delta = softplus(dt if dt_bias is None else dt + dt_bias)
    ys, states, at = [], [], 0
    for n, length in enumerate(lens):
        h = state[n]
        for t in range(at, at + length):
            h = torch.exp(delta[t][:, None] * A) * h + (delta[t] * x[t])[:, None] * B[t][group]
            y = (h * C[t][group]).sum(1)
            if D is not None:
                y = y + D * x[t]
            ys.append(y if z is None else y * silu(z[t]))
        at += length
        states.append(h)
    y = torch.stack(ys) if ys else x[:0]
    return y, torch.stack(states)


def scan_error(x, dt, A, B, C, D, z, dt_bias, state, lens, dtype):
    """Bounds on |y - y_ref| and |h - h_ref| of a scan in fp32.  Every factor of
    a step carries a relative error of at most k = 2^-21 (the exponential and the
    softplus are good to a few units of 2^-23, and an error of the exponent
    counts times its size), so with H the sum of the terms' sizes
      E_t = a E_{t-1} + k (a (1 + |delta A|) H_{t-1} + |u B|),  H_t = a H_{t-1} + |u B|.
    A state that comes through chunks is a product of sums over up to a chunk's
    tokens, whose exponents carry the same relative error."""
    k = 2.0 ** -21
    d, groups = x.shape[1], B.shape[1]
    group = torch.arange(d) // (d // groups)
    delta = softplus(dt if dt_bias is None else dt + dt_bias)
    ys, es, at = [], [], 0
    for n, length in enumerate(lens):
        H, E = state[n].abs(), torch.zeros_like(state[n])
        for t in range(at, at + length):
            e = delta[t][:, None] * A
            a, ub = torch.exp(e), ((delta[t] * x[t])[:, None] * B[t][group]).abs()
            E = a * E + k * (a * (1 + e.abs()) * H + ub)
            H = a * H + ub
            c = C[t][group].abs()
            err = (c * (E + k * H)).sum(1)
            size = (c * H).sum(1)
            if D is not None:
                err, size = err + k * (D * x[t]).abs(), size + (D * x[t]).abs()
            if z is not None:  # sigmoid: relative error 2^-22 (4 + |z|)
                g = silu(z[t]).abs()
                err = g * err + g * size * 2.0 ** -22 * (4 + z[t].abs())
            ys.append(err)
        at += length
        es.append(E)
    ey = torch.stack(ys) if ys else x[:0]
    return ey, torch.stack(es)


def grads(f, inputs, weights):
    """Gradients of sum_i <weights_i, f_i(inputs)> by autograd; inputs a dict of
    64-bit tensors (or None)."""
    leaves = {k: (None if v is None else v.detach().clone().requires_grad_(True)) for k, v in inputs.items()}
    outs = f(**leaves)
    loss = sum((o * w).sum() for o, w in zip(outs, weights) if w is not None)
    loss.backward()
    return {k: (None if v is None else (v.grad if v.grad is not None else torch.zeros_like(v)))
            for k, v in leaves.items()}


def rel_rms(got, ref):
    got, ref = got.detach().to("cpu", F64), ref.detach().to(F64)
    if ref.numel() == 0:
        return 0.0
    return float((got - ref).norm() / ref.norm().clamp_min(1e-30))


def within(got, ref, bound, what=""):
    got, ref = got.detach().to("cpu", F64), ref.detach().to(F64)
    over = (got - ref).abs() - bound
    assert bool((over <= 0).all()), f"{what}: {float(over.max()):.3e} over the bound at {int(over.argmax())}"
