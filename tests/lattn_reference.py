"""Plain 64-bit forms of linear attention with a decay for each head, of the norms
of queries and keys with rotation, for the tests: token by token on the CPU,
straight from the formulas, sharing no code with the package.  Each comes with the
sum of its terms' magnitudes, which the tolerances count roundings against."""
import math

import torch


def d64(t):
    return None if t is None else t.detach().double().cpu()


def softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def steps(delta, bias, act, shape):
    """dt [.., heads, L], float64."""
    if delta is None:
        return torch.ones(shape, dtype=torch.float64)
    x = delta if bias is None else delta + bias[:, None]
    return softplus(x) if act else x


def scan(q, k, v, decay, weight, D, s0, groups, scale):
    """q, k [batch, groups*N, L], v [batch, heads*P, L], decay (A dt) and weight (dt)
    [batch, heads, L], s0 [batch, heads*P, N] or None; returns (o, state)."""
    b, h, L = weight.shape
    p, n = v.shape[1] // h, q.shape[1] // groups
    q, k = (x.reshape(b, groups, 1, n, L).expand(b, groups, h // groups, n, L).reshape(b, h, n, L) for x in (q, k))
    v = v.reshape(b, h, p, L)
    s = torch.zeros(b, h, p, n, dtype=torch.float64) if s0 is None else s0.reshape(b, h, p, n)
    out = []
    a = torch.exp(decay)
    for t in range(L):
        s = a[:, :, t, None, None] * s + (weight[:, :, None, t] * v[..., t])[..., None] * k[:, :, None, :, t]
        o = scale * (s * q[:, :, None, :, t]).sum(-1)
        if D is not None:
            o = o + D[:, None] * v[..., t]
        out.append(o)
    o = torch.stack(out, -1) if out else torch.zeros(b, h, p, 0, dtype=torch.float64)
    return o.reshape(b, h * p, L), s.reshape(b, h * p, n)


def forward(q, k, v, A, delta, D, s0, groups, scale, bias=None, act=False):
    """(o, state, magnitudes of o's terms, of state's)."""
    q, k, v, A, delta, D, s0, bias = map(d64, (q, k, v, A, delta, D, s0, bias))
    dt = steps(delta, bias, act, (v.shape[0], A.shape[0], v.shape[2]))
    decay = A[:, None] * dt
    o, s = scan(q, k, v, decay, dt, D, s0, groups, scale)
    mag = [None if x is None else x.abs() for x in (q, k, v, dt, D, s0)]
    mo, ms = scan(mag[0], mag[1], mag[2], decay, mag[3], mag[4], mag[5], groups, abs(scale))
    return o, s, mo, ms


def _grads(q, k, v, decay, weight, D, s0, do, ds, groups, scale):
    leaves = [x.clone().requires_grad_() if x is not None else None for x in (q, k, v, decay, weight, D, s0)]
    o, s = scan(*leaves[:5], leaves[5], leaves[6], groups, scale)
    total = (o * do).sum() if ds is None else (o * do).sum() + (s * ds).sum()
    names = ("dq", "dk", "dv", "dg", "dw", "dD", "ds0")
    there = [(n, x) for n, x in zip(names, leaves) if x is not None]
    got = torch.autograd.grad(total, [x for _, x in there], allow_unused=True)
    return {n: (torch.zeros_like(x) if g is None else g) for (n, x), g in zip(there, got)}


def backward(q, k, v, A, delta, D, s0, do, ds, groups, scale, bias=None, act=False):
    """(gradients, magnitudes of their terms).  dg, of the exponents A dt, is among them."""
    q, k, v, A, delta, D, s0, do, ds, bias = map(d64, (q, k, v, A, delta, D, s0, do, ds, bias))
    dt = steps(delta, bias, act, (v.shape[0], A.shape[0], v.shape[2]))
    decay = A[:, None] * dt
    chain = 1.0
    if delta is not None and act:
        chain = 1 / (1 + torch.exp(-(delta if bias is None else delta + bias[:, None])))
    out = []
    for mag in (False, True):
        f = (lambda x: None if x is None else x.abs()) if mag else (lambda x: x)
        g = _grads(f(q), f(k), f(v), decay, f(dt), f(D), f(s0), f(do), f(ds), groups, abs(scale) if mag else scale)
        g["ddelta"] = (f(A)[:, None] * g["dg"] + g["dw"]) * chain
        g["ddelta_bias"] = g["ddelta"].sum((0, 2))
        g["dA"] = (g["dg"] * f(dt)).sum((0, 2))
        out.append(g)
    return out[0], out[1]


def largest_exponent(A, dt, chunk=128):
    """The largest sum of |A dt| over the tokens of a chunk."""
    x = (A.abs()[:, None] * dt.abs())
    if x.shape[-1] == 0:
        return 0.0
    return float(torch.nn.functional.avg_pool1d(torch.nn.functional.pad(x.reshape(-1, 1, x.shape[-1]), (chunk, chunk)), chunk, 1).max()) * chunk


def packed(q, k, v, A, delta, D, cu, slots, has, state, groups, scale, bias=None, act=False):
    """(o, state, magnitudes of both) of packed requests; q, k, v, delta without a batch dimension."""
    tokens = v.shape[1]
    state = d64(state)
    out, mag_state = state.clone(), state.abs()
    o = torch.zeros(v.shape, dtype=torch.float64)
    mo = torch.zeros_like(o)
    spans, at = [], 0
    for s in range(len(cu) - 1):
        if cu[s] > at:
            spans.append((None, at, cu[s]))
        spans.append((s, cu[s], cu[s + 1]))
        at = cu[s + 1]
    if at < tokens:
        spans.append((None, at, tokens))
    for s, a, b in spans:
        row = -1 if s is None else s if slots is None else slots[s]
        first = state[row][None] if row >= 0 and (has is None or has[s]) else torch.zeros(1, *state.shape[1:], dtype=torch.float64)
        cut = [None if x is None else x[None, :, a:b] for x in (q, k, v, delta)]
        y, last, my, mlast = forward(*cut[:3], A, cut[3], D, first, groups, scale, bias, act)
        o[:, a:b], mo[:, a:b] = y[0], my[0]
        if row >= 0:
            out[row], mag_state[row] = last[0], mlast[0]
    return o, out, mo, mag_state


def heads_norm(x, w, pos, freq, eps):
    """x [.., heads, D]; pos [..]; the normalised and turned heads."""
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    if freq is None:
        return y
    r = freq.shape[0]
    a = torch.remainder(pos[..., None] * freq, 2 * math.pi)[..., None, :]
    c, s = torch.cos(a), torch.sin(a)
    return torch.cat([y[..., :r] * c - y[..., r:2 * r] * s, y[..., r:2 * r] * c + y[..., :r] * s, y[..., 2 * r:]], -1)
