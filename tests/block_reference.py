"""Plain 64-bit forms of the operators around the scan, for the tests: loops
over requests and tokens in torch float64 on the CPU, straight from the
formulas.  They share no code with the package."""
import torch


def d64(t):
    return None if t is None else t.detach().double().cpu()


def silu(x):
    return x / (1 + torch.exp(-x))


def softplus(x):
    return torch.where(x > 0, x, torch.zeros_like(x)) + torch.log1p(torch.exp(-x.abs()))


def conv(x, weight, bias, before, act=True):
    """One sequence x [.., dim, L] after `before` [.., dim, W-1]; returns (y, last inputs, magnitude of c's terms)."""
    k = weight.shape[1]
    line = torch.cat([before, x], -1)
    n = x.shape[-1]
    terms = [weight[:, j, None] * line[..., j:j + n] for j in range(k)]
    c = sum(terms)
    size = sum(t.abs() for t in terms)
    if bias is not None:
        c, size = c + bias[:, None], size + bias.abs()[:, None]
    return (silu(c) if act else c), line[..., n:], size


def spans(cu, tokens):
    """(request or None, begin, end) over all tokens, in order."""
    out, at = [], 0
    for s in range(len(cu) - 1):
        if cu[s] > at:
            out.append((None, at, cu[s]))
        out.append((s, cu[s], cu[s + 1]))
        at = cu[s + 1]
    if at < tokens:
        out.append((None, at, tokens))
    return out


def _row(slots, s):
    if s is None:
        return -1
    return s if slots is None else slots[s]


def conv_packed(x, weight, bias, cu, slots, has, state, act=True):
    y, size, state = torch.empty_like(x), torch.empty_like(x), state.clone()
    out = state.clone()
    for s, a, b in spans(cu, x.shape[1]):
        row = _row(slots, s)
        before = state[row] if row >= 0 and (has is None or has[s]) else torch.zeros(state.shape[1:], dtype=state.dtype)
        y[:, a:b], after, size[:, a:b] = conv(x[:, a:b], weight, bias, before, act)
        if row >= 0:
            out[row] = after
    return y, out, size


def scan_packed(u, delta, A, B, C, D, cu, slots, has, state, z=None, bias=None, sp=False):
    """Returns (y, cache, magnitude of y's terms)."""
    dt = delta if bias is None else delta + bias[:, None]
    dt = softplus(dt) if sp else dt
    y, size, out = torch.empty_like(u), torch.empty_like(u), state.clone()
    for s, a, b in spans(cu, u.shape[1]):
        row = _row(slots, s)
        h = state[row].clone() if row >= 0 and (has is None or has[s]) else torch.zeros(state.shape[1:], dtype=state.dtype)
        for t in range(a, b):
            h = torch.exp(dt[:, t, None] * A) * h + (dt[:, t] * u[:, t])[:, None] * B[None, :, t]
            y[:, t] = h @ C[:, t]
            size[:, t] = h.abs() @ C[:, t].abs()
        if row >= 0:
            out[row] = h
    if D is not None:
        y, size = y + D[:, None] * u, size + (D[:, None] * u).abs()
    if z is not None:
        y, size = y * silu(z), size * silu(z).abs()
    return y, out, size


def rms(v, weight, eps):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * weight


def addnorm(x, residual, weight, scale, eps):
    r = scale * x if residual is None else residual + scale * x
    return rms(r, weight, eps), r


def gatenorm(y, z, weight, groups, norm_first, eps):
    """[batch, dim, L] or [rows, dim]."""
    if y.dim() == 3:  # channels last, and back
        y, z = y.transpose(1, 2), z.transpose(1, 2)
        return gatenorm_rows(y, z, weight, groups, norm_first, eps).transpose(1, 2)
    return gatenorm_rows(y, z, weight, groups, norm_first, eps)


def gatenorm_rows(y, z, weight, groups, norm_first, eps):
    v = y if norm_first else y * silu(z)
    parts = v.unflatten(-1, (groups, -1))
    out = rms(parts, weight.view(groups, -1), eps).flatten(-2)
    return out * silu(z) if norm_first else out
