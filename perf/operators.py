"""The operators around the selective scan, as cases to be timed and compared.

Four operators of one layer: the short causal convolution before the scan, the
scan over packed prompts and single tokens with its state cache, the RMS norm
before the layer fused with the residual addition, and the gated RMS norm after
the scan.  ``run`` computes a case with elementary torch operations in 32 bits
(``own`` false) or with this package's entry points (``own`` true); ``exact``
computes the same outputs from the definitions in 64 bits.

Common words: T tokens of several requests laid end to end along the time axis
(``packed``), ``cu`` their S + 1 offsets, ``slots`` the cache row of each
request (negative: a padding request that keeps no state), ``has`` whether a
request continues from its cached state or starts from zeros.
"""
import math
import random

import torch

own = False

EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one short chat turn through a d_inner = 5120 layer: launch latency
        dict(name="conv_prompt_chat", op="conv_prompt", dtype="bf16", dim=5120, tokens=37, requests=1, width=4),
        # a full prefill batch of mixed prompts, some empty, unaligned rows
        dict(name="conv_prompt_mixed", op="conv_prompt", dtype="bf16", dim=5120, tokens=16411, requests=48, width=4),
        # one decode step for 256 requests over a cache of 320 slots, padded as a fixed-size decode batch is
        dict(name="conv_step_b256", op="conv_step", dtype="bf16", dim=5120, batch=256, width=4, padding=7),
        # a training step (forward and gradients) at the 4 x 2048 x 2048 bf16 shape of the scan
        dict(name="conv_train", op="conv_train", dtype="bf16", batch=4, dim=2048, len=2048, width=4),
        # one short chat turn through the scan
        dict(name="scan_prompt_chat", op="scan_prompt", dtype="bf16", dim=5120, tokens=37, requests=1, states=16, options=True),
        # a prefill batch of mixed prompts with delta bias, softplus and gate, odd total
        dict(name="scan_prompt_mixed", op="scan_prompt", dtype="bf16", dim=2048, tokens=8209, requests=24, states=16, options=True),
        # one very long document in fp32 (the 1536 x 65536 shape of the scan)
        dict(name="scan_prompt_long", op="scan_prompt", dtype="f32", dim=1536, tokens=65536, requests=1, states=16, options=False),
        # one decode step for 256 requests of a d_inner = 5120 layer
        dict(name="scan_step_b256", op="scan_step", dtype="bf16", dim=5120, batch=256, states=16, padding=7),
        # the norm before the layer for a handful of decoded tokens: latency
        dict(name="addnorm_step", op="addnorm_step", dtype="bf16", rows=3, width=2560, scale=1.0),
        # a training step of it: 4 x 2048 tokens, fp32 residual
        dict(name="addnorm_train", op="addnorm_train", dtype="bf16", rows=8192, width=2560, scale=0.5),
        # the gated norm after the scan for 256 decoded tokens
        dict(name="gatenorm_step", op="gatenorm_step", dtype="bf16", batch=256, dim=5120, groups=1, norm_first=False),
        # a training step of it in the scan's channel-major layout
        dict(name="gatenorm_train", op="gatenorm_train", dtype="bf16", batch=4, dim=2048, len=2048, groups=1, norm_first=False),
    ]


def _log(rng, low, high):
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    n = min(high, max(low, n if rng.random() < 0.6 else n | 1))
    return n if n < 1024 or n % 1024 else n - 1  # the round sizes are among the listed cases


def _dim(rng, low=64, high=5120):
    n = _log(rng, low, high)
    return n | 1 if n < 80 or rng.random() < 0.3 else n // 80 * 80


def draw(rng):
    op = rng.choice(["conv_prompt", "conv_step", "conv_train", "scan_prompt", "scan_prompt", "scan_step",
                     "addnorm_step", "addnorm_train", "gatenorm_step", "gatenorm_train"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op in ("conv_prompt", "scan_prompt"):
        c["dim"] = _dim(rng)
        most = 40_000_000 if op == "conv_prompt" else 16_000_000
        c["tokens"] = _log(rng, 1, max(1, min(16384, most // c["dim"])))
        c["requests"] = _log(rng, 1, 64)
        if op == "conv_prompt":
            c["width"] = rng.choice([2, 3, 4, 4])
        else:
            c["states"] = rng.choice([4, 16, 16, 16, 24, 64])
            c["options"] = rng.random() < 0.6
    elif op in ("conv_step", "scan_step"):
        c["dim"], c["batch"], c["padding"] = _dim(rng), _log(rng, 1, 256), rng.randint(0, 8)
        if op == "conv_step":
            c["width"] = rng.choice([2, 3, 4, 4])
        else:
            c["states"] = rng.choice([4, 7, 16, 16])
    elif op in ("conv_train", "gatenorm_train"):
        c["batch"], c["dim"] = rng.randint(1, 4), _dim(rng, high=4096)
        c["len"] = _log(rng, 1, min(4096, 16_000_000 // (c["batch"] * c["dim"])))
        if op == "conv_train":
            c["width"] = rng.choice([2, 3, 4, 4])
        else:
            c["groups"] = rng.choice([g for g in (1, 1, 2, 8) if c["dim"] % g == 0])
            c["norm_first"] = rng.random() < 0.3
    elif op in ("addnorm_step", "addnorm_train"):
        c["rows"] = _log(rng, 1, 256 if op == "addnorm_step" else 8192)
        c["width"] = _dim(rng, high=2560)
        c["scale"] = rng.choice([1.0, 0.5, 0.22])
    else:
        c["batch"], c["dim"] = _log(rng, 1, 256), _dim(rng)
        c["groups"] = rng.choice([g for g in (1, 1, 2, 8) if c["dim"] % g == 0])
        c["norm_first"] = rng.random() < 0.3
    return c


def work(case):
    c, op, io = case, case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "conv_prompt":
        n, d, w = c["tokens"], c["dim"], c["width"]
        return dict(bytes=io * 2 * d * n + 4 * d * (w + 1) + 2 * io * c["requests"] * d * (w - 1), flops=d * n * (2 * w + 5))
    if op == "conv_step":
        n, d, w = c["batch"], c["dim"], c["width"]
        return dict(bytes=io * n * d * 2 + 2 * io * (n - min(c["padding"], n - 1)) * d * (w - 1) + 4 * d * (w + 1),
                    flops=d * n * (2 * w + 5))
    if op == "conv_train":
        n, w = c["batch"] * c["dim"] * c["len"], c["width"]
        return dict(bytes=io * 5 * n + 8 * c["dim"] * (w + 1), flops=n * (2 * w + 5 + 6 * w + 10))
    if op == "scan_prompt":
        n, d, s, z = c["tokens"], c["dim"], c["states"], 1 if c["options"] else 0
        return dict(bytes=io * (d * n * (3 + z) + 2 * s * n) + 4 * d * s + 8 * c["requests"] * d * s, flops=d * n * s * 7)
    if op == "scan_step":
        n, d, s = c["batch"], c["dim"], c["states"]
        return dict(bytes=io * 4 * n * d + 8 * (n - min(c["padding"], n - 1)) * d * s + 4 * d * s + io * 2 * n * s,
                    flops=d * n * s * 7)
    if op == "addnorm_step":
        n = c["rows"] * c["width"]
        return dict(bytes=n * (2 * io + 8) + 4 * c["width"], flops=7 * n)
    if op == "addnorm_train":
        n = c["rows"] * c["width"]
        return dict(bytes=n * (2 * io + 8) + n * (2 * io + 12) + 12 * c["width"], flops=20 * n)
    if op == "gatenorm_step":
        n = c["batch"] * c["dim"]
        return dict(bytes=n * 3 * io + 4 * c["dim"], flops=10 * n)
    n = c["batch"] * c["dim"] * c["len"]
    return dict(bytes=n * 8 * io + 12 * c["dim"], flops=40 * n)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _offsets(seed, tokens, requests):
    """S + 1 offsets of requests of very different lengths; about one in eight is empty."""
    r = random.Random(seed)
    share = [0.0 if requests > 1 and r.random() < 0.125 else math.exp(r.gauss(0, 1)) for _ in range(requests)]
    if not any(share):
        share[r.randrange(requests)] = 1.0
    total, at, cu = sum(share), 0.0, [0]
    for s in share:
        at += s
        cu.append(min(tokens, int(round(tokens * at / total))))
    cu[-1] = tokens
    return cu


def _cache(seed, requests, padding):
    """(slots, has, number of slots): distinct cache rows in mixed order; the last `padding` requests have none."""
    r = random.Random(seed + 1)
    n = requests + requests // 4 + 1
    slots = r.sample(range(n), requests)
    for i in range(min(padding, requests - 1)):
        slots[-1 - i] = -1
    return slots, [r.random() < 0.5 for _ in range(requests)], n


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    io = DTYPES[c["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device=dev) * std + mean).to(dtype)

    def cache(requests, padding):
        slots, has, n = _cache(seed, requests, padding)
        return (torch.tensor(slots, dtype=torch.int32, device=dev), torch.tensor(has, dtype=torch.bool, device=dev), n)

    s = dict(case=dict(c), io=io)
    op = c["op"]
    if op.startswith("conv"):
        d, w = c["dim"], c["width"]
        s["weight"] = normal(d, w, std=w ** -0.5)
        s["bias"] = normal(d, std=0.1)
    if op == "conv_prompt":
        # x is the first half of the joint projection of x and z
        s["x"] = normal(2 * d, c["tokens"], dtype=io)[:d]
        s["cu"] = torch.tensor(_offsets(seed, c["tokens"], c["requests"]), dtype=torch.int32, device=dev)
        s["slots"], s["has"], n = cache(c["requests"], 0)
        s["state"] = normal(n, d, w - 1, dtype=io)
    elif op == "conv_step":
        s["x"] = normal(c["batch"], d, dtype=io)
        s["slots"], _, n = cache(c["batch"], c["padding"])
        s["state"] = normal(n, d, w - 1, dtype=io)
    elif op == "conv_train":
        s["x"] = normal(c["batch"], 2 * d, c["len"], dtype=io)[:, :d]
        s["dy"] = normal(c["batch"], d, c["len"], dtype=io)
    elif op in ("scan_prompt", "scan_step"):
        d, n = c["dim"], c["states"]
        options = op == "scan_step" or c["options"]
        lead = (d, c["tokens"]) if op == "scan_prompt" else (c["batch"], d)
        side = (n, c["tokens"]) if op == "scan_prompt" else (c["batch"], n)
        s["u"] = normal(*lead, dtype=io)
        raw = normal(*lead, mean=-3.0 if c["dtype"] == "bf16" else -4.0, std=1.0 if c["dtype"] == "bf16" else 0.5)
        s["delta"] = raw.to(io) if options else torch.log1p(torch.exp(raw)).to(io)
        rate = torch.rand((d, n), generator=g, device=dev) + 0.5
        s["A"] = -torch.arange(1, n + 1, device=dev, dtype=torch.float32) * rate
        s["B"], s["C"] = normal(*side, dtype=io), normal(*side, dtype=io)
        s["D"] = normal(d)
        s["bias"] = normal(d, std=0.1) if options else None
        # z is the second half of the joint projection of x and z
        half = (2 * d, c["tokens"]) if op == "scan_prompt" else lead
        s["z"] = normal(*half, dtype=io)[-lead[0]:] if options else None
        if op == "scan_prompt":
            s["cu"] = torch.tensor(_offsets(seed, c["tokens"], c["requests"]), dtype=torch.int32, device=dev)
            s["slots"], s["has"], rows = cache(c["requests"], 0)
        else:
            s["slots"], _, rows = cache(c["batch"], c["padding"])
        s["state"] = normal(rows, d, n, std=0.5)
    elif op.startswith("addnorm"):
        s["x"] = normal(c["rows"], c["width"], dtype=io)
        s["residual"] = normal(c["rows"], c["width"], std=2.0)
        s["weight"] = normal(c["width"], std=0.1, mean=1.0)
        if op == "addnorm_train":
            s["dy"] = normal(c["rows"], c["width"], dtype=io)
            s["dr"] = normal(c["rows"], c["width"])
    else:
        shape = (c["batch"], c["dim"]) if op == "gatenorm_step" else (c["batch"], c["dim"], c["len"])
        s["y"] = normal(*shape, dtype=io)
        s["z"] = normal(shape[0], 2 * c["dim"], *shape[2:], dtype=io)[:, c["dim"]:]
        s["weight"] = normal(c["dim"], std=0.1, mean=1.0)
        if op == "gatenorm_train":
            s["dout"] = normal(*shape, dtype=io)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import linear_recurrence_gb300 as lr

    c, op = s["case"], s["case"]["op"]
    if op == "conv_prompt":
        y = lr.sconv_prompt(s["x"], s["weight"], s["bias"], cu_seqlens=s["cu"], state=s["state"], slots=s["slots"],
                            has_state=s["has"])
        return dict(y=y, state=s["state"])
    if op == "conv_step":
        y = lr.sconv_step(s["x"], s["weight"], s["bias"], state=s["state"], slots=s["slots"])
        return dict(y=y, state=s["state"])
    if op == "conv_train":
        y, last = lr.sconv_fwd(s["x"], s["weight"], s["bias"])
        g = lr.sconv_bwd(s["x"], s["weight"], s["bias"], None, s["dy"])
        return dict(y=y, last=last, dx=g["dx"], dweight=g["dweight"], dbias=g["dbias"])
    if op == "scan_prompt":
        y = lr.sscan_prompt(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], cu_seqlens=s["cu"], state=s["state"],
                            slots=s["slots"], has_state=s["has"], z=s["z"], delta_bias=s["bias"],
                            delta_softplus=c["options"])
        return dict(y=y, state=s["state"])
    if op == "scan_step":
        y = lr.sscan_step(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], state=s["state"], slots=s["slots"],
                          z=s["z"], delta_bias=s["bias"], delta_softplus=True)
        return dict(y=y, state=s["state"])
    if op == "addnorm_step":
        y, r = lr.addnorm_fwd(s["x"], s["residual"], s["weight"], scale=c["scale"], eps=EPS)
        return dict(y=y, residual=r)
    if op == "addnorm_train":
        y, r = lr.addnorm_fwd(s["x"], s["residual"], s["weight"], scale=c["scale"], eps=EPS)
        g = lr.addnorm_bwd(r, s["weight"], s["dy"], s["dr"], scale=c["scale"], eps=EPS)
        return dict(y=y, residual=r, dx=g["dx"], dresidual=g["dresidual"], dweight=g["dweight"])
    if op == "gatenorm_step":
        return dict(out=lr.gatenorm_step(s["y"], s["z"], s["weight"], groups=c["groups"], norm_first=c["norm_first"],
                                         eps=EPS))
    out = lr.gatenorm_fwd(s["y"], s["z"], s["weight"], groups=c["groups"], norm_first=c["norm_first"], eps=EPS)
    g = lr.gatenorm_bwd(s["y"], s["z"], s["weight"], s["dout"], groups=c["groups"], norm_first=c["norm_first"], eps=EPS)
    return dict(out=out, dy=g["dy"], dz=g["dz"], dweight=g["dweight"])


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


def _keep(cache, slots, new, padding):
    """Write each request's new state to its cache row; padding requests have none."""
    if not padding:
        cache.index_copy_(0, slots.long(), new.to(cache.dtype))
        return
    n, k = cache.shape[0], slots.shape[0]
    of = torch.full((n + 1,), -1, dtype=torch.long, device=cache.device)
    of[torch.where(slots < 0, n, slots).long()] = torch.arange(k, device=cache.device)
    of = of[:n]
    shape = (n,) + (1,) * (cache.dim() - 1)
    cache.copy_(torch.where((of >= 0).view(shape), new.to(cache.dtype)[of.clamp(min=0)], cache))


def _run_plain(s):
    return globals()["_plain_" + s["case"]["op"]](s)


def _plain_conv_prompt(s):
    x, w, cu = s["x"].float(), s["weight"], s["cu"].long()
    d, t, k = x.shape[0], x.shape[1], w.shape[1] - 1
    n = cu.shape[0] - 1
    first = torch.where(s["has"].view(n, 1, 1), s["state"][s["slots"].long()].float(), 0.0)
    both = torch.cat([x, first.permute(1, 0, 2).reshape(d, n * k)], 1)  # inputs, then every request's state
    at = torch.arange(t, device=x.device)
    of = torch.searchsorted(cu[1:], at, right=True)
    tap = at[:, None] + torch.arange(-k, 1, device=x.device)
    begin = cu[of][:, None]
    tap = torch.where(tap >= begin, tap, t + of[:, None] * k + k + tap - begin)
    a = (both[:, tap] * w[:, None, :]).sum(-1) + s["bias"][:, None]
    y = (a * _sigmoid(a)).to(s["io"])
    last = cu[1:, None] + torch.arange(-k, 0, device=x.device)
    last = torch.where(last >= cu[:-1, None], last,
                       t + torch.arange(n, device=x.device)[:, None] * k + k + last - cu[:-1, None])
    _keep(s["state"], s["slots"], both[:, last].permute(1, 0, 2), False)
    return dict(y=y, state=s["state"])


def _plain_conv_step(s):
    slots = s["slots"]
    first = torch.where((slots >= 0).view(-1, 1, 1), s["state"][slots.clamp(min=0).long()].float(), 0.0)
    taps = torch.cat([first, s["x"].float()[:, :, None]], 2)
    a = (taps * s["weight"]).sum(-1) + s["bias"]
    _keep(s["state"], slots, taps[:, :, 1:], s["case"]["padding"])
    return dict(y=(a * _sigmoid(a)).to(s["io"]), state=s["state"])


def _plain_conv_train(s):
    x, w, dy = s["x"].float(), s["weight"], s["dy"].float()
    k = w.shape[1] - 1
    b, d, n = x.shape
    none = torch.zeros(b, d, k, device=x.device)
    taps = torch.cat([none, x], 2).unfold(2, k + 1, 1)  # a view: [b, d, t, tap]
    a = (taps * w[:, None, :]).sum(-1) + s["bias"][:, None]
    g = _sigmoid(a)
    da = dy * g * (1 + a * (1 - g))
    dx = (torch.cat([da, none], 2).unfold(2, k + 1, 1) * w.flip(1)[:, None, :]).sum(-1)
    return dict(y=(a * g).to(s["io"]), last=torch.cat([none, x], 2)[:, :, n:].to(s["io"]), dx=dx.to(s["io"]),
                dweight=(taps * da[..., None]).sum((0, 2)), dbias=da.sum((0, 2)))


def _plain_scan_prompt(s):
    c = s["case"]
    u, delta, cu = s["u"].float(), s["delta"].float(), s["cu"].long()
    d, t = u.shape
    n = cu.shape[0] - 1
    if c["options"]:
        delta = _softplus(delta + s["bias"][:, None])
    first = torch.where(s["has"].view(n, 1, 1), s["state"][s["slots"].long()], 0.0)
    a = torch.exp(delta[:, None, :] * s["A"][:, :, None])
    h = (delta * u)[:, None, :] * s["B"].float()[None]
    # a request's first step takes its initial state in and cuts it off from the request before
    full = cu[1:] > cu[:-1]
    at = torch.where(full, cu[:-1], t)
    begins = torch.zeros(t + 1, dtype=torch.bool, device=u.device).index_fill_(0, at, True)[:t]
    inside = at.clamp(max=t - 1)
    h = h.index_add(2, inside, torch.where(at < t, a[:, :, inside] * first.permute(1, 2, 0), 0.0))
    a = torch.where(begins, 0.0, a)
    k = 1
    while k < t:  # inclusive scan of (a, h) by doubling strides
        h = torch.cat([h[..., :k], torch.addcmul(h[..., k:], a[..., k:], h[..., :-k])], -1)
        a = torch.cat([a[..., :k], a[..., k:] * a[..., :-k]], -1)
        k *= 2
    y = (h * s["C"].float()[None]).sum(1) + s["D"][:, None] * u
    if c["options"]:
        z = s["z"].float()
        y = y * z * _sigmoid(z)
    last = h[:, :, (cu[1:] - 1).clamp(min=0)].permute(2, 0, 1)
    _keep(s["state"], s["slots"], torch.where(full.view(n, 1, 1), last, first), False)
    return dict(y=y.to(s["io"]), state=s["state"])


def _plain_scan_step(s):
    slots = s["slots"]
    delta = _softplus(s["delta"].float() + s["bias"])[:, :, None]
    u, z = s["u"].float(), s["z"].float()
    first = torch.where((slots >= 0).view(-1, 1, 1), s["state"][slots.clamp(min=0).long()], 0.0)
    h = torch.exp(delta * s["A"]) * first + delta * u[:, :, None] * s["B"].float()[:, None, :]
    y = ((h * s["C"].float()[:, None, :]).sum(-1) + s["D"] * u) * z * _sigmoid(z)
    _keep(s["state"], slots, h, s["case"]["padding"])
    return dict(y=y.to(s["io"]), state=s["state"])


def _plain_addnorm_step(s):
    r = s["residual"] + s["case"]["scale"] * s["x"].float()
    y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["weight"]
    return dict(y=y.to(s["io"]), residual=r)


def _plain_addnorm_train(s):
    scale = s["case"]["scale"]
    r = s["residual"] + scale * s["x"].float()
    rstd = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    n = r * rstd
    dy = s["dy"].float()
    g = dy * s["weight"]
    dr = s["dr"] + rstd * (g - n * (g * n).mean(-1, keepdim=True))
    return dict(y=(n * s["weight"]).to(s["io"]), residual=r, dx=(scale * dr).to(s["io"]), dresidual=dr,
                dweight=(dy * n).sum(0))


def _plain_gatenorm_step(s):
    c = s["case"]
    y, z, w = s["y"].float(), s["z"].float(), s["weight"]
    gate = z * _sigmoid(z)
    v = y if c["norm_first"] else y * gate
    v = v.view(c["batch"], c["groups"], -1)
    out = (v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)).view(c["batch"], -1) * w
    return dict(out=(out * gate if c["norm_first"] else out).to(s["io"]))


def _plain_gatenorm_train(s):
    c = s["case"]
    shape = (c["batch"], c["groups"], c["dim"] // c["groups"], c["len"])
    y, z, do = (s[k].float().view(shape) for k in ("y", "z", "dout"))
    w = s["weight"].view(shape[1], shape[2], 1)
    sig = _sigmoid(z)
    gate = z * sig
    v = y if c["norm_first"] else y * gate
    rstd = torch.rsqrt((v * v).mean(2, keepdim=True) + EPS)
    n = v * rstd
    up = do * gate if c["norm_first"] else do  # gradient of n * w
    q = up * w
    dv = rstd * (q - n * (q * n).mean(2, keepdim=True))
    dgate = do * n * w if c["norm_first"] else dv * y
    out = n * w * gate if c["norm_first"] else n * w
    full = (c["batch"], c["dim"], c["len"])
    return dict(out=out.view(full).to(s["io"]), dy=(dv if c["norm_first"] else dv * gate).view(full).to(s["io"]),
                dz=(dgate * sig * (1 + z * (1 - sig))).view(full).to(s["io"]),
                dweight=(up * n).sum((0, 3)).reshape(-1))


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    return globals()["_exact_" + {"conv_prompt": "conv_packed", "scan_prompt": "scan_packed"}.get(case["op"], case["op"])](case, f)


def _conv64(x, before, w, bias):
    """One sequence [.., dim, L] with its W - 1 earlier inputs; also the inputs that the next one needs."""
    k = w.shape[1]
    line = torch.cat([before, x], -1)
    n = x.shape[-1]
    a = bias[:, None] + sum(w[:, j, None] * line[..., j:j + n] for j in range(k))
    return torch.nn.functional.silu(a), line[..., n:]


def _exact_conv_packed(case, f):
    cu, slots, has = f["cu"].tolist(), f["slots"].tolist(), f["has"].tolist()
    y, state = torch.empty_like(f["x"]), f["state"].clone()
    for i, row in enumerate(slots):
        before = state[row] if has[i] else torch.zeros_like(state[row])
        y[:, cu[i]:cu[i + 1]], state[row] = _conv64(f["x"][:, cu[i]:cu[i + 1]], before, f["weight"], f["bias"])
    return dict(y=y, state=state)


def _exact_conv_step(case, f):
    y, state = torch.empty_like(f["x"]), f["state"].clone()
    for i, row in enumerate(f["slots"].tolist()):
        before = state[row] if row >= 0 else torch.zeros_like(state[0])
        out, after = _conv64(f["x"][i][:, None], before, f["weight"], f["bias"])
        y[i] = out[:, 0]
        if row >= 0:
            state[row] = after
    return dict(y=y, state=state)


def _exact_conv_train(case, f):
    x, w, b = (f[k].detach().clone().requires_grad_() for k in ("x", "weight", "bias"))
    y, last = _conv64(x, torch.zeros_like(x[..., :1]).expand(-1, -1, case["width"] - 1), w, b)
    dx, dw, db = torch.autograd.grad(y, (x, w, b), f["dy"])
    return dict(y=y.detach(), last=last.detach(), dx=dx, dweight=dw, dbias=db)


def _exact_scan_packed(case, f):
    u, A, B, C = f["u"], f["A"], f["B"], f["C"]
    dt = torch.nn.functional.softplus(f["delta"] + f["bias"][:, None], threshold=40) if case["options"] else f["delta"]
    cu, slots, has = f["cu"].tolist(), f["slots"].tolist(), f["has"].tolist()
    y, state = torch.empty_like(u), f["state"].clone()
    dts, ins, Bs, Cs = dt.t().contiguous(), (dt * u).t().contiguous(), B.t().contiguous(), C.t().contiguous()
    out = torch.empty_like(dts)
    for i, row in enumerate(slots):
        h = state[row].clone() if has[i] else torch.zeros_like(state[row])
        for t in range(cu[i], cu[i + 1]):
            h = torch.addr(torch.exp(dts[t, :, None] * A).mul_(h), ins[t], Bs[t])
            torch.mv(h, Cs[t], out=out[t])
        state[row] = h
    y = out.t() + f["D"][:, None] * u
    if case["options"]:
        y = y * torch.nn.functional.silu(f["z"])
    return dict(y=y.contiguous(), state=state)


def _exact_scan_step(case, f):
    y, state = torch.empty_like(f["u"]), f["state"].clone()
    for i, row in enumerate(f["slots"].tolist()):
        dt = torch.nn.functional.softplus(f["delta"][i] + f["bias"], threshold=40)
        h = state[row] if row >= 0 else torch.zeros_like(state[0])
        h = torch.exp(torch.outer(dt, torch.ones_like(f["B"][i])) * f["A"]) * h + torch.outer(dt * f["u"][i], f["B"][i])
        y[i] = (h @ f["C"][i] + f["D"] * f["u"][i]) * torch.nn.functional.silu(f["z"][i])
        if row >= 0:
            state[row] = h
    return dict(y=y, state=state)


def _norm64(v, w):
    return v / (v.square().sum(-1, keepdim=True) / v.shape[-1] + EPS).sqrt() * w


def _exact_addnorm_step(case, f):
    r = f["residual"] + case["scale"] * f["x"]
    return dict(y=_norm64(r, f["weight"]), residual=r)


def _exact_addnorm_train(case, f):
    x, res, w = (f[k].detach().clone().requires_grad_() for k in ("x", "residual", "weight"))
    r = res + case["scale"] * x
    y = _norm64(r, w)
    dx, dres, dw = torch.autograd.grad((y, r), (x, res, w), (f["dy"], f["dr"]))
    return dict(y=y.detach(), residual=r.detach(), dx=dx, dresidual=dres, dweight=dw)


def _gated64(case, y, z, w):
    """Channels last."""
    gate = torch.nn.functional.silu(z)
    parts = (y if case["norm_first"] else y * gate).unflatten(-1, (case["groups"], -1))
    out = _norm64(parts, w.view(case["groups"], -1)).flatten(-2)
    return out * gate if case["norm_first"] else out


def _exact_gatenorm_step(case, f):
    return dict(out=_gated64(case, f["y"], f["z"], f["weight"]))


def _exact_gatenorm_train(case, f):
    y, z, w = (f[k].detach().clone().requires_grad_() for k in ("y", "z", "weight"))
    out = _gated64(case, y.transpose(1, 2), z.transpose(1, 2), w).transpose(1, 2)
    dy, dz, dw = torch.autograd.grad(out, (y, z, w), f["dout"])
    return dict(out=out.detach().contiguous(), dy=dy, dz=dz, dweight=dw)
