"""Linear attention with a decay for each head, and what stands around it, as cases to be timed and compared.

Three operators: linear attention with a decay for each head (the scan with one
rate a head and a matrix of states: training, packed prompts and single tokens
over a cache), the norm of queries and keys for each head with the rotation by
position, and the copying, forking, compacting and freeing of cache rows.
``run`` computes a case with elementary torch operations (``own`` false) or with
this package's entry points (``own`` true); ``exact`` computes the same outputs
from the definitions in 64 bits.

Common words: T tokens of several requests laid end to end along the time axis,
``cu`` their S + 1 offsets, ``slots`` the cache row of each request (negative: a
padding request that keeps no state), ``has`` whether a request continues from
its cached state or starts from zeros.  A head of ``value`` channels keeps a
state [value, key]; ``groups`` sets of queries and keys are shared by equal
numbers of heads.
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
        # one decode step of 256 requests through a d_inner = 5120 layer of 80 heads, padded as a fixed-size batch is
        dict(name="lattn_step_b256", op="lattn_step", dtype="bf16", heads=80, value=64, key=128, groups=1, batch=256, padding=7),
        # one short chat turn through that layer: latency
        dict(name="lattn_prompt_chat", op="lattn_prompt", dtype="bf16", heads=80, value=64, key=128, groups=1, tokens=37,
             requests=1),
        # a prefill batch of mixed prompts, some empty, rows of odd length
        dict(name="lattn_prompt_mixed", op="lattn_prompt", dtype="bf16", heads=80, value=64, key=128, groups=8, tokens=8209,
             requests=24),
        # one very long document with few heads: time itself has to be split (the 1536 x 65536 shape of the scan)
        dict(name="lattn_prompt_long", op="lattn_prompt", dtype="bf16", heads=24, value=64, key=64, groups=1, tokens=65536,
             requests=1),
        # a training step (forward and gradients) at the 4 x 2048 x 2048 bf16 shape of the scan
        dict(name="lattn_train", op="lattn_train", dtype="bf16", heads=32, value=64, key=128, groups=1, batch=4, len=2048,
             steps=True),
        # a training step in fp32 with one fixed decay a head and queries and keys of each head's own
        dict(name="lattn_train_fixed", op="lattn_train", dtype="f32", heads=8, value=64, key=64, groups=8, batch=1, len=2047,
             steps=False),
        # the norms and rotation of a handful of decoded tokens: latency
        dict(name="qknorm_step", op="qknorm_step", dtype="bf16", heads=32, key_heads=8, dim=128, rotated=128, batch=3),
        # prompts of odd total length, a long context behind them, half of each head rotated
        dict(name="qknorm_prompt", op="qknorm_prompt", dtype="bf16", heads=40, key_heads=8, dim=128, rotated=64, tokens=8209,
             requests=24),
        # a training step of them, forward and gradients
        dict(name="qknorm_train", op="qknorm_train", dtype="bf16", heads=16, key_heads=16, dim=128, rotated=128, batch=4,
             len=2048),
        # one request forked into four beams across 8 layers of convolution states
        dict(name="move_fork", op="move", dtype="bf16", layers=8, rows=64, dim=5120, states=3, moves=4, kind="fork"),
        # a full cache of scan states compacted, some rows freed
        dict(name="move_compact", op="move", dtype="f32", layers=2, rows=320, dim=5120, states=128, moves=160, kind="compact"),
    ]


def _log(rng, low, high):
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    n = min(high, max(low, n if rng.random() < 0.6 else n | 1))
    return n if n < 1024 or n % 1024 else n - 1  # the round sizes are among the listed cases


def draw(rng):
    op = rng.choice(["lattn_step", "lattn_prompt", "lattn_prompt", "lattn_train", "lattn_train", "qknorm_step",
                     "qknorm_prompt", "qknorm_train", "move"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op.startswith("lattn"):
        c["groups"] = rng.choice([1, 1, 2, 4])
        c["heads"] = c["groups"] * _log(rng, 1, 80 // c["groups"])
        c["value"] = rng.choice([64, 64, 64, 32, 128, 48, 17])
        c["key"] = rng.choice([128, 128, 64, 64, 16, 40, 33])
        if op == "lattn_step":
            c["batch"], c["padding"] = _log(rng, 1, 256), rng.randint(0, 8)
        elif op == "lattn_prompt":
            most = 5_000_000 if c["dtype"] == "bf16" else 1_500_000
            c["tokens"] = _log(rng, 1, max(1, min(16384, most // (c["heads"] * 64))))
            c["requests"] = _log(rng, 1, 64)
        else:
            c["heads"] = min(c["heads"], 16 * c["groups"])
            c["batch"] = rng.randint(1, 3)
            most = 3_000_000 if c["dtype"] == "bf16" else 1_000_000
            c["len"] = _log(rng, 1, max(1, min(1500, most // (c["batch"] * c["heads"] * 64))))
            c["steps"] = rng.random() < 0.7
    elif op.startswith("qknorm"):
        c["key_heads"] = _log(rng, 1, 16)
        c["heads"] = c["key_heads"] * rng.randint(1, 4)
        c["dim"] = rng.choice([128, 128, 64, 96, 256, 18])
        c["rotated"] = rng.choice([c["dim"], c["dim"], c["dim"] // 4 * 2, 0])
        if op == "qknorm_step":
            c["batch"] = _log(rng, 1, 256)
        elif op == "qknorm_prompt":
            c["tokens"], c["requests"] = _log(rng, 1, min(16384, 32_000_000 // (2 * c["heads"] * c["dim"]))), _log(rng, 1, 32)
        else:
            c["batch"] = rng.randint(1, 4)
            c["len"] = _log(rng, 1, min(4096, 16_000_000 // (2 * c["heads"] * c["dim"] * c["batch"])))
    else:
        c["kind"] = rng.choice(["fork", "compact"])
        c["layers"], c["rows"] = rng.randint(1, 4), _log(rng, 2, 320)
        c["dim"], c["states"] = _log(rng, 64, 5120), rng.choice([1, 2, 3, 7, 16, 64])
        c["moves"] = rng.randint(1, max(1, c["rows"] // 2))
    return c


def work(case):
    c, op, io = case, case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("lattn"):
        h, p, n, g = c["heads"], c["value"], c["key"], c["groups"]
        state = 4 * h * p * n
        if op == "lattn_step":
            b = c["batch"]
            kept = b - min(c["padding"], b - 1)
            return dict(bytes=io * b * (2 * h * p + 2 * g * n + h) + 2 * kept * state, flops=5 * b * h * p * n)
        if op == "lattn_prompt":
            t = c["tokens"]
            return dict(bytes=io * t * (2 * h * p + 2 * g * n + h) + 2 * c["requests"] * state, flops=t * h * p * n * 4)
        t = c["batch"] * c["len"]
        s = 1 if c["steps"] else 0
        # forward: q, k, v, the steps and o; gradients: q, k, v, do, the steps and dq, dk, dv, dsteps
        return dict(bytes=io * t * (h * p * (2 + 3) + g * n * (2 + 4) + 3 * s * h) + c["batch"] * state, flops=t * h * p * n * 16)
    if op.startswith("qknorm"):
        n = (c["heads"] + c["key_heads"]) * c["dim"]
        if op == "qknorm_train":
            t = c["batch"] * c["len"]
            return dict(bytes=io * 5 * t * n + 8 * t + 12 * c["dim"], flops=20 * t * n)
        t = c["batch"] if op == "qknorm_step" else c["tokens"]
        return dict(bytes=io * 2 * t * n + 4 * t + 8 * c["dim"], flops=7 * t * n)
    row = c["dim"] * c["states"] * io * c["layers"]
    return dict(bytes=2 * c["moves"] * row + 8 * c["moves"], flops=0)


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


def _moves(seed, c):
    """(from, to) of each move: a fork copies a few rows to free ones, a compaction closes gaps and frees what it leaves."""
    r = random.Random(seed + 2)
    rows, n = c["rows"], min(c["moves"], c["rows"])
    to = r.sample(range(rows), n)
    if c["kind"] == "fork":
        one = r.randrange(rows)
        return [one if r.random() < 0.75 else r.randrange(rows) for _ in to], to
    # rows move among themselves, in any order: some are read after another move has named them as its target
    return [-1 if r.random() < 0.125 else r.randrange(rows) for _ in to], to


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    io = DTYPES[c["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device=dev) * std + mean).to(dtype)

    def uniform(*shape, low=0.0, high=1.0):
        return torch.rand(shape, generator=g, device=dev) * (high - low) + low

    def table(values, dtype=torch.int32):
        return torch.tensor(values, dtype=dtype, device=dev)

    s = dict(case=dict(c), io=io)
    op = c["op"]
    if op.startswith("lattn"):
        h, p, n, gr = c["heads"], c["value"], c["key"], c["groups"]
        lead, tail = {"lattn_step": ((c.get("batch"),), ()), "lattn_prompt": ((), (c.get("tokens"),)),
                      "lattn_train": ((c.get("batch"),), (c.get("len"),))}[op]
        # v, k and q are parts of one projection
        both = normal(*lead, h * p + 2 * gr * n, *tail, dtype=io)
        at = len(lead)
        s["v"], s["k"], s["q"] = both.narrow(at, 0, h * p), both.narrow(at, h * p, gr * n), both.narrow(at, h * p + gr * n, gr * n)
        s["scale"] = n ** -0.5
        s["D"] = normal(h)
        s["delta"] = s["bias"] = s["s0"] = None
        if c.get("steps", True):
            # steps before the bias and softplus, and decays of many lengths, as trained layers have
            s["delta"] = normal(*lead, h, *tail, mean=-1.0, dtype=io)
            s["bias"] = normal(h, mean=-2.0)
            s["A"] = -uniform(h, low=1.0, high=16.0)
        else:
            s["A"] = torch.log1p(-torch.exp2(-3.0 - 5.0 * torch.arange(h, device=dev) / h))
        if op == "lattn_train":
            s["do"] = normal(*lead, h * p, *tail, dtype=io)
        elif op == "lattn_prompt":
            s["cu"] = table(_offsets(seed, c["tokens"], c["requests"]))
            slots, has, rows = _cache(seed, c["requests"], 0)
            s["slots"], s["has"] = table(slots), table(has, torch.bool)
            s["state"] = normal(rows, h * p, n, std=0.5)
        else:
            slots, _, rows = _cache(seed, c["batch"], c["padding"])
            s["slots"] = table(slots)
            s["state"] = normal(rows, h * p, n, std=0.5)
    elif op.startswith("qknorm"):
        d, nq, nk, r = c["dim"], c["heads"], c["key_heads"], c["rotated"]
        lead, tail = {"qknorm_step": ((c.get("batch"),), ()), "qknorm_prompt": ((), (c.get("tokens"),)),
                      "qknorm_train": ((c.get("batch"),), (c.get("len"),))}[op]
        both = normal(*lead, (nq + nk) * d, *tail, dtype=io)  # q and k are parts of one projection
        s["q"], s["k"] = both.narrow(len(lead), 0, nq * d), both.narrow(len(lead), nq * d, nk * d)
        s["qw"], s["kw"] = normal(d, std=0.1, mean=1.0), normal(d, std=0.1, mean=1.0)
        s["freq"] = 10000.0 ** (-torch.arange(0, r, 2, device=dev, dtype=torch.float32) / r) if r else None
        if op == "qknorm_step":  # requests at very different positions, some far into a long context
            s["pos"] = torch.exp(uniform(c["batch"], high=13.0)).int() if r else None
        elif op == "qknorm_prompt":
            cu = _offsets(seed, c["tokens"], c["requests"])
            rnd = random.Random(seed + 3)
            first = [int(math.exp(rnd.uniform(0, 13))) for _ in range(c["requests"])]
            pos = [first[i] + t for i in range(c["requests"]) for t in range(cu[i + 1] - cu[i])]
            s["pos"] = table(pos) if r else None
        else:
            s["pos"] = torch.arange(c["len"], device=dev, dtype=torch.int32).repeat(c["batch"], 1) if r else None
            s["do"] = normal(*both.shape, dtype=io)
            s["dq"], s["dk"] = (t.contiguous() for t in (s["do"].narrow(len(lead), 0, nq * d), s["do"].narrow(len(lead), nq * d, nk * d)))
    else:
        s["cache"] = normal(c["layers"], c["rows"], c["dim"], c["states"], dtype=io)
        src, dst = _moves(seed, c)
        s["src"], s["dst"] = table(src), table(dst)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import linear_recurrence_gb300 as lr

    c, op = s["case"], s["case"]["op"]
    if op.startswith("lattn"):
        options = dict(groups=c["groups"], scale=s["scale"], delta_bias=s["bias"], delta_softplus=s["delta"] is not None)
    if op == "lattn_step":
        o = lr.lattn_step(s["q"], s["k"], s["v"], s["A"], s["delta"], s["D"], state=s["state"], slots=s["slots"], **options)
        return dict(o=o, state=s["state"])
    if op == "lattn_prompt":
        o = lr.lattn_prompt(s["q"], s["k"], s["v"], s["A"], s["delta"], s["D"], cu_seqlens=s["cu"], state=s["state"],
                            slots=s["slots"], has_state=s["has"], **options)
        return dict(o=o, state=s["state"])
    if op == "lattn_train":
        o, last = lr.lattn_fwd(s["q"], s["k"], s["v"], s["A"], s["delta"], s["D"], **options)
        g = lr.lattn_bwd(s["q"], s["k"], s["v"], s["A"], s["delta"], s["D"], None, s["do"], **options)
        return dict(o=o, state=last, dq=g["dq"], dk=g["dk"], dv=g["dv"], ddelta=g["ddelta"], dA=g["dA"], dD=g["dD"],
                    dbias=g["ddelta_bias"])
    if op == "qknorm_step":
        q, k = lr.qknorm_step(s["q"], s["k"], s["qw"], s["kw"], s["pos"], s["freq"], eps=EPS)
        return dict(q=q, k=k)
    if op == "move":
        lr.state_move(s["cache"], s["src"], s["dst"], layers=True)
        return dict(cache=s["cache"])
    one = op == "qknorm_prompt"  # packed tokens are a batch of one
    q, k, pos = (t if t is None or not one else t[None] for t in (s["q"], s["k"], s["pos"]))
    qo, ko = lr.qknorm_fwd(q, k, s["qw"], s["kw"], pos, s["freq"], eps=EPS)
    if one:
        return dict(q=qo[0], k=ko[0])
    g = lr.qknorm_bwd(q, k, s["qw"], s["kw"], s["dq"], s["dk"], pos, s["freq"], eps=EPS)
    return dict(q=qo, k=ko, dq=g["dq"], dk=g["dk"], dqw=g["dq_weight"], dkw=g["dk_weight"])


def _run_plain(s):
    return globals()["_plain_" + s["case"]["op"]](s)


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


def _steps(s, shape, bias_shape):
    """The step of every head and token, in 64 bits: a sum of many of them is an exponent."""
    if s["delta"] is None:
        return torch.ones(shape, dtype=torch.float64, device=s["A"].device)
    x = s["delta"].double()
    return _softplus(x + s["bias"].double().view(bias_shape))


def _keep(cache, slots, new):
    """Write each request's new state to its cache row; padding requests have none."""
    n, k = cache.shape[0], slots.shape[0]
    of = torch.full((n + 1,), -1, dtype=torch.long, device=cache.device)
    of[torch.where(slots < 0, n, slots).long()] = torch.arange(k, device=cache.device)
    of = of[:n]
    cache.copy_(torch.where((of >= 0).view(n, 1, 1), new[of.clamp(min=0)], cache))


def _plain_lattn_step(s):
    c, slots = s["case"], s["slots"]
    b, h, p, n, g = slots.shape[0], c["heads"], c["value"], c["key"], c["groups"]
    dt = _steps(s, (b, h), (1, h)).float()
    q, k = (s[x].float().view(b, g, 1, 1, n).expand(b, g, h // g, 1, n).reshape(b, h, 1, n) for x in "qk")
    v = s["v"].float().view(b, h, p)
    first = torch.where((slots >= 0).view(-1, 1, 1), s["state"][slots.clamp(min=0).long()], 0.0).view(b, h, p, n)
    new = torch.exp(dt * s["A"])[:, :, None, None] * first + (dt[:, :, None] * v)[..., None] * k
    o = s["scale"] * (new * q).sum(-1) + s["D"][:, None] * v
    _keep(s["state"], slots, new.view(b, h * p, n))
    return dict(o=o.reshape(b, h * p).to(s["io"]), state=s["state"])


def _plain_lattn_prompt(s):
    """Pieces of C tokens: products inside a piece, the states between pieces by one product with the decays among them."""
    c, C = s["case"], 64
    h, p, n, g, t = c["heads"], c["value"], c["key"], c["groups"], c["tokens"]
    dev, cu = s["q"].device, s["cu"].long()
    m = -(-t // C)
    pad = m * C - t
    A = s["A"].double().view(h, 1, 1)

    def pieces(x, rows):  # [rows, t] -> [rows, m, C]
        return torch.nn.functional.pad(x, (0, pad)).view(*rows, m, C)

    dt = pieces(_steps(s, (h, t), (h, 1)), (h,))
    q, k, v = (pieces(s[x].float(), r) for x, r in (("q", (g, n)), ("k", (g, n)), ("v", (h, p))))
    of = torch.searchsorted(cu[1:], torch.arange(m * C, device=dev).clamp(max=t - 1), right=True).view(m, C)  # the request of each token
    run = dt.cumsum(-1)  # the steps of a piece up to each token
    low = torch.ones(C, C, dtype=torch.bool, device=dev).tril() & (of[:, :, None] == of[:, None, :])
    w = torch.where(low, torch.exp((A[..., None] * (run[..., :, None] - run[..., None, :])).float()) * dt.float()[..., None, :], 0.0)
    score = s["scale"] * torch.einsum("gnmt,gnms->gmts", q, k)
    score = (score[:, None] * w.view(g, h // g, m, C, C)).view(h, m, C, C)
    o = torch.einsum("hmts,hpms->hpmt", score, v)
    # what a piece adds to the state behind it: the tokens of its last request
    total = run[..., -1:]
    tail = torch.where(of == of[:, -1:], torch.exp((A * (total - run)).float()) * dt.float(), 0.0)
    kh = k.view(g, 1, n, m, C).expand(g, h // g, n, m, C).reshape(h, n, m, C)
    qh = q.view(g, 1, n, m, C).expand(g, h // g, n, m, C).reshape(h, n, m, C)
    add = torch.einsum("hpms,hnms->hmpn", v * tail[:, None], kh)
    # the initial state of request r enters as a piece of its own right before the request
    r = cu.shape[0] - 1
    first = torch.where(s["has"].view(r, 1, 1), s["state"][s["slots"].long()], 0.0).view(r, h, p, n).permute(1, 0, 2, 3)
    through = torch.cat([torch.zeros(h, 1, dtype=torch.float64, device=dev), (run[..., -1]).cumsum(-1)], 1)  # steps before each piece
    begin = torch.cat([(through[:, :m, None] + run - dt).view(h, m * C), through[:, m:]], 1)[:, cu[:-1]]  # steps before each request
    mine = of[:, 0]  # the request that a piece begins with; its tokens before the piece lie in pieces that end with it
    over = torch.where((of[None, :, -1] == mine[:, None]) & torch.ones(m, m, dtype=torch.bool, device=dev).tril(-1),
                       torch.exp((A * (through[:, :m, None] - through[:, None, 1:])).float()), 0.0)
    enter = torch.where((mine[:, None] == torch.arange(r, device=dev)) & (cu[:-1] <= C * torch.arange(m, device=dev)[:, None]),
                        torch.exp((A * (through[:, :m, None] - begin[:, None, :])).float()), 0.0)
    at = torch.bmm(over, add.reshape(h, m, p * n)) + torch.bmm(enter, first.reshape(h, r, p * n))
    into = torch.exp((A * run).float()) * (of == of[:, :1])
    o = o + s["scale"] * torch.einsum("hmpn,hnmt->hpmt", at.view(h, m, p, n), qh) * into[:, None]
    # requests that begin inside a piece bring their initial state to the rest of it
    bq = cu[:-1] // C
    inside = (cu[:-1] % C != 0) & (cu[1:] > cu[:-1])
    start = torch.where(inside, bq, 0).clamp(max=m - 1)
    since = through[:, start, None] + run[:, start] - begin[:, :, None]  # [h, r, C]
    lit = inside[:, None] & (of[start] == torch.arange(r, device=dev)[:, None])
    extra = s["scale"] * torch.einsum("hrpn,hnrt->hprt", first, qh[:, :, start]) * torch.where(lit, torch.exp((A * since).float()), 0.0)[:, None]
    o = o.index_add(2, start, extra).reshape(h, p, m * C)[..., :t]
    o = o + s["D"].view(h, 1, 1) * s["v"].float().view(h, p, t)
    # the state behind each request's last token: what entered its last piece, what that piece adds, or its own beginning
    last = ((cu[1:] - 1).clamp(min=0)) // C
    end = torch.gather(run, 1, last.view(1, r, 1).expand(h, r, C))
    end = torch.gather(end, 2, ((cu[1:] - 1).clamp(min=0) % C).view(1, r, 1).expand(h, r, 1))  # steps of that piece up to the request's end
    part = (of[last] == torch.arange(r, device=dev)[:, None]) & (torch.arange(C, device=dev) <= ((cu[1:] - 1).clamp(min=0) % C)[:, None])
    wt = torch.where(part, torch.exp((A * (end - run[:, last])).float()) * dt.float()[:, last], 0.0)
    new = torch.einsum("hprs,hnrs->hrpn", v[:, :, last] * wt[:, None], kh[:, :, last])
    crossed = (cu[:-1] <= C * last)[None, :, None]
    new = new + torch.where(crossed, torch.exp((A * end).float()), 0.0)[..., None] * at.view(h, m, p, n)[:, last]
    own_start = torch.exp((A * (through[:, last, None] + end - begin[:, :, None])).float())
    new = new + torch.where(crossed, 0.0, own_start)[..., None] * first
    new = torch.where((cu[1:] > cu[:-1]).view(1, r, 1, 1), new, first)
    _keep(s["state"], s["slots"], new.permute(1, 0, 2, 3).reshape(r, h * p, n))
    return dict(o=o.reshape(h * p, t).to(s["io"]), state=s["state"])


def _plain_lattn_train(s):
    """Every pair of tokens at once."""
    c = s["case"]
    b, h, p, n, g, t = c["batch"], c["heads"], c["value"], c["key"], c["groups"], c["len"]
    q, k = (s[x].float().view(b, g, n, t) for x in "qk")
    v, do = (s[x].float().view(b, h, p, t) for x in ("v", "do"))
    dt = _steps(s, (b, h, t), (1, h, 1))
    A, dtf, D = s["A"].double().view(h, 1, 1), dt.float(), s["D"].view(h, 1, 1)
    run = dt.cumsum(-1)
    low = torch.ones(t, t, dtype=torch.bool, device=q.device).tril()
    e = torch.where(low, torch.exp((A * (run[..., :, None] - run[..., None, :])).float()), 0.0)  # [b, h, t, s]
    qk = s["scale"] * torch.matmul(q.transpose(-1, -2), k)

    def heads(x):  # of a group -> of each head
        return x[:, :, None].expand(b, g, h // g, *x.shape[2:]).reshape(b, h, *x.shape[2:])

    f = e * heads(qk)  # scores without the step of their token
    o = torch.matmul(v, (f * dtf[..., None, :]).transpose(-1, -2)) + D * v
    last = torch.matmul(v * (torch.exp((A[None] * (run[..., -1:] - run).unsqueeze(2)).float()) * dtf[:, :, None, :]), heads(k).transpose(-1, -2))
    dp = torch.matmul(do.transpose(-1, -2), v)  # [b, h, t, s]
    dvw = torch.matmul(do, f)
    pair = f * dp
    de = s["scale"] * e * dp * dtf[..., None, :]
    de = de.view(b, g, h // g, t, t).sum(2)
    dq = torch.matmul(k, de.transpose(-1, -2))
    dk = torch.matmul(q, de)
    dtw = pair.sum(-2)  # of the step as the weight of its token
    off = (pair - torch.diag_embed(torch.diagonal(pair, dim1=-2, dim2=-1))).double() * dt[..., None, :]
    row, col = off.sum(-1), off.sum(-2)
    dg = (row - col).flip(-1).cumsum(-1).flip(-1)  # of the exponent that a token adds: all pairs around it
    ddt = A.squeeze(-1) * dg + dtw.double()
    out = dict(o=o.reshape(b, h * p, t).to(s["io"]), state=last.reshape(b, h * p, n), dq=dq.reshape(b, g * n, t).to(s["io"]),
               dk=dk.reshape(b, g * n, t).to(s["io"]), dv=(dvw * dtf[:, :, None, :] + D * do).reshape(b, h * p, t).to(s["io"]),
               dA=(dg * dt).sum((0, 2)).float(), dD=(do * v).double().sum((0, 2, 3)).float() if t else None)
    out["ddelta"] = out["dbias"] = None
    if s["delta"] is not None:
        x = s["delta"].double() + s["bias"].double().view(1, h, 1)
        ddt = ddt / (1 + torch.exp(-x))
        out["ddelta"], out["dbias"] = ddt.to(s["io"]), ddt.sum((0, 2)).float()
    return out


def _rotation(pos, freq):
    """cos and sin [.., rotated / 2]; the angles of far positions need 64 bits."""
    a = pos.double()[..., None] * freq.double()
    return torch.cos(a).float(), torch.sin(a).float()


def _plain_norm(x, w, cs):
    """x [.., heads, dim] of each token; returns the output and the normalised x."""
    xh = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return _turn(xh * w, cs, 1.0), xh


def _turn(y, cs, sign):
    if cs is None:
        return y
    c, sn = cs[0][..., None, :], sign * cs[1][..., None, :]
    r = c.shape[-1]
    a, b = y[..., :r], y[..., r:2 * r]
    return torch.cat([a * c - b * sn, b * c + a * sn, y[..., 2 * r:]], -1)


def _plain_qknorm_step(s):
    c = s["case"]
    cs = _rotation(s["pos"], s["freq"]) if s["freq"] is not None else None
    q, k = (_plain_norm(s[x].float().unflatten(-1, (-1, c["dim"])), s[w], cs)[0].flatten(-2).to(s["io"]) for x, w in (("q", "qw"), ("k", "kw")))
    return dict(q=q, k=k)


def _plain_qknorm_prompt(s):
    c = s["case"]
    cs = _rotation(s["pos"], s["freq"]) if s["freq"] is not None else None
    q, k = (_plain_norm(s[x].float().t().unflatten(-1, (-1, c["dim"])), s[w], cs)[0].flatten(-2).t().to(s["io"]) for x, w in (("q", "qw"), ("k", "kw")))
    return dict(q=q, k=k)


def _plain_qknorm_train(s):
    c, out = s["case"], {}
    cs = _rotation(s["pos"], s["freq"]) if s["freq"] is not None else None
    for x, w, dx, dw in (("q", "qw", "dq", "dqw"), ("k", "kw", "dk", "dkw")):
        v = s[x].float().transpose(1, 2).unflatten(-1, (-1, c["dim"]))
        y, xh = _plain_norm(v, s[w], cs)
        dy = _turn(s[dx].float().transpose(1, 2).unflatten(-1, (-1, c["dim"])), cs, -1.0)
        gx = dy * s[w]
        rstd = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
        grad = rstd * (gx - xh * (gx * xh).mean(-1, keepdim=True))
        out[x] = y.flatten(-2).transpose(1, 2).to(s["io"])
        out[dx] = grad.flatten(-2).transpose(1, 2).to(s["io"])
        out[dw] = (dy * xh).sum((0, 1, 2))
    return out


def _plain_move(s):
    cache, src, dst = s["cache"], s["src"].long(), s["dst"].long()
    taken = torch.where((src >= 0).view(1, -1, 1, 1), cache[:, src.clamp(min=0)], 0.0)
    cache.index_copy_(1, dst, taken)
    return dict(cache=cache)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    return globals()["_exact_" + case["op"]](case, f)


def _step64(f, x, h):
    """[.., heads] steps of one token, from its delta."""
    return torch.nn.functional.softplus(x + f["bias"], threshold=40) if x is not None else torch.ones(h, dtype=torch.float64, device=f["A"].device)


def _advance(f, case, state, q, k, v, dt):
    """One token of requests [r]: state [r, heads, value, key] in place, and its output [r, heads, value]."""
    g, n = case["groups"], case["key"]
    h = case["heads"]
    q, k = (x.reshape(-1, g, 1, n).expand(-1, g, h // g, n).reshape(-1, h, n) for x in (q, k))
    state.mul_(torch.exp(dt * f["A"])[..., None, None]).add_((dt[..., None] * v)[..., None] * k[:, :, None, :])
    return f["scale"] * torch.matmul(state, q[..., None])[..., 0] + f["D"][:, None] * v


def _exact_lattn_step(case, f):
    h, p, n, b = case["heads"], case["value"], case["key"], case["batch"]
    state = f["state"].clone()
    first = torch.zeros(b, h, p, n, dtype=torch.float64, device=state.device)
    slots = f["slots"].tolist()
    for i, row in enumerate(slots):
        if row >= 0:
            first[i] = state[row].view(h, p, n)
    o = _advance(f, case, first, f["q"], f["k"], f["v"].reshape(b, h, p), _step64(f, f["delta"], h))
    for i, row in enumerate(slots):
        if row >= 0:
            state[row] = first[i].view(h * p, n)
    return dict(o=o.reshape(b, h * p), state=state)


def _exact_lattn_prompt(case, f):
    h, p, n, t = case["heads"], case["value"], case["key"], case["tokens"]
    if t * h * p * n > 9e9:
        return None
    q, k, v = (f[x].t().contiguous() for x in "qkv")
    dt = _step64(f, f["delta"].t(), h).contiguous()
    state, o = f["state"].clone(), torch.empty(t, h, p, dtype=torch.float64, device=q.device)
    cu, slots, has = f["cu"].tolist(), f["slots"].tolist(), f["has"].tolist()
    for i, row in enumerate(slots):
        now = (state[row] if has[i] else torch.zeros_like(state[row])).view(1, h, p, n).clone()
        for j in range(cu[i], cu[i + 1]):
            o[j] = _advance(f, case, now, q[j], k[j], v[j].view(1, h, p), dt[j][None])[0]
        state[row] = now.view(h * p, n)
    return dict(o=o.view(t, h * p).t().contiguous(), state=state)


def _exact_lattn_train(case, f):
    b, h, p, n, g, t = case["batch"], case["heads"], case["value"], case["key"], case["groups"], case["len"]
    if b * t * h * p * n * 8 > 4e10:
        return None
    q, k = (f[x].permute(2, 0, 1).reshape(t, b, g, 1, n).expand(t, b, g, h // g, n).reshape(t, b, h, n) for x in "qk")
    v, do = (f[x].permute(2, 0, 1).reshape(t, b, h, p) for x in ("v", "do"))
    raw = f["delta"].permute(2, 0, 1) if f["delta"] is not None else None
    dt = _step64(f, raw, h).expand(t, b, h)
    a = torch.exp(dt * f["A"])
    states = torch.zeros(t + 1, b, h, p, n, dtype=torch.float64, device=q.device)
    o = torch.empty_like(v)
    for j in range(t):
        states[j + 1] = states[j]
        o[j] = _advance(f, case, states[j + 1], f["q"][..., j], f["k"][..., j], v[j], dt[j])
    ds = torch.zeros_like(states[0])
    dq, dk, dv, dg, dw = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(dt), torch.empty_like(dt)
    for j in reversed(range(t)):
        ds = ds + f["scale"] * do[j][..., None] * q[j][:, :, None, :]
        dq[j] = f["scale"] * torch.matmul(do[j][:, :, None, :], states[j + 1])[:, :, 0]
        into = torch.matmul(ds, k[j][..., None])[..., 0]
        dv[j] = dt[j][..., None] * into + f["D"][:, None] * do[j]
        dk[j] = dt[j][..., None] * torch.matmul(v[j][:, :, None, :], ds)[:, :, 0]
        dw[j] = (into * v[j]).sum(-1)
        ds = ds * a[j][..., None, None]
        dg[j] = (ds * states[j]).sum((-1, -2))

    def back(x):  # [t, b, heads, w] -> [b, heads * w, t]
        return x.reshape(t, b, -1).permute(1, 2, 0).contiguous()

    out = dict(o=back(o), state=states[t].reshape(b, h * p, n), dq=back(dq.view(t, b, g, h // g, n).sum(3)),
               dk=back(dk.view(t, b, g, h // g, n).sum(3)), dv=back(dv), dA=(dg * dt).sum((0, 1)), dD=(do * v).sum((0, 1, 3)))
    out["ddelta"] = out["dbias"] = None
    if raw is not None:
        ddt = (f["A"] * dg + dw) * torch.sigmoid(raw + f["bias"])
        out["ddelta"], out["dbias"] = back(ddt), ddt.sum((0, 1))
    return out


def _exact_head(f, x, w, width, pos):
    """x [.., heads * width] of tokens at pos: normalised and turned as complex numbers."""
    v = x.unflatten(-1, (-1, width))
    y = v / (v.square().sum(-1, keepdim=True) / width + EPS).sqrt() * w
    if f["freq"] is None:
        return y.flatten(-2)
    r = f["freq"].shape[0]
    angle = pos[..., None].double() * f["freq"]
    turned = torch.complex(y[..., :r].contiguous(), y[..., r:2 * r].contiguous()) * torch.polar(torch.ones_like(angle), angle)[..., None, :]
    return torch.cat([turned.real, turned.imag, y[..., 2 * r:]], -1).flatten(-2)


def _exact_qknorm_step(case, f):
    return dict(q=_exact_head(f, f["q"], f["qw"], case["dim"], f["pos"]), k=_exact_head(f, f["k"], f["kw"], case["dim"], f["pos"]))


def _exact_qknorm_prompt(case, f):
    return dict(q=_exact_head(f, f["q"].t(), f["qw"], case["dim"], f["pos"]).t(), k=_exact_head(f, f["k"].t(), f["kw"], case["dim"], f["pos"]).t())


def _exact_qknorm_train(case, f):
    out = {}
    for x, w, dx, dw in (("q", "qw", "dq", "dqw"), ("k", "kw", "dk", "dkw")):
        a, b = f[x].detach().clone().requires_grad_(), f[w].detach().clone().requires_grad_()
        y = _exact_head(f, a.transpose(1, 2), b, case["dim"], f["pos"]).transpose(1, 2)
        out[dx], out[dw] = torch.autograd.grad(y, (a, b), f[dx])
        out[x] = y.detach()
    return out


def _exact_move(case, f):
    cache = f["cache"].clone()
    for a, b in zip(f["src"].tolist(), f["dst"].tolist()):
        cache[:, b] = f["cache"][:, a] if a >= 0 else 0
    return dict(cache=cache)
