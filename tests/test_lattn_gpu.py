"""Linear attention with a decay for each head against its definition in 64 bits.

Tolerances count roundings.  A sum of K terms in fp32 is off by at most K * 2^-24 of
its terms' magnitudes; a chain of products over N key channels and a chunk of 128
tokens by their number of terms; an exponent x in fp32 by 4 * 2^-24 * |x| of its
factor (its sum, product and rounding), the exponent unit adds 2^-22, the steps' softplus
2^-20 of a step, and so of an exponent.  bf16 outputs are rounded once (2^-8), and in
bf16 the products inside a chunk take scores, weights and states rounded to bf16 on one side
(2^-8 of their magnitudes)."""
import pytest
import torch

import lattn_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


def make(seed, dtype, batch, heads, groups, value, key, L, *, delta=True, options=True, D=True, s0=True, packed=False, offset=0):
    """Inputs as views of one projection; offset shifts their first token off a 16-byte boundary."""
    g = torch.Generator().manual_seed(seed)
    io = DT[dtype]
    wide = torch.randn(batch, heads * value + 2 * groups * key + heads, L + offset, generator=g).to(io)
    wide = wide.cuda()[..., offset:]
    hp, gn = heads * value, groups * key
    v, k, q = wide[:, :hp], wide[:, hp:hp + gn], wide[:, hp + gn:hp + 2 * gn]
    f = dict(v=v, k=k, q=q, delta=None, bias=None, D=None, s0=None)
    if delta:
        d = wide[:, hp + 2 * gn:]
        if options:
            f["delta"], f["bias"] = d, (torch.randn(heads, generator=g) - 2.0).cuda()
        else:
            f["delta"] = torch.nn.functional.softplus(d.float() - 2.5).to(io)
        f["A"] = -(torch.rand(heads, generator=g) * 15 + 1).cuda()
    else:
        f["A"] = -torch.exp2(-1.0 - 6.0 * torch.arange(heads) / heads).cuda()
    if D:
        f["D"] = torch.randn(heads, generator=g).cuda()
    if s0:
        f["s0"] = torch.randn(batch, hp, key, generator=g).cuda()
    if packed:
        for x in ("q", "k", "v", "delta"):
            f[x] = None if f[x] is None else f[x][0]
    f["act"] = f["delta"] is not None and options
    return f


def coarse(dtype):
    """What products on one side rounded to the I/O type add, of the magnitudes."""
    return 2.0 ** -8 if dtype == "bf16" else 0.0


def fine(f, key, L):
    """Roundings in fp32, of the magnitudes: two chained sums, exponents and steps."""
    A, delta, bias = ref.d64(f["A"]), ref.d64(f["delta"]), ref.d64(f["bias"])
    dt = ref.steps(delta, bias, f["act"], (A.shape[0], L))
    x = ref.largest_exponent(A, dt)
    return 2.0 ** -24 * (key + 128 + 64 + 8 * x) + 2.0 ** -20 * (1 + min(x, 20.0)) + 2.0 ** -21


def near(got, want, mag, rel, what):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, what
    off = (got - want).abs()
    bound = rel[0] * want.abs() + rel[1] * mag + 1e-30
    worst = float((off / bound).max()) if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of what its roundings allow"


SHAPES = [  # heads, groups, value, key
    (4, 1, 64, 128), (2, 2, 64, 64), (3, 1, 17, 33), (2, 1, 128, 16), (4, 2, 48, 40), (1, 1, 1, 1), (2, 1, 200, 128), (8, 8, 64, 128)]
LENGTHS = [1, 2, 17, 63, 64, 65, 127, 128, 129, 200, 259]


def run_fwd(lr, f, dtype, groups, scale, **kw):
    return lr.lattn_fwd(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], f["s0"], groups=groups, scale=scale,
                        delta_bias=f["bias"], delta_softplus=f["act"], **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", LENGTHS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(lr, dtype, L, shape):
    heads, groups, value, key = shape
    n = LENGTHS.index(L) + SHAPES.index(shape)
    f = make(n, dtype, 2, heads, groups, value, key, L, delta=n % 3 != 0, options=n % 2 == 0, D=n % 4 != 0, s0=n % 5 != 0, offset=n % 4)
    scale = key ** -0.5
    o, s = run_fwd(lr, f, dtype, groups, scale)
    assert lr.get_last_error() == lr.SSCAN_OK
    want = ref.forward(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], f["s0"], groups, scale, f["bias"], f["act"])
    c = fine(f, key, L)
    near(o, want[0], want[2], (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24, c + coarse(dtype)), "o")
    # states are held in fp32 whatever the I/O type; the product that adds a chunk keeps 24 bits of its weights
    near(s, want[1], want[3], (2.0 ** -24, c), "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pieces", [1, 2, 3, 7])
def test_pieces(lr, dtype, pieces):
    f = make(pieces, dtype, 1, 2, 1, 64, 64, 901, s0=True)
    o, s = run_fwd(lr, f, dtype, 1, 0.125, pieces=pieces)
    want = ref.forward(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], f["s0"], 1, 0.125, f["bias"], f["act"])
    c = fine(f, 64, 901)
    near(o, want[0], want[2], (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24, c + coarse(dtype)), "o")
    near(s, want[1], want[3], (2.0 ** -24, c), "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pieces", [0, 40, 60])
def test_many_parts(lr, dtype, pieces):
    """One head over a long sequence: its state passes through all parts that time is cut into."""
    f = make(pieces, dtype, 1, 1, 1, 33, 24, 7777, delta=False)
    f["A"] = torch.tensor([-0.002], device="cuda")
    o, s = run_fwd(lr, f, dtype, 1, 0.2, pieces=pieces)
    assert int(lr.last_plan().split("=")[1]) > 30  # (61 chunks of 128 tokens are 31 parts of two)
    want = ref.forward(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], f["s0"], 1, 0.2)
    c = fine(f, 24, 7777) + 2.0 ** -24 * 122  # and a join a part
    near(o, want[0], want[2], (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24, c + coarse(dtype)), "o")
    near(s, want[1], want[3], (2.0 ** -24, c), "state")
    do = f["v"].contiguous()
    got = lr.lattn_bwd(f["q"], f["k"], f["v"], f["A"], None, f["D"], f["s0"], do, groups=1, scale=0.2)
    short = lr.lattn_bwd(f["q"][..., -700:], f["k"][..., -700:], f["v"][..., -700:], f["A"], None, f["D"],
                         run_fwd(lr, dict(f, **{x: f[x][..., :-700] for x in "qkv"}), dtype, 1, 0.2)[1], do[..., -700:].contiguous(), groups=1, scale=0.2)
    for name in ("dq", "dk", "dv"):  # the last tokens' gradients from the state before them
        off = (got[name][..., -700:].double() - short[name].double()).norm() / short[name].double().norm()
        # (each is rounded from sums whose factors have 8 bits in bf16: 2^-9 each on the average, of two factors and the result)
        assert float(off) < (2.0 ** -7 if dtype == "bf16" else 1e-5), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_growth_and_negative_steps(lr, dtype):
    """Rates above zero and negative steps are followed like any other: nothing is cut off."""
    f = make(3, dtype, 1, 2, 1, 64, 64, 300, options=False)
    f["A"] = torch.tensor([0.05, -0.02], device="cuda")
    f["delta"] = (f["delta"].float() - 0.08).to(DT[dtype])
    o, s = run_fwd(lr, f, dtype, 1, 0.125, pieces=2)
    want = ref.forward(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], f["s0"], 1, 0.125)
    c = fine(f, 64, 300)
    near(o, want[0], want[2], (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24, c + coarse(dtype)), "o")
    near(s, want[1], want[3], (2.0 ** -24, c), "state")


def test_instant_decay(lr):
    """Steps so long that nothing of a state is left: o_t = scale dt_t (q.k) v_t + D v_t."""
    f = make(4, "bf16", 1, 2, 1, 64, 64, 200, options=False)
    f["delta"] = torch.full_like(f["delta"], 30.0)
    f["A"] = torch.tensor([-16.0, -40.0], device="cuda")
    o, s = run_fwd(lr, f, "bf16", 1, 0.125)
    want = ref.forward(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], f["s0"], 1, 0.125)
    c = 2.0 ** -24 * 300 + 2.0 ** -20
    near(o, want[0], want[2], (2.0 ** -8, c + 2.0 ** -8), "o")
    near(s, want[1], want[3], (2.0 ** -24, c), "state")


def offsets(kind, tokens, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        return [0, tokens]
    if kind == "gaps":  # tokens before the first request and behind the last
        a, b = tokens // 5, tokens - tokens // 7
        return [a, (a + b) // 2, b]
    if kind == "short":
        cuts = sorted(torch.randint(0, tokens + 1, (tokens // 3,), generator=g).tolist())
        return [0] + cuts + [tokens]
    cuts = sorted(torch.randint(0, tokens + 1, (6,), generator=g).tolist())
    return [0] + cuts[:3] + [cuts[3]] * 3 + cuts[3:] + [tokens]  # some requests empty


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["one", "gaps", "short", "mixed"])
@pytest.mark.parametrize("tokens,pieces", [(1, 0), (5, 0), (64, 1), (131, 1), (131, 0), (333, 3), (1001, 0), (1024, 5)])
def test_prompt(lr, dtype, kind, tokens, pieces):
    heads, groups, value, key = [(4, 1, 64, 128), (2, 2, 33, 20), (2, 1, 128, 64)][tokens % 3]
    f = make(tokens + pieces, dtype, 1, heads, groups, value, key, tokens, packed=True, s0=False, offset=tokens % 2)
    cu = offsets(kind, tokens, tokens)
    n = len(cu) - 1
    g = torch.Generator().manual_seed(7)
    rows = n + 3
    slots = torch.randperm(rows, generator=g)[:n].tolist()
    if n > 2:
        slots[1] = -1
    has = (torch.rand(n, generator=g) < 0.6).tolist()
    state = torch.randn(rows, heads * value, key, generator=g)
    state[[i for i in range(rows) if i not in slots]] = float("nan")  # rows of nobody stay as they are
    dev = state.cuda()
    o = lr.lattn_prompt(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                        state=dev, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"),
                        has_state=torch.tensor(has, device="cuda"), groups=groups, scale=0.1, delta_bias=f["bias"],
                        delta_softplus=f["act"], pieces=pieces)
    assert lr.get_last_error() == lr.SSCAN_OK
    want = ref.packed(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], cu, slots, has, state, groups, 0.1, f["bias"], f["act"])
    c = fine(f, key, tokens)
    near(o, want[0], want[2], (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24, c + coarse(dtype)), "o")
    mine = [r for r in slots if r >= 0]
    near(dev.cpu()[mine], want[1][mine], want[3][mine], (2.0 ** -24, c), "state")
    other = [i for i in range(rows) if i not in mine]
    assert torch.equal(dev.cpu()[other].view(torch.int32), state[other].view(torch.int32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 1, 64, 128), (3, 3, 5, 7), (2, 2, 256, 128), (4, 1, 33, 16), (1, 1, 40, 30), (2, 1, 64, 64)], ids=str)
@pytest.mark.parametrize("pieces", [0, 3])
def test_short_requests(lr, dtype, shape, pieces):
    """Requests of 1 to 17 tokens between long ones, empty ones, tokens of nobody: each by its own way."""
    heads, groups, value, key = shape
    sizes = [16, 17, 1, 0, 15, 200, 16, 16, 2, 0, 0, 33, 1, 1, 130] + [3] * 40 + [0, 18, 9]
    cu = [3]
    for x in sizes:
        cu.append(cu[-1] + x)
    tokens, n = cu[-1] + 5, len(sizes)
    assert 0 < tokens <= 128 * n
    f = make(value, dtype, 1, heads, groups, value, key, tokens, packed=True, s0=False, offset=value % 2)
    g = torch.Generator().manual_seed(value)
    slots = torch.randperm(n + 2, generator=g)[:n].tolist()
    slots[4] = slots[7] = slots[11] = -1
    has = (torch.rand(n, generator=g) < 0.5).tolist()
    state = torch.randn(n + 2, heads * value, key, generator=g)
    for i in range(n):  # what a row held before a request that does not continue is not read
        if slots[i] >= 0 and not has[i]:
            state[slots[i]] = float("nan")
    dev = state.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    o = lr.lattn_prompt(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], cu_seqlens=torch.tensor(cu, **i32), state=dev,
                        slots=torch.tensor(slots, **i32), has_state=torch.tensor(has, device="cuda"), groups=groups, scale=0.1,
                        delta_bias=f["bias"], delta_softplus=f["act"], pieces=pieces)
    assert lr.get_last_error() == lr.SSCAN_OK
    want = ref.packed(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], cu, slots, has, state, groups, 0.1, f["bias"], f["act"])
    c = fine(f, key, tokens)
    inside = slice(cu[0], cu[-1])
    near(o[:, inside], want[0][:, inside], want[2][:, inside], (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24, c + coarse(dtype)), "o")
    mine = [r for r in slots if r >= 0]
    near(dev.cpu()[mine], want[1][mine], want[3][mine], (2.0 ** -24, c), "state")
    other = [i for i in range(n + 2) if i not in mine]
    assert torch.equal(dev.cpu()[other].view(torch.int32), state[other].view(torch.int32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("sizes", [[40, 70, 33, 150, 9], [5, 12, 3, 70, 9, 1, 1]], ids=["long", "short"])
def test_requests_are_apart(lr, dtype, bad, sizes):
    """What one request holds reaches no other: the others' bits stay."""
    heads, value, key = 2, 64, 128
    cu = torch.tensor([0] + sizes, dtype=torch.int32).cumsum(0).int()
    tokens = int(cu[-1])
    f = make(5, dtype, 1, heads, 1, value, key, tokens, packed=True, s0=False)
    s0 = torch.randn(len(sizes), heads * value, key, generator=torch.Generator().manual_seed(1)).cuda()

    def run(x):
        state = s0.clone()
        o = lr.lattn_prompt(x["q"], x["k"], x["v"], x["A"], x["delta"], x["D"], cu_seqlens=cu.cuda(), state=state, scale=0.1,
                            delta_bias=x["bias"], delta_softplus=True, pieces=2)
        return o, state

    want = run(f)
    for r in range(len(sizes)):
        a, b = int(cu[r]), int(cu[r + 1])
        x = dict(f)
        for name in ("q", "k", "v", "delta"):
            x[name] = f[name].clone()
            x[name][:, a:b] = bad
        got = run(x)
        keep = [i for i in range(len(sizes)) if i != r]
        assert torch.equal(got[1][keep], want[1][keep])
        assert torch.equal(got[0][:, :a], want[0][:, :a]) and torch.equal(got[0][:, b:], want[0][:, b:])
        assert not got[0][:, a].isfinite().any()  # (positive infinities alone add up to one)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES + [(3, 3, 64, 12), (80, 1, 64, 128)], ids=str)
@pytest.mark.parametrize("batch", [1, 5])
def test_step(lr, dtype, shape, batch):
    heads, groups, value, key = shape
    f = make(batch + heads, dtype, batch, heads, groups, value, key, 3, s0=False, D=batch > 1)
    one = {x: None if f[x] is None else f[x].transpose(1, 2).contiguous()[:, 1] for x in ("q", "k", "v", "delta")}  # rows of a strided view
    rows = batch + 2
    g = torch.Generator().manual_seed(9)
    state = torch.randn(rows, heads * value, key, generator=g)
    slots = torch.randperm(rows, generator=g)[:batch].tolist()
    if batch > 2:
        slots[2] = -1
    dev = state.cuda()
    o = lr.lattn_step(one["q"], one["k"], one["v"], f["A"], one["delta"], f["D"], state=dev,
                      slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), groups=groups, scale=0.3, delta_bias=f["bias"],
                      delta_softplus=f["act"])
    assert lr.get_last_error() == lr.SSCAN_OK
    first = torch.stack([state[r] if r >= 0 else torch.zeros_like(state[0]) for r in slots])
    cut = [x if x is None else x[..., None] for x in (one["q"], one["k"], one["v"], one["delta"])]
    want = ref.forward(*cut[:3], f["A"], cut[3], f["D"], first, groups, 0.3, f["bias"], f["act"])
    c = fine(f, key, 3)
    near(o, want[0][..., 0], want[2][..., 0], (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24, c), "o")
    for i, r in enumerate(slots):
        if r >= 0:
            near(dev[r], want[1][i], want[3][i], (2.0 ** -24, c), "state")
    other = [i for i in range(rows) if i not in slots]
    assert torch.equal(dev.cpu()[other], state[other])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 63, 64, 65, 128, 129, 200, 259])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(lr, dtype, L, shape):
    heads, groups, value, key = shape
    n = LENGTHS.index(L) + SHAPES.index(shape) if L in LENGTHS else SHAPES.index(shape)
    f = make(n + 50, dtype, 2, heads, groups, value, key, L, delta=n % 3 != 0, options=n % 2 == 0, D=n % 4 != 0, s0=n % 5 != 0, offset=n % 4)
    g = torch.Generator().manual_seed(n)
    do = torch.randn(2, heads * value, L, generator=g).to(DT[dtype]).cuda()
    ds = torch.randn(2, heads * value, key, generator=g).cuda() if n % 2 else None
    scale = key ** -0.5
    got = lr.lattn_bwd(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], f["s0"], do, ds, groups=groups, scale=scale,
                       delta_bias=f["bias"], delta_softplus=f["act"])
    assert lr.get_last_error() == lr.SSCAN_OK
    want, mag = ref.backward(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], f["s0"], do, ds, groups, scale, f["bias"], f["act"])
    check_gradients(f, got, want, mag, dtype, key, value, L, heads)


def chunk_sums(x, chunk=128):
    """[.., L] -> for each token the sum over the 2 * chunk - 1 around it: those of any chunk that holds it."""
    flat = torch.nn.functional.pad(x.reshape(-1, 1, x.shape[-1]), (chunk - 1, chunk - 1))
    return (torch.nn.functional.avg_pool1d(flat, 2 * chunk - 1, 1) * (2 * chunk - 1)).reshape(x.shape)


def check_gradients(f, got, want, mag, dtype, key, value, L, heads):
    io = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    # sums over value channels join those over keys and tokens; heads are added up for dq and dk
    c = fine(f, key, L) + 2.0 ** -24 * (value + heads)
    # in bf16 two factors beside the inputs may be rounded to it (a weight and a state): two half steps
    two = 2 * coarse(dtype)
    for name in ("dq", "dk", "dv"):
        near(got[name], want[name], mag[name], (io, c + two), name)
    if "ds0" in want:
        near(got["ds0"], want["ds0"], mag["ds0"], (2.0 ** -24, c), "ds0")
    # the exponents' gradients are sums over a chunk of row sums less column sums, each as large as all
    # of the chunk's pairs; in bf16 the states come in two terms of bf16 (2^-16)
    two_terms = 2.0 ** -16 if dtype == "bf16" else 0.0
    mg = chunk_sums(mag["dg"])
    cg = 2 * c + two_terms
    A = ref.d64(f["A"]).abs()
    dt = ref.steps(ref.d64(f["delta"]), ref.d64(f["bias"]), f["act"], (f["v"].shape[0], heads, L)).abs()
    near(got["dA"], want["dA"], (mg * dt).sum((0, 2)), (2.0 ** -24, cg + 2.0 ** -24 * 64), "dA")
    if "dD" in want:
        near(got["dD"], want["dD"], mag["dD"], (2.0 ** -24, 2.0 ** -24 * (value + 256)), "dD")
    if f["delta"] is None:
        assert got["ddelta"] is None and got["ddelta_bias"] is None
        return
    size = A[:, None] * mg + mag["dw"]
    near(got["ddelta"], want["ddelta"], size, (io, cg + 2.0 ** -20), "ddelta")
    if f["bias"] is not None:
        near(got["ddelta_bias"], want["ddelta_bias"], size.sum((0, 2)), (2.0 ** -24, cg + 2.0 ** -20), "ddelta_bias")
    else:
        assert got["ddelta_bias"] is None


def test_gradients_against_differences(lr):
    """Central differences of the kernels' own forward pass in fp32."""
    f = make(11, "f32", 1, 2, 1, 24, 16, 70)
    g = torch.Generator().manual_seed(1)
    do = torch.randn(1, 48, 70, generator=g).cuda()
    ds = torch.randn(1, 48, 16, generator=g).cuda()
    f = {k: v.contiguous() if torch.is_tensor(v) else v for k, v in f.items()}

    def loss():
        o, s = run_fwd(lr, f, "f32", 1, 0.25)
        return float((o.double() * do.double()).sum() + (s.double() * ds.double()).sum())

    got = lr.lattn_bwd(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], f["s0"], do, ds, groups=1, scale=0.25,
                       delta_bias=f["bias"], delta_softplus=True)
    pairs = dict(q="dq", k="dk", v="dv", A="dA", delta="ddelta", D="dD", s0="ds0", bias="ddelta_bias")
    for name, grad in pairs.items():
        x = f[name]
        d = torch.randn(x.shape, generator=g).cuda()
        keep = x.clone()
        h = 2.0 ** -9
        f[name] = keep + h * d
        up = loss()
        f[name] = keep - h * d
        down = loss()
        f[name] = keep
        want = float((got[grad].double() * d.double()).sum())
        # differences: h^2 of a third derivative, and the forward's fp32 errors over h
        scale = float((got[grad].double().abs() * d.double().abs()).sum())
        assert abs((up - down) / (2 * h) - want) <= 2e-3 * scale + 1e-3, name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rate,bias", [(-16.0, 0.0), (-16.0, 2.0), (-4.0, 1.0), (-1.0, -2.0), (0.0, 0.0)])
def test_rates_gradient_of_fast_decays(lr, dtype, rate, bias):
    """dA where only neighbours count: its terms are W (T_t - T_s) with W off by 2^-21 (its sums of 64 products,
    the exponential) and 2^-16 where a kept state in two bf16 terms is a factor (bf16), against their magnitudes."""
    f = make(17, dtype, 1, 4, 1, 64, 32, 400, D=False, s0=False)
    f["A"] = torch.full((4,), rate, device="cuda")
    f["bias"] = torch.full((4,), bias, device="cuda")
    do = torch.randn(1, 256, 400, generator=torch.Generator().manual_seed(2)).to(DT[dtype]).cuda()
    got = lr.lattn_bwd(f["q"], f["k"], f["v"], f["A"], f["delta"], None, None, do, groups=1, scale=0.2, delta_bias=f["bias"], delta_softplus=True)
    want, _ = ref.backward(f["q"], f["k"], f["v"], f["A"], f["delta"], None, None, do, None, 1, 0.2, f["bias"], True)
    size = want["dA"].norm()
    assert float((got["dA"].double().cpu() - want["dA"]).norm() / size) <= (2.0 ** -16 if dtype == "bf16" else 2.0 ** -18)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_queries_and_repeatable(lr, dtype):
    """Twelve heads over one set of queries and keys, few chunks: parts of the sums are joined in a fixed order."""
    f = make(12, dtype, 1, 12, 1, 64, 64, 130)
    do = torch.randn(1, 12 * 64, 130, generator=torch.Generator().manual_seed(5)).to(DT[dtype]).cuda()
    run = lambda: lr.lattn_bwd(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], f["s0"], do, groups=1, scale=0.2,  # noqa: E731
                               delta_bias=f["bias"], delta_softplus=f["act"])
    got, again = run(), run()
    for name in got:
        if got[name] is not None:
            assert torch.equal(got[name], again[name]), name
    want, mag = ref.backward(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], f["s0"], do, None, 1, 0.2, f["bias"], f["act"])
    check_gradients(f, got, want, mag, dtype, 64, 64, 130, 12)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_then_steps(lr, dtype):
    """A prompt in two parts and then single tokens: the same as the whole sequence at once."""
    heads, value, key, total = 4, 64, 128, 150
    f = make(21, dtype, 1, heads, 1, value, key, total, packed=True, s0=False)
    state = torch.zeros(2, heads * value, key, device="cuda")
    slot = torch.tensor([1], dtype=torch.int32, device="cuda")
    args = dict(groups=1, scale=0.1, delta_bias=f["bias"], delta_softplus=True)
    parts = []
    for a, b, cont in ((0, 90, False), (90, 140, True)):
        cut = [f[x][:, a:b] for x in ("q", "k", "v")] + [f["A"], f["delta"][:, a:b], f["D"]]
        parts.append(lr.lattn_prompt(*cut, cu_seqlens=torch.tensor([0, b - a], dtype=torch.int32, device="cuda"), state=state,
                                     slots=slot, has_state=torch.tensor([cont], device="cuda"), **args))
    for t in range(140, total):
        cut = [f[x][:, t][None].contiguous() for x in ("q", "k", "v")] + [f["A"], f["delta"][:, t][None].contiguous(), f["D"]]
        parts.append(lr.lattn_step(*cut, state=state, slots=slot, **args).t())
    want = ref.forward(f["q"][None], f["k"][None], f["v"][None], f["A"], f["delta"][None], f["D"], None, 1, 0.1, f["bias"], True)
    c = fine(f, key, total) * 2
    near(torch.cat(parts, 1), want[0][0], want[2][0], (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24, c + coarse(dtype)), "o")
    near(state[1], want[1][0], want[3][0], (2.0 ** -24, c), "state")
    assert not state[0].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_tables_are_reported(lr, dtype):
    f = make(31, dtype, 1, 2, 1, 64, 64, 100, packed=True, s0=False)
    state = torch.zeros(2, 128, 64, device="cuda")
    for cu, slots in (([0, 50, 400], [0, 1]), ([0, 60, 30], [0, 1]), ([-5, 50, 100], [0, 1]), ([0, 50, 100], [0, 2])):
        lr.lattn_prompt(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                        state=state, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), delta_bias=f["bias"], delta_softplus=True)
        assert lr.get_last_error() == lr.SSCAN_ERR_INVALID
        assert lr.get_last_error() == lr.SSCAN_OK


def test_empty(lr):
    f = make(1, "bf16", 2, 2, 1, 64, 64, 0)
    o, s = run_fwd(lr, f, "bf16", 1, 1.0)
    assert o.shape == (2, 128, 0) and torch.equal(s, f["s0"])
    f["s0"] = None
    assert not run_fwd(lr, f, "bf16", 1, 1.0)[1].any()
    got = lr.lattn_bwd(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], f["s0"], f["v"].contiguous(), groups=1, delta_bias=f["bias"], delta_softplus=True)
    assert not got["dA"].any() and not got["dD"].any() and not got["ddelta_bias"].any()
    state = torch.ones(3, 128, 64, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    p = make(1, "bf16", 1, 2, 1, 64, 64, 0, packed=True)
    lr.lattn_prompt(p["q"], p["k"], p["v"], p["A"], p["delta"], p["D"], cu_seqlens=torch.tensor([0, 0, 0], **i32), state=state,
                    slots=torch.tensor([0, 2], **i32), has_state=torch.tensor([True, False], device="cuda"), delta_bias=p["bias"])
    assert state[0].all() and state[1].all() and not state[2].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_graph_and_streams(lr, dtype):
    """Two captured graphs and two streams: each call has its own workspace."""
    fs = [make(40 + i, dtype, 1, 2, 1, 64, 64, 700) for i in range(2)]
    dos = [torch.randn(1, 128, 700, device="cuda").to(DT[dtype]) for _ in range(2)]

    def both(i):
        f = fs[i]
        o, s = run_fwd(lr, f, dtype, 1, 0.125, pieces=3)
        g = lr.lattn_bwd(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], f["s0"], dos[i], groups=1, scale=0.125,
                         delta_bias=f["bias"], delta_softplus=True)
        return [o, s] + [x for x in g.values() if x is not None]

    want = [both(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for i, st in enumerate(streams):
        with torch.cuda.stream(st):
            got[i] = both(i)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = both(i)
        graphs.append((g, outs))
    for _ in range(2):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                graphs[i][0].replay()
    torch.cuda.synchronize()
    for i in range(2):
        for a, b, c in zip(want[i], got[i], graphs[i][1]):
            assert torch.equal(a, b) and torch.equal(a, c)
