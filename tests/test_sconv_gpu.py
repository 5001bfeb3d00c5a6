"""GPU parity of the short causal convolution with its 64-bit form.

Tolerances.  c is a sum of W products and a bias in fp32: at most W + 1
roundings of 2^-24 of the terms' magnitudes m, and silu has a derivative
below 1.1 and a few roundings of its own: |err| <= 8 * 2^-24 * (m + |y|) is
taken twice over, 1e-6 * (m + |y|) + 1e-7.  bf16 outputs add their rounding,
2^-8 |y| (half an ulp is 2^-9).  States are copies: exact.  Gradient sums over
n terms: pairwise in lanes and warps, sequential over at most a few hundred
per lane: 1e-5 of the sum of magnitudes."""
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


def _near(got, want, size, dtype, k=1e-6):
    got = got.double().cpu()
    tol = k * (size + want.abs()) + 1e-7
    if dtype == "bf16":
        tol = tol + want.abs() * 2.0 ** -8
    bad = (got - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / tol).max()))
    assert torch.isfinite(got).all()


def _params(g, dim, width, bias=True):
    w = torch.randn(dim, width, generator=g)
    return w, torch.randn(dim, generator=g) if bias else None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,dim,L,width", [
    (1, 1, 1, 4), (2, 3, 2, 4), (1, 5, 3, 3), (3, 4, 8, 2), (2, 9, 255, 4), (1, 17, 256, 3), (2, 8, 257, 4),
    (1, 33, 1000, 2), (4, 16, 520, 4)])
@pytest.mark.parametrize("form", ["plain", "view", "state"])
def test_forward(lr, dtype, batch, dim, L, width, form):
    g = torch.Generator().manual_seed(L * 7 + width)
    x = torch.randn(batch, 2 * dim, L, generator=g).to(IO[dtype]).cuda()
    x = x[:, dim:] if form == "view" else x[:, :dim].contiguous()
    w, b = _params(g, dim, width, bias=form != "view")
    x0 = torch.randn(batch, dim, width - 1, generator=g).to(IO[dtype]) if form == "state" else None
    act = form != "view"
    y, last = lr.sconv_fwd(x, w.cuda(), None if b is None else b.cuda(), None if x0 is None else x0.cuda(), silu=act)
    assert lr.get_last_error() == 0 and lr.last_launch_count() == 1
    before = torch.zeros(batch, dim, width - 1, dtype=torch.float64) if x0 is None else ref.d64(x0)
    yr, lastr, size = ref.conv(ref.d64(x), ref.d64(w), ref.d64(b), before, act)
    assert y.dtype == IO[dtype] and y.is_contiguous()
    _near(y, yr, size, dtype)
    assert torch.equal(last.double().cpu(), lastr)


def test_forward_misaligned_base_and_other_stream(lr):
    """Rows of x and y that lie differently against 16-byte boundaries, on a stream of the caller's."""
    g = torch.Generator().manual_seed(3)
    dim, L = 7, 301
    raw = torch.randn(dim * L + 3, generator=g).bfloat16().cuda()
    x = raw[3:].view(1, dim, L)
    w, b = _params(g, dim, 4)
    wd, bd = w.cuda(), b.cuda()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        y, _ = lr.sconv_fwd(x, wd, bd)
    st.synchronize()
    assert "vec=0" in lr.last_plan()
    yr, _, size = ref.conv(ref.d64(x), ref.d64(w), ref.d64(b), torch.zeros(1, dim, 3, dtype=torch.float64))
    _near(y, yr, size, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,dim,L,width", [
    (1, 1, 1, 4), (2, 3, 2, 4), (1, 5, 3, 3), (2, 4, 8, 2), (2, 6, 248, 4), (1, 7, 249, 3), (3, 5, 700, 4), (1, 2, 4100, 4)])
@pytest.mark.parametrize("form", ["plain", "view", "state"])
def test_backward(lr, dtype, batch, dim, L, width, form):
    g = torch.Generator().manual_seed(L * 5 + width)
    x = torch.randn(batch, 2 * dim, L, generator=g).to(IO[dtype]).cuda()
    x = x[:, dim:] if form == "view" else x[:, :dim].contiguous()
    w, b = _params(g, dim, width, bias=form != "view")
    x0 = torch.randn(batch, dim, width - 1, generator=g).to(IO[dtype]) if form == "state" else None
    dfin = torch.randn(batch, dim, width - 1, generator=g).to(IO[dtype]) if form == "state" else None
    dy = torch.randn(batch, dim, L, generator=g).to(IO[dtype])
    act = form != "view"
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = lr.sconv_bwd(x, w.cuda(), cu(b), cu(x0), dy.cuda(), cu(dfin), silu=act)
    again = lr.sconv_bwd(x, w.cuda(), cu(b), cu(x0), dy.cuda(), cu(dfin), silu=act)
    assert lr.get_last_error() == 0

    leaf = {"x": ref.d64(x).requires_grad_(), "weight": ref.d64(w).requires_grad_()}
    if b is not None:
        leaf["bias"] = ref.d64(b).requires_grad_()
    leaf["x0"] = (torch.zeros(batch, dim, width - 1, dtype=torch.float64) if x0 is None else ref.d64(x0)).requires_grad_()
    y, last, _ = ref.conv(leaf["x"], leaf["weight"], leaf.get("bias"), leaf["x0"], act)
    total = (y * ref.d64(dy)).sum() + (0 if dfin is None else (last * ref.d64(dfin)).sum())
    want = dict(zip(leaf, torch.autograd.grad(total, list(leaf.values()))))
    # magnitudes: |dc| <= 1.1 |dy|, so the sums' terms are below 1.1 |dy| |w|, 1.1 |dy| |x|
    wide = torch.cat([ref.d64(dy).abs(), torch.zeros(batch, dim, width - 1, dtype=torch.float64)], 2)
    size_x = 1.1 * sum(ref.d64(w)[:, k, None].abs() * wide[..., width - 1 - k:width - 1 - k + L] for k in range(width))
    # c's own rounding passes through silu' (slope below 0.5) times dy
    size_x = size_x + size_x * (1 + ref.d64(x).abs().amax())
    _near(got["dx"], want["x"], size_x, dtype, 2e-6)
    n = ref.d64(dy).abs().sum((0, 2)) * 1.1
    big = torch.maximum(ref.d64(x).abs().amax((0, 2)), leaf["x0"].detach().abs().amax((0, 2)))
    _near(got["dweight"], want["weight"], (n * (1 + big) ** 2)[:, None].expand(-1, width), "f32", 1e-5)
    if b is not None:
        _near(got["dbias"], want["bias"], n * (1 + big), "f32", 1e-5)
    else:
        assert got["dbias"] is None
    if x0 is not None:
        top = ref.d64(dy).abs().amax() * ref.d64(w).abs().sum(1).amax() * 2
        _near(got["dx0"], want["x0"], top.expand_as(want["x0"]), dtype, 2e-6)
    for k in got:
        assert got[k] is None or torch.equal(got[k], again[k]), k


def test_backward_against_differences(lr):
    """The gradients predict the forward's change along a random direction (64-bit central differences)."""
    g = torch.Generator().manual_seed(11)
    batch, dim, L, width = 2, 3, 21, 4
    t = {"x": torch.randn(batch, dim, L, generator=g), "weight": torch.randn(dim, width, generator=g),
         "bias": torch.randn(dim, generator=g), "x0": torch.randn(batch, dim, width - 1, generator=g)}
    dy, dfin = torch.randn(batch, dim, L, generator=g), torch.randn(batch, dim, width - 1, generator=g)
    got = lr.sconv_bwd(t["x"].cuda(), t["weight"].cuda(), t["bias"].cuda(), t["x0"].cuda(), dy.cuda(), dfin.cuda())

    def value(v):
        y, last, _ = ref.conv(v["x"], v["weight"], v["bias"], v["x0"])
        return float((y * dy.double()).sum() + (last * dfin.double()).sum())

    for name in t:
        way = torch.randn(t[name].shape, generator=g, dtype=torch.float64)
        hi, lo = ({k: v.double() for k, v in t.items()} for _ in range(2))
        hi[name], lo[name] = hi[name] + 1e-5 * way, lo[name] - 1e-5 * way
        slope = (value(hi) - value(lo)) / 2e-5
        mine = float((got["d" + name].double().cpu() * way).sum())
        assert abs(mine - slope) <= 1e-4 * (1 + abs(slope)), name


CUTS = {
    "one": [0, 700],
    "ragged": [0, 0, 1, 2, 4, 7, 7, 7, 256, 259, 511, 512, 515, 700, 700],
    "singles": list(range(0, 41)) + [700],
    "gaps": [5, 9, 9, 300, 650],  # tokens before, between no requests and after belong to none
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("cuts", list(CUTS))
@pytest.mark.parametrize("tokens,dim", [(700, 9), (701, 40)])
def test_prompt(lr, dtype, width, cuts, tokens, dim):
    g = torch.Generator().manual_seed(tokens + width)
    cu = CUTS[cuts]
    n = len(cu) - 1
    x = torch.randn(dim, tokens, generator=g).to(IO[dtype])
    w, b = _params(g, dim, width)
    state = torch.randn(n + 3, dim, width - 1, generator=g).to(IO[dtype])
    slots = torch.randperm(n + 3, generator=g)[:n].int()
    if n > 3:
        slots[2] = -1
    has = torch.rand(n, generator=g) < 0.5
    for s in range(n):  # rows that nothing may read hold NaN
        if not has[s] and slots[s] >= 0:
            state[slots[s]] = float("nan")
    got_state = state.cuda()
    y = lr.sconv_prompt(x.cuda(), w.cuda(), b.cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
                        state=got_state, slots=slots.cuda(), has_state=has.cuda())
    assert lr.get_last_error() == 0
    clean = torch.nan_to_num(ref.d64(state))
    yr, sr, size = ref.conv_packed(ref.d64(x), ref.d64(w), ref.d64(b), cu, slots.tolist(), has.tolist(), clean)
    _near(y, yr, size, dtype)
    touched = [int(v) for v in slots if v >= 0]
    assert torch.equal(got_state.double().cpu()[touched], sr[touched])
    rest = [i for i in range(n + 3) if i not in touched]
    assert torch.equal(got_state.cpu()[rest].float(), state[rest].float())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,dim,width", [(1, 1, 4), (3, 7, 3), (5, 64, 4), (9, 520, 2), (300, 24, 4), (700, 2056, 4)])
def test_step_continues_a_prompt(lr, dtype, batch, dim, width):
    """Steps from a cache equal the packed form with one token a request, and the reference."""
    g = torch.Generator().manual_seed(batch + dim)
    both = torch.randn(batch, 2 * dim, generator=g).to(IO[dtype]).cuda()
    w, b = _params(g, dim, width)
    state = torch.randn(batch + 2, dim, width - 1, generator=g).to(IO[dtype])
    slots = torch.randperm(batch + 2, generator=g)[:batch].int()
    if batch > 2:
        slots[1] = -1
    s1, s2 = state.cuda(), state.cuda()
    x = both[:, dim:]
    y = lr.sconv_step(x, w.cuda(), b.cuda(), state=s1, slots=slots.cuda())
    assert lr.get_last_error() == 0 and lr.last_launch_count() == 1
    cu = list(range(batch + 1))
    yr, sr, size = ref.conv_packed(ref.d64(x).t().contiguous(), ref.d64(w), ref.d64(b), cu, slots.tolist(), None, ref.d64(state))
    _near(y, yr.t(), size.t(), dtype)
    assert torch.equal(s1.double().cpu(), sr)
    yp = lr.sconv_prompt(x.t().contiguous(), w.cuda(), b.cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
                         state=s2, slots=slots.cuda())
    torch.cuda.synchronize()
    assert torch.equal(s1, s2)
    _near(yp, yr, size, dtype)


def test_empty_calls(lr):
    w = torch.ones(4, 4).cuda()
    x0 = torch.randn(2, 4, 3).cuda()
    y, last = lr.sconv_fwd(torch.empty(2, 4, 0).cuda(), w, None, x0)
    assert y.shape == (2, 4, 0) and torch.equal(last, x0)
    g = lr.sconv_bwd(torch.empty(2, 4, 0).cuda(), w, None, x0, torch.empty(2, 4, 0).cuda(), x0 * 2)
    torch.cuda.synchronize()
    assert torch.equal(g["dx0"], x0 * 2) and not g["dweight"].any()
    state = torch.ones(3, 4, 3).cuda()
    lr.sconv_prompt(torch.empty(4, 0).cuda(), w, cu_seqlens=torch.zeros(3, dtype=torch.int32).cuda(), state=state,
                    slots=torch.tensor([2, 0], dtype=torch.int32).cuda(), has_state=torch.tensor([False, True]).cuda())
    torch.cuda.synchronize()
    assert not state[2].any() and bool((state[:2] == 1).all())


def test_tables_outside_the_arrays_are_reported(lr):
    """Offsets and slots out of range are clamped on the device and reported; rows in range keep their values."""
    x, w = torch.randn(4, 10).cuda(), torch.ones(4, 4).cuda()
    state = torch.zeros(2, 4, 3).cuda()
    lr.sconv_prompt(x, w, cu_seqlens=torch.tensor([0, 5, 12], dtype=torch.int32).cuda(), state=state)
    assert lr.get_last_error() == lr.SSCAN_ERR_INVALID
    lr.sconv_prompt(x, w, cu_seqlens=torch.tensor([0, 5, 10], dtype=torch.int32).cuda(), state=state.zero_(),
                    slots=torch.tensor([7, 1], dtype=torch.int32).cuda())
    assert lr.get_last_error() == lr.SSCAN_ERR_INVALID
    assert not state[0].any() and torch.equal(state[1], x[:, 7:])
    lr.sconv_step(torch.ones(2, 4).cuda(), w, state=state, slots=torch.tensor([0, 2], dtype=torch.int32).cuda())
    assert lr.get_last_error() == lr.SSCAN_ERR_INVALID
    lr.sconv_step(torch.ones(2, 4).cuda(), w, state=state)
    assert lr.get_last_error() == 0
