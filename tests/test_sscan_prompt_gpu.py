"""GPU parity of the packed selective scan and the cached decode step with the
64-bit form.

Tolerances: those of the scan (1e-4 (1 + |y|) in fp32, 2e-2 (1 + |y|) in bf16,
states 1e-4 (1 + |h|)).  Per step the decay has about 2^-22 of relative error,
which a state forgets with its own decay, so sums over a memory of m steps
stay within m * 2^-22 of their magnitude: below 1e-4 for the memories of a
few hundred steps here."""
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
IO = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"f32": 1e-4, "bf16": 2e-2}


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


def _near(got, want, tol):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    err = float(((got - want).abs() / (1 + want.abs())).max()) if want.numel() else 0.0
    assert err <= tol, err


def _inputs(g, dtype, lead, side, dim, N, options, slow=False):
    io = IO[dtype]
    raw = torch.randn(*lead, generator=g) * 0.7 - (4.5 if slow else 2.0)
    x = {"u": torch.randn(*lead, generator=g).to(io), "delta": (raw if options else torch.log1p(raw.exp())).to(io),
         "A": -(torch.arange(1, N + 1) * (torch.rand(dim, N, generator=g) + 0.5)).float(),
         "B": torch.randn(*side, generator=g).to(io), "C": torch.randn(*side, generator=g).to(io),
         "D": torch.randn(dim, generator=g),
         "z": torch.randn(*lead, generator=g).to(io) if options else None,
         "bias": torch.randn(dim, generator=g) * 0.1 if options else None}
    return x


def _run(lr, x, cu, state, slots, has, options, segments=0):
    c = {k: None if v is None else v.cuda() for k, v in x.items()}
    return lr.sscan_prompt(c["u"], c["delta"], c["A"], c["B"], c["C"], c["D"],
                           cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), state=state,
                           slots=None if slots is None else slots.cuda(), has_state=None if has is None else has.cuda(),
                           z=c["z"], delta_bias=c["bias"], delta_softplus=options, segments=segments)


def _want(x, cu, state, slots, has, options):
    d = {k: ref.d64(v) for k, v in x.items()}
    return ref.scan_packed(d["u"], d["delta"], d["A"], d["B"], d["C"], d["D"], cu, None if slots is None else slots.tolist(),
                           None if has is None else has.tolist(), ref.d64(state), d["z"], d["bias"], options)


CUTS = {
    "one": [0, 331],
    "ragged": [0, 0, 1, 3, 16, 32, 33, 33, 47, 48, 64, 200, 331, 331],
    "singles": list(range(0, 37)) + [331],
    "gaps": [5, 9, 9, 130, 300],
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cuts", list(CUTS))
@pytest.mark.parametrize("options", [False, True])
@pytest.mark.parametrize("segments", [0, 1, 3, 21])
def test_ragged_prompts(lr, dtype, cuts, options, segments):
    g = torch.Generator().manual_seed(segments)
    cu, tokens, dim, N = CUTS[cuts], 331, 35, 16
    n = len(cu) - 1
    x = _inputs(g, dtype, (dim, tokens), (N, tokens), dim, N, options)
    state = torch.randn(n + 2, dim, N, generator=g)
    slots = torch.randperm(n + 2, generator=g)[:n].int()
    if n > 3:
        slots[3] = -1
    has = torch.rand(n, generator=g) < 0.5
    for s in range(n):
        if not has[s] and slots[s] >= 0:
            state[slots[s]] = float("nan")
    got = state.cuda()
    y = _run(lr, x, cu, got, slots, has, options, segments)
    assert lr.get_last_error() == 0
    yr, sr, _ = _want(x, cu, torch.nan_to_num(state), slots, has, options)
    _near(y, yr, TOL[dtype])
    touched = [int(v) for v in slots if v >= 0]
    _near(got[touched], sr[touched], 1e-4)
    rest = [i for i in range(n + 2) if i not in touched]
    assert torch.equal(got.cpu()[rest], state[rest])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,N", [(1, 1), (130, 3), (70, 8), (33, 17), (20, 32), (9, 33), (40, 64), (257, 16)])
@pytest.mark.parametrize("tokens", [1, 15, 16, 144])
def test_state_counts_and_widths(lr, dtype, dim, N, tokens):
    g = torch.Generator().manual_seed(dim + tokens)
    cu = [0, tokens // 3, tokens]
    x = _inputs(g, dtype, (dim, tokens), (N, tokens), dim, N, True)
    state = torch.randn(2, dim, N, generator=g)
    for segments in (1, 4):
        got = state.cuda()
        y = _run(lr, x, cu, got, None, None, True, segments)
        assert lr.get_last_error() == 0
        yr, sr, _ = _want(x, cu, state, None, None, True)
        _near(y, yr, TOL[dtype])
        _near(got, sr, 1e-4)


def test_slow_decay_crosses_many_segments(lr):
    """States that remember over all borders: A of zero, slow and (briefly) growing rates."""
    g = torch.Generator().manual_seed(2)
    dim, N, tokens = 40, 16, 512
    x = _inputs(g, "f32", (dim, tokens), (N, tokens), dim, N, False, slow=True)
    x["A"][:, 0] = 0.0
    x["A"][:, 1] = -1e-3
    x["A"][:, 2] = 0.02
    state = torch.randn(1, dim, N, generator=g)
    for segments in (1, 8, 32):
        got = state.cuda()
        y = _run(lr, x, [0, tokens], got, None, None, False, segments)
        assert lr.get_last_error() == 0
        assert f"segments={segments} " in lr.last_plan()
        yr, sr, _ = _want(x, [0, tokens], state, None, None, False)
        _near(y, yr, 1e-4)
        _near(got, sr, 1e-4)


def test_nan_of_one_request_stays_in_it(lr):
    g = torch.Generator().manual_seed(4)
    dim, N, tokens, cu = 33, 16, 200, [0, 70, 131, 200]
    x = _inputs(g, "f32", (dim, tokens), (N, tokens), dim, N, True)
    state = torch.randn(3, dim, N, generator=g)
    clean = {k: None if v is None else v.clone() for k, v in x.items()}
    for k in ("u", "delta", "z", "B", "C"):
        x[k][:, 70:131] = float("nan")
    state[1] = float("inf")
    for segments in (1, 5, 13):
        got = state.cuda()
        y = _run(lr, x, cu, got, None, None, True, segments)
        yr, sr, _ = _want(clean, cu, torch.nan_to_num(state, posinf=0.0), None, None, True)
        keep = [t for t in range(tokens) if not 70 <= t < 131]
        _near(y[:, keep], yr[:, keep], 1e-4)
        _near(got[[0, 2]], sr[[0, 2]], 1e-4)
        assert torch.isnan(y[:, 70:131]).all()


def test_prompt_in_parts_and_single_tokens(lr):
    """A prompt in two calls and then token by token equals the prompt at once, through one cache row."""
    g = torch.Generator().manual_seed(5)
    dim, N, tokens = 64, 16, 90
    x = _inputs(g, "f32", (dim, tokens), (N, tokens), dim, N, True)
    whole = torch.zeros(1, dim, N)
    yr, sr, _ = _want(x, [0, tokens], whole, None, torch.tensor([False]), True)
    cache = torch.full((3, dim, N), 7.0).cuda()
    slots = torch.tensor([2], dtype=torch.int32)
    at = [0, 33, 80]
    out = []
    for i, (a, b) in enumerate(zip(at, at[1:])):
        part = {k: v[:, a:b].contiguous() if v is not None and v.dim() == 2 and v.shape[1] == tokens else v for k, v in x.items()}
        out.append(_run(lr, part, [0, b - a], cache, slots, torch.tensor([i > 0]), True))
    c = {k: None if v is None else v.cuda() for k, v in x.items()}
    for t in range(80, tokens):
        row = lambda k: c[k][:, t][None].contiguous()  # noqa: E731
        out.append(lr.sscan_step(row("u"), row("delta"), c["A"], row("B"), row("C"), c["D"], state=cache,
                                 slots=slots.cuda(), z=row("z"), delta_bias=c["bias"], delta_softplus=True).t())
    assert lr.get_last_error() == 0
    _near(torch.cat(out, 1), yr, 1e-4)
    _near(cache[2:], sr, 1e-4)
    assert bool((cache[:2] == 7).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,dim,N", [(1, 1, 1), (3, 7, 3), (4, 33, 16), (2, 130, 64), (5, 17, 5), (2, 9, 24), (300, 8, 8)])
def test_step_over_slots(lr, dtype, batch, dim, N):
    g = torch.Generator().manual_seed(batch + N)
    x = _inputs(g, dtype, (batch, dim), (batch, N), dim, N, True)
    both = torch.randn(batch, 2 * dim, generator=g).to(IO[dtype])
    x["z"] = both[:, dim:]
    state = torch.randn(batch + 3, dim, N, generator=g)
    slots = torch.randperm(batch + 3, generator=g)[:batch].int()
    if batch > 2:
        slots[0] = -1
    got = state.cuda()
    c = {k: v.cuda() for k, v in x.items()}
    y = lr.sscan_step(c["u"], c["delta"], c["A"], c["B"], c["C"], c["D"], state=got, slots=slots.cuda(),
                      z=both.cuda()[:, dim:], delta_bias=c["bias"], delta_softplus=True)
    assert lr.get_last_error() == 0 and lr.last_launch_count() == 1
    yr, sr = torch.empty(batch, dim, dtype=torch.float64), ref.d64(state)
    for b in range(batch):
        one = {k: v[b:b + 1].t().contiguous() if k in ("u", "delta", "B", "C", "z") else v for k, v in x.items()}
        ys, ss, _ = _want(one, [0, 1], state, slots[b:b + 1], None, True)
        yr[b] = ys[:, 0]
        if slots[b] >= 0:
            sr[slots[b]] = ss[slots[b]]
    _near(y, yr, TOL[dtype])
    _near(got, sr, 1e-4)


def test_tables_outside_the_arrays_are_reported(lr):
    g = torch.Generator().manual_seed(6)
    x = _inputs(g, "f32", (8, 40), (4, 40), 8, 4, False)
    state = torch.zeros(2, 8, 4).cuda()
    _run(lr, x, [0, 50, 40], state, None, None, False)
    assert lr.get_last_error() == lr.SSCAN_ERR_INVALID
    _run(lr, x, [0, 20, 40], state, torch.tensor([0, 9], dtype=torch.int32), None, False, 2)
    assert lr.get_last_error() == lr.SSCAN_ERR_INVALID
    _run(lr, x, [0, 20, 40], state, torch.tensor([1, 0], dtype=torch.int32), None, False)
    assert lr.get_last_error() == 0


def test_no_tokens(lr):
    x = _inputs(torch.Generator().manual_seed(1), "bf16", (8, 0), (4, 0), 8, 4, True)
    state = torch.ones(2, 8, 4).cuda()
    y = _run(lr, x, [0, 0, 0], state, None, torch.tensor([True, False]), True)
    assert lr.get_last_error() == 0 and y.shape == (8, 0)
    assert bool((state[0] == 1).all()) and not state[1].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("options", [False, True])
@pytest.mark.parametrize("N,dim", [(3, 8200), (8, 8192), (16, 4100), (20, 2050), (64, 1028)])
@pytest.mark.parametrize("tokens", [331, 336])
def test_calls_large_enough_for_wide_threads(lr, dtype, options, N, dim, tokens):
    """The form for calls that fill the GPU (eight states of two channels a thread), rows aligned and not."""
    g = torch.Generator().manual_seed(N + tokens)
    cu = [0, 0, 1, 3, 16, 32, 33, 33, 47, 48, 64, 200, tokens, tokens]
    n = len(cu) - 1
    x = _inputs(g, dtype, (dim, tokens), (N, tokens), dim, N, options)
    state = torch.randn(n, dim, N, generator=g)
    slots = torch.randperm(n, generator=g).int()
    slots[4] = -1
    has = torch.rand(n, generator=g) < 0.5
    got0 = state.clone()
    yr, sr, _ = _want(x, cu, state, slots, has, options)
    for segments in (0, 1, 7):
        got = got0.cuda()
        y = _run(lr, x, cu, got, slots, has, options, segments)
        assert lr.get_last_error() == 0 and "narrow" not in lr.last_plan()
        _near(y, yr, TOL[dtype])
        _near(got, sr, 1e-4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1280, 1283])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
def test_states_that_fade_in_any_order(lr, dtype, tokens, order):
    """Four states of a group that fade far apart, the first or the last of them
    first, across borders of segments longer and shorter than their memories."""
    g = torch.Generator().manual_seed(tokens)
    dim, N = 70, 10
    options = dtype == "bf16"
    x = _inputs(g, dtype, (dim, tokens), (N, tokens), dim, N, options)
    rates = torch.tensor([0.05, 0.6, 7.0, 80.0])
    if order == "falling":
        rates = rates.flip(0)
    elif order == "mixed":
        rates = rates[[2, 0, 3, 1]]
    x["A"] = -(rates.repeat(3)[:N] * (torch.rand(dim, N, generator=g) + 0.5)).float()
    state = torch.randn(2, dim, N, generator=g)
    cu = [0, tokens - 500, tokens]
    for segments in (0, 3, 16):
        got = state.cuda()
        y = _run(lr, x, cu, got, None, None, options, segments)
        assert lr.get_last_error() == 0
        yr, sr, _ = _want(x, cu, state, None, None, options)
        _near(y, yr, TOL[dtype])
        _near(got, sr, 1e-4)
