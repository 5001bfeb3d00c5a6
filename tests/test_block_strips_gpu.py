"""Calls large enough that the convolution's warps walk strips of several tiles,
with requests that begin just before and after every tile's border, and packed
calls of many very short requests.  Sampled channels are checked against the
64-bit forms with the tolerances of the operators' own tests."""
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    yield m
    torch.cuda.empty_cache()


def _near(got, want, size, dtype):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    tol = 1e-6 * (size + want.abs()) + 1e-7 + (want.abs() * 2.0 ** -8 if dtype == "bf16" else 0)
    assert bool(((got - want).abs() <= tol).all())


def _tables(g, cu):
    n = len(cu) - 1
    slots = torch.randperm(n + 5, generator=g)[:n].int()
    slots[torch.randperm(n, generator=g)[:n // 20]] = -1
    return slots, torch.rand(n, generator=g) < 0.5, n + 5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [16411, 16416])
@pytest.mark.parametrize("dim", [1000, 5120])
@pytest.mark.parametrize("width", [2, 4])
def test_requests_around_every_tile_border(lr, dtype, tokens, dim, width):
    g = torch.Generator().manual_seed(tokens + dim)
    tile = 31 * (4 if dtype == "f32" else 8)
    # starts from 18 tokens before to 3 after each border, of one or two tokens, and the rest between
    steps = [1 + (i + m) % 2 for m in range(2) for i in range(24)]
    cu = {0, tokens}
    for i, border in enumerate(range(tile, tokens, tile)):
        at = border - 18
        while at <= border + 3:
            cu.add(min(max(at, 0), tokens))
            at += steps[(at + i) % len(steps)]
    cu = sorted(cu)
    cu = cu[:len(cu) // 2] + [cu[len(cu) // 2]] * 3 + cu[len(cu) // 2:]  # some empty ones
    slots, has, rows = _tables(g, cu)
    gd = torch.Generator(device="cuda").manual_seed(dim)
    x = torch.randn(dim, tokens, generator=gd, device="cuda").to(IO[dtype])
    w, b = torch.randn(dim, width, generator=gd, device="cuda"), torch.randn(dim, generator=gd, device="cuda")
    state = torch.randn(rows, dim, width - 1, generator=gd, device="cuda").to(IO[dtype])
    old = state.clone()
    y = lr.sconv_prompt(x, w, b, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), state=state, slots=slots.cuda(),
                        has_state=has.cuda())
    assert lr.get_last_error() == 0 and lr.last_launch_count() == 2
    pick = [0, 7, 8, 333, dim - 1]
    yr, sr, size = ref.conv_packed(ref.d64(x[pick]), ref.d64(w[pick]), ref.d64(b[pick]), cu, slots.tolist(), has.tolist(),
                                   ref.d64(old[:, pick]))
    _near(y[pick], yr, size, dtype)
    assert torch.equal(state[:, pick].double().cpu(), sr)
    # and every channel's cache: a request's last inputs, or its row before them where it continues
    cuts = torch.tensor(cu)
    long_enough = (cuts[1:] - cuts[:-1] >= width - 1) & (slots >= 0)
    ends, to = cuts[1:][long_enough], slots[long_enough].long().cuda()
    last = x[:, (ends[:, None] + torch.arange(-(width - 1), 0)).cuda()].permute(1, 0, 2)
    assert torch.equal(state[to], last)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [2000, 2003])
@pytest.mark.parametrize("before", [False, True])
def test_training_shape(lr, dtype, L, before):
    g = torch.Generator(device="cuda").manual_seed(L)
    batch, dim, width = 4, 2048, 4
    x, dy = (torch.randn(batch, dim, L, generator=g, device="cuda").to(IO[dtype]) for _ in range(2))
    w, b = torch.randn(dim, width, generator=g, device="cuda"), torch.randn(dim, generator=g, device="cuda")
    x0 = torch.randn(batch, dim, width - 1, generator=g, device="cuda").to(IO[dtype]) if before else None
    y, last = lr.sconv_fwd(x, w, b, x0)
    got = lr.sconv_bwd(x, w, b, x0, dy)
    assert lr.get_last_error() == 0
    pick = [0, 1, 7, 8, 1023, 2040, 2047]
    zero = torch.zeros(batch, len(pick), width - 1, dtype=torch.float64)
    xs, ws, bs = (t.requires_grad_() for t in (ref.d64(x[:, pick]), ref.d64(w[pick]), ref.d64(b[pick])))
    yr, lastr, size = ref.conv(xs, ws, bs, zero if x0 is None else ref.d64(x0[:, pick]))
    dx, dw, db = torch.autograd.grad((yr * ref.d64(dy[:, pick])).sum(), (xs, ws, bs))
    _near(y[:, pick], yr.detach(), size.detach(), dtype)
    assert torch.equal(last[:, pick].double().cpu(), lastr.detach())
    # |dc| <= 1.1 |dy|; c's rounding passes through silu', whose slope is below 0.5
    scale = 1.1 * float(dy.abs().max()) * ref.d64(w[pick]).abs().sum(1).view(1, -1, 1) * (2 + float(x.abs().max()))
    _near(got["dx"][:, pick], dx, scale.expand_as(dx), dtype)
    n, big = ref.d64(dy[:, pick]).abs().sum((0, 2)), float(x.abs().max())
    assert bool(((got["dweight"][pick].double().cpu() - dw).abs() <= 1e-5 * 1.1 * (n * (1 + big) ** 2)[:, None]).all())
    assert bool(((got["dbias"][pick].double().cpu() - db).abs() <= 1e-5 * 1.1 * n * (1 + big)).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [40, 4100])
@pytest.mark.parametrize("tokens", [900, 907])
@pytest.mark.parametrize("options", [False, True])
def test_scan_of_hundreds_of_short_requests(lr, dtype, dim, tokens, options):
    """Requests of none to three tokens: nearly every token begins one."""
    g = torch.Generator().manual_seed(tokens)
    N, cu = 16, [0]
    while cu[-1] < tokens:
        cu.append(min(tokens, cu[-1] + int(torch.randint(0, 4, (1,), generator=g))))
    slots, has, rows = _tables(g, cu)
    gd = torch.Generator(device="cuda").manual_seed(dim)
    r = lambda *s: torch.randn(*s, generator=gd, device="cuda")  # noqa: E731
    u, z, B, C = (r(*s).to(IO[dtype]) for s in ((dim, tokens), (dim, tokens), (N, tokens), (N, tokens)))
    raw = r(dim, tokens) * 0.7 - 2
    delta = (raw if options else torch.log1p(raw.exp())).to(IO[dtype])
    A, D, bias = -(torch.rand(dim, N, generator=gd, device="cuda") + 0.5), r(dim), r(dim) * 0.1
    first = r(rows, dim, N)
    pick = [0, 1, 17, 31, 32, dim - 1]
    d = ref.d64
    yr, sr, _ = ref.scan_packed(d(u[pick]), d(delta[pick]), d(A[pick]), d(B), d(C), d(D[pick]), cu, slots.tolist(), has.tolist(),
                                d(first[:, pick]), d(z[pick]) if options else None, d(bias[pick]) if options else None, options)
    for segments in (0, 1, 7):
        state = first.clone()
        y = lr.sscan_prompt(u, delta, A, B, C, D, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), state=state,
                            slots=slots.cuda(), has_state=has.cuda(), z=z if options else None,
                            delta_bias=bias if options else None, delta_softplus=options, segments=segments)
        assert lr.get_last_error() == 0
        tol = 1e-4 if dtype == "f32" else 2e-2
        assert float(((y[pick].double().cpu() - yr).abs() / (1 + yr.abs())).max()) <= tol
        assert float(((state[:, pick].double().cpu() - sr).abs() / (1 + sr.abs())).max()) <= 1e-4
