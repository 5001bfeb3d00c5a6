"""The operators around the scan where sizes leave the ordinary: arrays and
caches of more than 2^31 elements, more batches or groups than a grid
dimension holds, channel groups too wide for shared memory, and captured
graphs.  Sampled rows are checked with the 64-bit forms; the tolerances are those of
the operators' own tests."""
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    yield m
    torch.cuda.empty_cache()


def _close(got, want, tol):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    err = float(((got - want).abs() / (1 + want.abs())).max())
    assert err <= tol, err


def test_packed_rows_beyond_32_bits(lr):
    g = torch.Generator(device="cuda").manual_seed(1)
    dim, tokens, N = 140000, 16001, 2
    assert dim * tokens > 1 << 31
    x = torch.randn(dim, tokens, generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(dim, 4, generator=g, device="cuda")
    cu = [0, 9000, 9001, tokens]
    table = torch.tensor(cu, dtype=torch.int32, device="cuda")
    conv_state = torch.randn(3, dim, 3, generator=g, device="cuda").bfloat16()
    old = conv_state.clone()
    y = lr.sconv_prompt(x, w, cu_seqlens=table, state=conv_state)
    assert lr.get_last_error() == 0
    rows = [0, 70001, dim - 1]
    want, last, _ = ref.conv_packed(ref.d64(x[rows]), ref.d64(w[rows]), None, cu, None, None, ref.d64(old[:, rows]))
    _close(y[rows], want, 8e-3)
    assert torch.equal(conv_state[:, rows].double().cpu(), last)
    del y
    delta = torch.rand(dim, tokens, generator=g, device="cuda", dtype=torch.bfloat16) * 0.2
    A = -torch.rand(dim, N, generator=g, device="cuda") - 0.5
    B, C = (torch.randn(N, tokens, generator=g, device="cuda").bfloat16() for _ in range(2))
    state = torch.randn(3, dim, N, generator=g, device="cuda")
    h0 = state.clone()
    y = lr.sscan_prompt(x, delta, A, B, C, cu_seqlens=table, state=state)
    assert lr.get_last_error() == 0
    want, last, _ = ref.scan_packed(ref.d64(x[rows]), ref.d64(delta[rows]), ref.d64(A[rows]), ref.d64(B), ref.d64(C), None, cu,
                                    None, None, ref.d64(h0[:, rows]))
    _close(y[rows], want, 2e-2)
    _close(state[:, rows], last, 1e-4)


def test_cache_rows_beyond_32_bits(lr):
    g = torch.Generator(device="cuda").manual_seed(2)
    rows, dim, N = 70000, 2048, 16
    assert rows * dim * N > 1 << 31
    state = torch.zeros(rows, dim, N, device="cuda")
    slots = torch.tensor([rows - 1, 0, 65537, rows - 2], dtype=torch.int32, device="cuda")
    state[slots.long()] = torch.randn(4, dim, N, generator=g, device="cuda")
    h0 = state[slots.long()].clone()
    u, delta = torch.randn(4, dim, generator=g, device="cuda"), torch.rand(4, dim, generator=g, device="cuda")
    A = -torch.rand(dim, N, generator=g, device="cuda")
    B, C = (torch.randn(4, N, generator=g, device="cuda") for _ in range(2))
    y = lr.sscan_step(u, delta, A, B, C, state=state, slots=slots)
    assert lr.get_last_error() == 0
    h = torch.exp(ref.d64(delta)[:, :, None] * ref.d64(A)) * ref.d64(h0) + ref.d64(delta * u)[:, :, None] * ref.d64(B)[:, None]
    _close(state[slots.long()], h, 1e-4)
    _close(y, (h * ref.d64(C)[:, None]).sum(-1), 1e-4)
    # the packed form through the same far rows
    got = lr.sscan_prompt(u.t().contiguous(), delta.t().contiguous(), A, B.t().contiguous(), C.t().contiguous(),
                          cu_seqlens=torch.arange(5, dtype=torch.int32, device="cuda"), state=state, slots=slots)
    assert lr.get_last_error() == 0
    h = torch.exp(ref.d64(delta)[:, :, None] * ref.d64(A)) * h + ref.d64(delta * u)[:, :, None] * ref.d64(B)[:, None]
    _close(state[slots.long()], h, 1e-4)
    _close(got.t(), (h * ref.d64(C)[:, None]).sum(-1), 1e-4)


def test_more_batches_than_a_grid_dimension(lr):
    g = torch.Generator(device="cuda").manual_seed(3)
    batch = 65600
    x = torch.randn(batch, 2, 5, generator=g, device="cuda")
    w, b = torch.randn(2, 4, generator=g, device="cuda"), torch.randn(2, generator=g, device="cuda")
    dy = torch.randn(batch, 2, 5, generator=g, device="cuda")
    y, last = lr.sconv_fwd(x, w, b)
    got = lr.sconv_bwd(x, w, b, None, dy)
    xs, ws, bs = (ref.d64(t).requires_grad_() for t in (x, w, b))
    yr, lastr, _ = ref.conv(xs, ws, bs, torch.zeros(batch, 2, 3, dtype=torch.float64))
    dx, dw, db = torch.autograd.grad((yr * ref.d64(dy)).sum(), (xs, ws, bs))
    _close(y, yr.detach(), 1e-5)
    assert torch.equal(last.double().cpu(), lastr.detach())
    _close(got["dx"], dx, 1e-5)
    scale = float(ref.d64(dy).abs().sum())
    assert float((got["dweight"].double().cpu() - dw).abs().max()) <= 1e-5 * scale
    assert float((got["dbias"].double().cpu() - db).abs().max()) <= 1e-5 * scale
    z = torch.randn(batch, 2, 5, generator=g, device="cuda")
    out = lr.gatenorm_fwd(x, z, b)
    grads = lr.gatenorm_bwd(x, z, b, dy)
    ys, zs, ws = (ref.d64(t).requires_grad_() for t in (x, z, b))
    want = ref.gatenorm(ys, zs, ws, 1, False, 1e-5)
    dys, dzs, dws = torch.autograd.grad((want * ref.d64(dy)).sum(), (ys, zs, ws))
    _close(out, want.detach(), 1e-5)
    # a norm over two channels can have a large slope: errors in terms of the largest gradient
    assert float((grads["dy"].double().cpu() - dys).abs().max()) <= 1e-5 * float(dys.abs().max())
    assert float((grads["dz"].double().cpu() - dzs).abs().max()) <= 1e-5 * float(dzs.abs().max())
    assert float((grads["dweight"].double().cpu() - dws).abs().max()) <= 1e-5 * scale


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L", [5, 16])
@pytest.mark.parametrize("norm_first", [False, True])
def test_channel_groups_wider_than_shared_memory(lr, dtype, L, norm_first):
    g = torch.Generator().manual_seed(4)
    dim = 16400
    y, z, do = (torch.randn(1, dim, L, generator=g).to(dtype) for _ in range(3))
    w = 1 + 0.1 * torch.randn(dim, generator=g)
    kw = dict(norm_first=norm_first)
    out = lr.gatenorm_fwd(y.cuda(), z.cuda(), w.cuda(), **kw)
    assert "cluster=0" in lr.last_plan()
    got = lr.gatenorm_bwd(y.cuda(), z.cuda(), w.cuda(), do.cuda(), **kw)
    assert "cluster=0" in lr.last_plan() and lr.get_last_error() == 0
    ys, zs, ws = (ref.d64(t).requires_grad_() for t in (y, z, w))
    want = ref.gatenorm(ys, zs, ws, 1, norm_first, 1e-5)
    dy, dz, dw = torch.autograd.grad((want * ref.d64(do)).sum(), (ys, zs, ws))
    tol = 1e-5 if dtype == torch.float32 else 2.0 ** -8
    _close(out, want.detach(), tol)
    _close(got["dy"], dy, tol)
    _close(got["dz"], dz, tol)
    _close(got["dweight"], dw, 2e-5)


def test_many_single_tokens(lr):
    g = torch.Generator(device="cuda").manual_seed(5)
    batch, dim, N = 140001, 8, 4
    x = torch.randn(batch, dim, generator=g, device="cuda")
    w = torch.randn(dim, 4, generator=g, device="cuda")
    cs = torch.randn(batch, dim, 3, generator=g, device="cuda")
    line = torch.cat([ref.d64(cs), ref.d64(x)[:, :, None]], 2)
    y = lr.sconv_step(x, w, state=cs, silu=False)
    assert lr.get_last_error() == 0
    _close(y, (line * ref.d64(w)).sum(-1), 1e-5)
    assert torch.equal(cs.double().cpu(), line[:, :, 1:])
    delta = torch.rand(batch, dim, generator=g, device="cuda")
    A = -torch.rand(dim, N, generator=g, device="cuda")
    B, C = (torch.randn(batch, N, generator=g, device="cuda") for _ in range(2))
    st = torch.randn(batch, dim, N, generator=g, device="cuda")
    h = torch.exp(ref.d64(delta)[:, :, None] * ref.d64(A)) * ref.d64(st) + ref.d64(delta * x)[:, :, None] * ref.d64(B)[:, None]
    out = lr.sscan_step(x, delta, A, B, C, state=st, delta_bias=torch.zeros(dim, device="cuda"))
    assert lr.get_last_error() == 0
    _close(out, (h * ref.d64(C)[:, None]).sum(-1), 1e-4)
    _close(st, h, 1e-4)


def test_steps_in_a_captured_graph(lr):
    """A decode step's operators capture into a graph (outputs given, after one ordinary call)."""
    g = torch.Generator(device="cuda").manual_seed(6)
    batch, dim, N = 4, 64, 16
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, delta, z, w, A = r(batch, dim), torch.rand(batch, dim, generator=g, device="cuda"), r(batch, dim), r(dim, 4), -r(dim, N).abs()
    B, C, res, nw = r(batch, N), r(batch, N), r(batch, dim), torch.ones(dim, device="cuda")
    slots = torch.tensor([3, -1, 0, 5], dtype=torch.int32, device="cuda")
    cs0, st0 = r(6, dim, 3), r(6, dim, N)
    outs = [torch.empty(batch, dim, device="cuda") for _ in range(5)]

    def step(cs, st, o):
        lr.addnorm_fwd(x, res, nw, out=o[0], residual_out=o[1])
        lr.sconv_step(o[0], w, state=cs, slots=slots, out=o[2])
        lr.sscan_step(o[2], delta, A, B, C, state=st, slots=slots, delta_bias=nw, delta_softplus=True, out=o[3])
        lr.gatenorm_step(o[3], z, nw, out=o[4])

    want = [torch.empty_like(t) for t in outs]
    cs, st = cs0.clone(), st0.clone()
    step(cs, st, want)
    step(cs, st, want)
    cs1, st1 = cs0.clone(), st0.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cs1, st1, outs)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cs, cs1) and torch.equal(st, st1)
    for a, b in zip(want, outs):
        assert torch.equal(a, b)
