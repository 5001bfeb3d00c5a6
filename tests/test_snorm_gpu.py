"""GPU parity of the fused norms with their 64-bit forms.

Tolerances.  A norm over n values sums n squares in fp32, pairwise over lanes
and sequentially over at most 64 a lane: relative error below 1e-5 of the sum,
half of that in its root; the products add a few 2^-24.  Outputs: 1e-5 of the
value's magnitude; gradients 1e-5 of the magnitude of the terms they
subtract; bf16 adds its rounding, 2^-8 of the value (half an ulp is 2^-9).
Weight gradients sum T terms: 2e-5 of their magnitudes."""
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


def _near(got, want, size, dtype, k=1e-5):
    got = got.double().cpu()
    tol = k * (size + want.abs()) + 1e-7
    if dtype == "bf16":
        tol = tol + want.abs() * 2.0 ** -8
    bad = (got - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / tol).max()))
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (2, 64), (5, 100), (700, 24), (2, 2561), (3, 2560), (2, 8200), (1, 16384), (1, 16383)])
@pytest.mark.parametrize("first", [False, True])
def test_addnorm(lr, dtype, rows, width, first):
    g = torch.Generator().manual_seed(rows + width)
    x = torch.randn(rows, width, generator=g).to(IO[dtype])
    res = None if first else torch.randn(rows, width, generator=g) * 2
    w = 1 + 0.1 * torch.randn(width, generator=g)
    dy = torch.randn(rows, width, generator=g).to(IO[dtype])
    dr = None if first else torch.randn(rows, width, generator=g)
    scale, eps = 0.37, 1e-5
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    y, r = lr.addnorm_fwd(x.cuda(), cu(res), w.cuda(), scale=scale, eps=eps)
    got = lr.addnorm_bwd(r, w.cuda(), dy.cuda(), cu(dr), scale=scale, eps=eps)
    again = lr.addnorm_bwd(r, w.cuda(), dy.cuda(), cu(dr), scale=scale, eps=eps)
    assert lr.get_last_error() == 0

    xs, ws = ref.d64(x).requires_grad_(), ref.d64(w).requires_grad_()
    rs = (torch.zeros(rows, width, dtype=torch.float64) if first else ref.d64(res)).requires_grad_()
    yr, rr = ref.addnorm(xs, rs, ws, scale, eps)
    total = (yr * ref.d64(dy)).sum() + (0 if first else (rr * ref.d64(dr)).sum())
    dx, dres, dw = torch.autograd.grad(total, (xs, rs, ws))
    yr, rr = yr.detach(), rr.detach()
    _near(y, yr, yr.abs(), dtype)
    _near(r, rr, rr.abs(), "f32", 1e-6)
    rstd = 1 / torch.sqrt((rr * rr).mean(-1, keepdim=True) + eps)
    q = (ref.d64(dy) * ref.d64(w)).abs()
    n = (rr * rstd).abs()
    size = rstd * (q + n * (q * n).mean(-1, keepdim=True)) + (0 if first else ref.d64(dr).abs())
    _near(got["dresidual"], dres, size, "f32")
    _near(got["dx"], dx, scale * size, dtype)
    _near(got["dweight"], dw, (ref.d64(dy).abs() * n).sum(0), "f32", 2e-5)
    for k in got:
        assert torch.equal(got[k], again[k]), k


def test_addnorm_in_place_and_other_stream(lr):
    g = torch.Generator().manual_seed(1)
    x, res = torch.randn(9, 640, generator=g).bfloat16(), torch.randn(9, 640, generator=g)
    w = torch.ones(640)
    r, xd, wd = res.cuda(), x.cuda(), w.cuda()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        y, same = lr.addnorm_fwd(xd, r, wd, residual_out=r)
    st.synchronize()
    yr, rr = ref.addnorm(ref.d64(x), ref.d64(res), ref.d64(w), 1.0, 1e-5)
    assert same is r
    _near(y, yr, yr.abs(), "bf16")
    _near(r, rr, rr.abs(), "f32", 1e-6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,dim,L", [(1, 1, 1), (2, 6, 7), (1, 64, 32), (3, 130, 33), (2, 96, 40), (1, 2000, 64), (2, 512, 257), (1, 5120, 16)])
@pytest.mark.parametrize("groups", [1, 2])
@pytest.mark.parametrize("norm_first", [False, True])
@pytest.mark.parametrize("view", [False, True])
def test_gatenorm(lr, dtype, batch, dim, L, groups, norm_first, view):
    if dim % groups:
        pytest.skip("groups divide the channels")
    g = torch.Generator().manual_seed(dim + L)
    y = torch.randn(batch, dim, L, generator=g).to(IO[dtype])
    z = torch.randn(batch, 2 * dim, L, generator=g).to(IO[dtype]).cuda()
    z = z[:, dim:] if view else z[:, :dim].contiguous()
    w = 1 + 0.1 * torch.randn(dim, generator=g)
    do = torch.randn(batch, dim, L, generator=g).to(IO[dtype])
    kw = dict(groups=groups, norm_first=norm_first, eps=1e-5)
    out = lr.gatenorm_fwd(y.cuda(), z, w.cuda(), **kw)
    got = lr.gatenorm_bwd(y.cuda(), z, w.cuda(), do.cuda(), **kw)
    again = lr.gatenorm_bwd(y.cuda(), z, w.cuda(), do.cuda(), **kw)
    assert lr.get_last_error() == 0

    ys, zs, ws = (ref.d64(t).requires_grad_() for t in (y, z, w))
    outr = ref.gatenorm(ys, zs, ws, groups, norm_first, 1e-5)
    dy, dz, dw = torch.autograd.grad((outr * ref.d64(do)).sum(), (ys, zs, ws))
    outr = outr.detach()
    _near(out, outr, outr.abs(), dtype)
    with torch.no_grad():
        gate = ref.silu(zs)
        sig = 1 / (1 + torch.exp(-zs))
        slope = (sig * (1 + zs * (1 - sig))).abs()
        v = (ys if norm_first else ys * gate).unflatten(1, (groups, -1))
        rstd = 1 / torch.sqrt((v * v).mean(2, keepdim=True) + 1e-5)
        n = (v * rstd).abs()
        up = (ref.d64(do) * (gate if norm_first else 1)).abs()
        q = (up * ref.d64(w)[:, None]).unflatten(1, (groups, -1))
        dv = (rstd * (q + n * (q * n).mean(2, keepdim=True))).flatten(1, 2)
        n = n.flatten(1, 2)
        size_y = dv if norm_first else dv * gate.abs()
        size_z = (ref.d64(do).abs() * n * ref.d64(w)[:, None].abs() if norm_first else dv * ys.abs()) * slope
        # silu' near its zero is a difference of terms of size sigmoid * (1 + |z|)
        size_z = size_z + (dv * ys.abs() + ref.d64(do).abs() * n) * sig * (1 + zs.abs()) * 0.1
    _near(got["dy"], dy, size_y, dtype)
    _near(got["dz"], dz, size_z, dtype)
    _near(got["dweight"], dw, (up * n).sum((0, 2)), "f32", 2e-5)
    for k in got:
        assert torch.equal(got[k], again[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim,groups", [(1, 1, 1), (3, 7, 1), (5, 96, 3), (9, 5120, 1), (300, 64, 2), (2, 5122, 2), (1, 16384, 1), (2, 4098, 1)])
@pytest.mark.parametrize("norm_first", [False, True])
def test_gatenorm_step(lr, dtype, rows, dim, groups, norm_first):
    g = torch.Generator().manual_seed(rows + dim)
    y = torch.randn(rows, dim, generator=g).to(IO[dtype])
    z = torch.randn(rows, 2 * dim, generator=g).to(IO[dtype]).cuda()[:, dim:]
    w = 1 + 0.1 * torch.randn(dim, generator=g)
    out = lr.gatenorm_step(y.cuda(), z, w.cuda(), groups=groups, norm_first=norm_first)
    assert lr.get_last_error() == 0 and lr.last_launch_count() == 1
    want = ref.gatenorm(ref.d64(y), ref.d64(z), ref.d64(w), groups, norm_first, 1e-5)
    _near(out, want, want.abs(), dtype)


@pytest.mark.parametrize("norm_first", [False, True])
def test_gradients_against_differences(lr, norm_first):
    """The gradients predict the forwards' change along random directions (64-bit central differences)."""
    g = torch.Generator().manual_seed(8)
    t = {"y": torch.randn(2, 12, 5, generator=g), "z": torch.randn(2, 12, 5, generator=g),
         "weight": torch.randn(12, generator=g)}
    do = torch.randn(2, 12, 5, generator=g)
    got = lr.gatenorm_bwd(t["y"].cuda(), t["z"].cuda(), t["weight"].cuda(), do.cuda(), groups=3, norm_first=norm_first)

    def gate(v):
        return float((ref.gatenorm(v["y"], v["z"], v["weight"], 3, norm_first, 1e-5) * do.double()).sum())

    a = {"x": torch.randn(4, 10, generator=g), "residual": torch.randn(4, 10, generator=g), "weight": torch.randn(10, generator=g)}
    dy, dr = torch.randn(4, 10, generator=g), torch.randn(4, 10, generator=g)
    _, r = lr.addnorm_fwd(a["x"].cuda(), a["residual"].cuda(), a["weight"].cuda(), scale=0.5)
    got2 = lr.addnorm_bwd(r, a["weight"].cuda(), dy.cuda(), dr.cuda(), scale=0.5)

    def add(v):
        y, r = ref.addnorm(v["x"], v["residual"], v["weight"], 0.5, 1e-5)
        return float((y * dy.double()).sum() + (r * dr.double()).sum())

    for ins, grads, value in ((t, got, gate), (a, got2, add)):
        for name in ins:
            way = torch.randn(ins[name].shape, generator=g, dtype=torch.float64)
            hi, lo = ({k: v.double() for k, v in ins.items()} for _ in range(2))
            hi[name], lo[name] = hi[name] + 1e-5 * way, lo[name] - 1e-5 * way
            slope = (value(hi) - value(lo)) / 2e-5
            mine = float((grads["d" + name].double().cpu() * way).sum())
            assert abs(mine - slope) <= 1e-4 * (1 + abs(slope)), name


def test_empty_and_masked_rows(lr):
    """No rows; a row of zeros (its norm is eps alone); infinities and NaN stay in their own token."""
    w = torch.ones(8).cuda()
    g = lr.addnorm_bwd(torch.empty(0, 8).cuda(), w, torch.empty(0, 8).cuda())
    out = lr.gatenorm_fwd(torch.empty(2, 8, 0).cuda(), torch.empty(2, 8, 0).cuda(), w)
    gg = lr.gatenorm_bwd(torch.empty(2, 8, 0).cuda(), torch.empty(2, 8, 0).cuda(), w, torch.empty(2, 8, 0).cuda())
    torch.cuda.synchronize()
    assert not g["dweight"].any() and out.shape == (2, 8, 0) and not gg["dweight"].any()
    y, r = lr.addnorm_fwd(torch.zeros(3, 8).cuda(), None, w)
    torch.cuda.synchronize()
    assert not y.any() and not r.any()
    y = torch.randn(1, 8, 45).cuda()
    z = torch.randn(1, 8, 45).cuda()
    clean = lr.gatenorm_fwd(y, z, w)
    y[0, 3, 7], z[0, 2, 40] = float("nan"), float("inf")
    dirty = lr.gatenorm_fwd(y, z, w)
    torch.cuda.synchronize()
    keep = [t for t in range(45) if t not in (7, 40)]
    assert torch.equal(clean[..., keep], dirty[..., keep]) and torch.isnan(dirty[..., 7]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,width", [(5000, 33), (300, 1023), (300, 1025), (3, 2049), (2, 4095), (2, 4097), (700, 5001),
                                        (500, 4864), (40, 4104), (9, 6144)])
def test_addnorm_rows_of_every_plan(lr, dtype, rows, width):
    """Widths around each change of vectors a thread, and weight gradients summed over many partial rows."""
    test_addnorm(lr, dtype, rows, width, False)


def test_addnorm_in_place_odd_rows(lr):
    g = torch.Generator().manual_seed(12)
    x, res = torch.randn(7, 2049, generator=g).bfloat16(), torch.randn(7, 2049, generator=g)
    w = 1 + 0.1 * torch.randn(2049, generator=g)
    r, xd = res.cuda(), x.cuda()
    y, same = lr.addnorm_fwd(xd, r, w.cuda(), residual_out=r, out=xd)
    assert same is r and y is xd
    yr, rr = ref.addnorm(ref.d64(x), ref.d64(res), ref.d64(w), 1.0, 1e-5)
    _near(y, yr, yr.abs(), "bf16")
    _near(r, rr, rr.abs(), "f32", 1e-6)
