"""Norms of queries and keys for each head and their rotation, against 64 bits.

Roundings: the sum of squares of D channels in fp32 is off by D * 2^-24, its root and
reciprocal by a few more; cosines and sines by 2^-22 (position 2^31 included, as their
angles are exact modulo a turn); outputs are rounded once."""
import pytest
import torch

import lattn_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


def make(seed, dtype, batch, qh, kh, dim, rot, L, far=False, offset=0):
    g = torch.Generator().manual_seed(seed)
    both = torch.randn(batch, (qh + kh) * dim, L + offset, generator=g).to(DT[dtype]).cuda()[..., offset:]
    q, k = both[:, :qh * dim], both[:, qh * dim:]
    w = [(torch.randn(dim, generator=g) * 0.2 + 1).cuda() for _ in range(2)]
    freq = (10000.0 ** (-torch.arange(rot, dtype=torch.float32) / max(rot, 1))).cuda() if rot else None
    pos = torch.randint(-5, 2 ** 31 - 1 if far else 70000, (batch, L), generator=g, dtype=torch.int32).cuda() if rot else None
    return q, k, w[0], w[1], pos, freq


def want_fwd(x, w, pos, freq):
    v = ref.d64(x).transpose(1, 2).unflatten(-1, (-1, w.shape[0]))
    return ref.heads_norm(v, ref.d64(w), ref.d64(pos), ref.d64(freq), EPS).flatten(-2).transpose(1, 2)


def close(got, want, mag, io, c, what):
    off = (got.detach().double().cpu() - want).abs()
    worst = float((off / (io * want.abs() + c * mag + 1e-30)).max()) if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of what its roundings allow"


def pair_size(y, dim, rot):
    """The magnitude that a turned channel is made of: both of its pair."""
    v = y.abs().transpose(1, 2).unflatten(-1, (-1, dim))
    out = v.clone()
    if rot:
        out[..., :2 * rot] = (v[..., :rot] + v[..., rot:2 * rot]).repeat(1, 1, 1, 2)
    return out.flatten(-2).transpose(1, 2)


SIZES = [(2, 2, 1, 128, 64, 65), (1, 4, 2, 64, 32, 1), (2, 3, 3, 18, 4, 130), (1, 1, 1, 256, 128, 64), (2, 5, 0, 96, 24, 77),
         (1, 2, 2, 1, 0, 33), (2, 2, 1, 129, 0, 40), (1, 40, 8, 128, 32, 200), (3, 1, 1, 7, 3, 2)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward_and_gradients(lr, dtype, far, size):
    batch, qh, kh, dim, rot, L = size
    q, k, qw, kw, pos, freq = make(dim + L, dtype, batch, qh, kh, dim, rot, L, far, offset=L % 3)
    io = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    c = 2.0 ** -24 * (dim + 16) + (2.0 ** -21 if rot else 0.0)
    if far and rot:
        # the reference's own angle in 64 bits: 2^-53 of up to 2^31 radians, and of the frequency's turn as often
        c += 2.0 ** -20
    ins = (q, k, qw, kw) if kh else (q, None, qw, None)
    qo, ko = lr.qknorm_fwd(*ins, pos, freq, eps=EPS)
    assert lr.get_last_error() == lr.SSCAN_OK
    for x, w, y in ((q, qw, qo), (k, kw, ko)):
        if y is None:
            continue
        want = want_fwd(x, w, pos, freq)
        plain = want_fwd(x, w, pos, None) if not rot else want
        close(y, want, pair_size(plain, dim, rot) * 2, io, c, "out")
    g = torch.Generator().manual_seed(3)
    dqo = torch.randn(q.shape, generator=g).to(DT[dtype]).cuda()
    dko = torch.randn(k.shape, generator=g).to(DT[dtype]).cuda() if kh else None
    got = lr.qknorm_bwd(*ins, dqo, dko, pos, freq, eps=EPS)
    again = lr.qknorm_bwd(*ins, dqo, dko, pos, freq, eps=EPS)
    for x, w, dy, name, wname in ((q, qw, dqo, "dq", "dq_weight"), (k, kw, dko, "dk", "dk_weight")):
        if not kh and name == "dk":
            assert got[name] is None and got[wname] is None
            continue
        a, b = ref.d64(x).transpose(1, 2).unflatten(-1, (-1, dim)).requires_grad_(), ref.d64(w).requires_grad_()
        y = ref.heads_norm(a, b, ref.d64(pos), ref.d64(freq), EPS).flatten(-2).transpose(1, 2)
        da, db = torch.autograd.grad(y, (a, b), ref.d64(dy))
        # dx = rstd (g - n mean(g n)): terms of the pair's gradients and of the whole head's
        up = pair_size(ref.d64(dy), dim, rot).transpose(1, 2).unflatten(-1, (-1, dim))
        xs = a.detach()
        rstd = 1 / torch.sqrt((xs * xs).mean(-1, keepdim=True) + EPS)
        n = (xs * rstd).abs()
        gw = up * b.detach().abs()
        mag = rstd * (gw + n * (gw * n).mean(-1, keepdim=True))
        close(got[name], da.flatten(-2).transpose(1, 2), mag.flatten(-2).transpose(1, 2), io, 4 * c, name)
        close(got[wname], db, (up * n).sum((0, 1, 2)), 2.0 ** -24, 2 * c + 2.0 ** -24 * 256, wname)
        assert torch.equal(got[wname], again[wname]) and torch.equal(got[name], again[name])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_step(lr, dtype, size):
    batch, qh, kh, dim, rot, _ = size
    q, k, qw, kw, pos, freq = make(dim, dtype, batch, qh, kh, dim, rot, 3, far=True)
    io = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    c = 2.0 ** -24 * (dim + 16) + (2.0 ** -21 + 2.0 ** -20 if rot else 0.0)
    rows = torch.cat([q, k], 1).transpose(1, 2).contiguous()[:, 1]  # [batch, channels], a view with row stride
    p1 = None if pos is None else pos[:, 1].contiguous()
    got = lr.qknorm_step(rows[:, :qh * dim], rows[:, qh * dim:] if kh else None, qw, kw if kh else None, p1, freq, eps=EPS)
    for x, w, y in ((q, qw, got[0]), (k, kw, got[1])):
        if y is None:
            continue
        want = want_fwd(x[:, :, 1:2], w, None if pos is None else pos[:, 1:2], freq)
        close(y[..., None], want, pair_size(want, dim, rot) * 2, io, c, "step")


def test_values_that_are_not_finite_stay_in_their_token(lr):
    q, k, qw, kw, pos, freq = make(5, "f32", 1, 2, 1, 64, 32, 100)
    want, _ = lr.qknorm_fwd(q, k, qw, kw, pos, freq)
    x = q.clone()
    x[0, 3, 50] = float("nan")
    x[0, 70, 51] = float("inf")
    got, _ = lr.qknorm_fwd(x, k, qw, kw, pos, freq)
    bad = torch.isnan(got[0])
    assert bad[:64, 50].all() and bad[64:, 51].any()
    bad[:64, 50] = bad[64:, 51] = False
    keep = torch.ones_like(got[0], dtype=torch.bool)
    keep[:64, 50] = keep[64:, 51] = False
    assert not bad.any() and torch.equal(got[0][keep], want[0][keep])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,rot", [(64, 32), (128, 64), (256, 40), (17, 8), (66, 0), (130, 65)])
def test_lengths_and_views(lr, dtype, dim, rot):
    """Every length around a tile of 32 tokens, rows of every alignment, more (tile, head) pairs than CTAs."""
    io = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    c = 2.0 ** -24 * (dim + 16) + (2.0 ** -21 if rot else 0.0)
    for i, L in enumerate((1, 2, 7, 8, 9, 31, 32, 33, 39, 40, 41, 63, 64, 65, 71, 96, 97)):
        batch, qh, kh = (3, 5, 4) if i % 2 else (1, 3, 1)
        q, k, qw, kw, pos, freq = make(L, dtype, batch, qh, kh, dim, rot, L + 3, offset=i % 9)
        q, k = q[..., :L], k[..., :L]
        pos = None if pos is None else pos[:, :L].contiguous()
        # what lies beside the rows is never written, and never counts
        qo, ko = lr.qknorm_fwd(q, k, qw, kw, pos, freq, eps=EPS)
        g = torch.Generator().manual_seed(L)
        do = [torch.randn(x.shape, generator=g).to(DT[dtype]).cuda() for x in (q, k)]
        got = lr.qknorm_bwd(q, k, qw, kw, *do, pos, freq, eps=EPS)
        for x, w, y, dy, name in ((q, qw, qo, do[0], "dq"), (k, kw, ko, do[1], "dk")):
            want = want_fwd(x, w, pos, freq)
            close(y, want, pair_size(want, dim, rot) * 2, io, c, "out")
            a, b = ref.d64(x).transpose(1, 2).unflatten(-1, (-1, dim)).requires_grad_(), ref.d64(w).requires_grad_()
            z = ref.heads_norm(a, b, ref.d64(pos), ref.d64(freq), EPS).flatten(-2).transpose(1, 2)
            da, db = torch.autograd.grad(z, (a, b), ref.d64(dy))
            up = pair_size(ref.d64(dy), dim, rot).transpose(1, 2).unflatten(-1, (-1, dim))
            xs = a.detach()
            rstd = 1 / torch.sqrt((xs * xs).mean(-1, keepdim=True) + EPS)
            n = (xs * rstd).abs()
            gw = up * b.detach().abs()
            mag = rstd * (gw + n * (gw * n).mean(-1, keepdim=True))
            close(got[name], da.flatten(-2).transpose(1, 2), mag.flatten(-2).transpose(1, 2), io, 4 * c, name)
            close(got[name + "_weight"], db, (up * n).sum((0, 1, 2)), 2.0 ** -24, 2 * c + 2.0 ** -24 * 256, name + "_weight")
    assert lr.get_last_error() == lr.SSCAN_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_units(lr, dtype):
    """Runs of heads that pass from queries to keys and from tile to tile within a CTA."""
    q, k, qw, kw, pos, freq = make(8, dtype, 3, 24, 8, 64, 32, 1001)
    do = [torch.randn_like(x.contiguous()) for x in (q, k)]
    qo, ko = lr.qknorm_fwd(q, k, qw, kw, pos, freq, eps=EPS)
    got = lr.qknorm_bwd(q, k, qw, kw, *do, pos, freq, eps=EPS)
    for b in range(3):
        one = [x[b:b + 1] for x in (q, k)]
        for t0 in (0, 500, 970):  # any stretch by itself gives the same bits
            cut = [x[..., t0:t0 + 31] for x in one]
            y = lr.qknorm_fwd(*cut, qw, kw, pos[b:b + 1, t0:t0 + 31].contiguous(), freq, eps=EPS)
            assert torch.equal(y[0], qo[b:b + 1, :, t0:t0 + 31]) and torch.equal(y[1], ko[b:b + 1, :, t0:t0 + 31])
            z = lr.qknorm_bwd(*cut, qw, kw, *[x[b:b + 1, :, t0:t0 + 31].contiguous() for x in do], pos[b:b + 1, t0:t0 + 31].contiguous(), freq, eps=EPS)
            assert torch.equal(z["dq"], got["dq"][b:b + 1, :, t0:t0 + 31]) and torch.equal(z["dk"], got["dk"][b:b + 1, :, t0:t0 + 31])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_graphs_and_streams(lr, dtype):
    """Two captured graphs and two streams at once: each call has its own workspace."""
    sets = [make(20 + i, dtype, 2, 6, 2, 64, 32, 333 + i) for i in range(2)]
    dos = [[torch.randn_like(x.contiguous()) for x in s[:2]] for s in sets]

    def both(i):
        q, k, qw, kw, pos, freq = sets[i]
        g = lr.qknorm_bwd(q, k, qw, kw, *dos[i], pos, freq, eps=EPS)
        return [*lr.qknorm_fwd(q, k, qw, kw, pos, freq, eps=EPS), *g.values()]

    want = [both(i) for i in range(2)]
    torch.cuda.synchronize()
    streams, graphs = [torch.cuda.Stream() for _ in range(2)], []
    got = []
    for i, st in enumerate(streams):
        with torch.cuda.stream(st):
            got.append(both(i))
    torch.cuda.synchronize()
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = both(i)
        graphs.append((graph, outs))
    for _ in range(2):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                graphs[i][0].replay()
    torch.cuda.synchronize()
    for i in range(2):
        for a, b, c in zip(want[i], got[i], graphs[i][1]):
            assert torch.equal(a, b) and torch.equal(a, c)
