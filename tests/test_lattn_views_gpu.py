"""Linear attention and the norms of its queries and keys on views: broadcast along batches, heads and channels
(strides of zero), and batches inside the channels.  The bits are those of contiguous copies."""
import pytest
import torch

from test_lattn_gpu import DT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


def views(kind, batch, channels, L, io, g):
    if kind == "batch":  # one set of rows for all batches
        return torch.randn(1, channels, L, generator=g).to(io).cuda().expand(batch, channels, L)
    if kind == "channels":  # one row for all channels
        return torch.randn(batch, 1, L, generator=g).to(io).cuda().expand(batch, channels, L)
    if kind == "inside":  # [channels, batch, L]
        return torch.randn(channels, batch, L, generator=g).to(io).cuda().transpose(0, 1)
    return torch.randn(batch, channels, L, generator=g).to(io).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["batch", "channels", "inside"])
@pytest.mark.parametrize("which", ["q", "k", "v", "delta", "all"])
@pytest.mark.parametrize("L", [1, 136, 200, 203])
def test_linear_attention(lr, dtype, kind, which, L):
    heads, groups, value, key, batch = 4, 2, 64, 32, 3
    g, io = torch.Generator().manual_seed(L), DT[dtype]
    x = {n: views(kind if which in (n, "all") else "", batch, c, L, io, g)
         for n, c in (("q", groups * key), ("k", groups * key), ("v", heads * value), ("delta", heads))}
    A, D, bias = (-(torch.rand(heads, generator=g) * 15 + 1)).cuda(), torch.randn(heads, generator=g).cuda(), (torch.randn(heads, generator=g) - 2).cuda()
    do = torch.randn(batch, heads * value, L, generator=g).to(io).cuda()

    def run(x):
        options = dict(groups=groups, scale=0.2, delta_bias=bias, delta_softplus=True)
        grads = lr.lattn_bwd(x["q"], x["k"], x["v"], A, x["delta"], D, None, do, **options)
        return [*lr.lattn_fwd(x["q"], x["k"], x["v"], A, x["delta"], D, pieces=2, **options), *(t for t in grads.values() if t is not None)]

    for a, b in zip(run(x), run({n: t.contiguous() for n, t in x.items()})):
        assert torch.equal(a, b)
    assert lr.get_last_error() == lr.SSCAN_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["batch", "channels", "inside"])
@pytest.mark.parametrize("L", [1, 64, 77])
def test_norms(lr, dtype, kind, L):
    dim, batch = 64, 3
    g, io = torch.Generator().manual_seed(L), DT[dtype]
    q, k = views(kind, batch, 3 * dim, L, io, g), views(kind, batch, dim, L, io, g)
    w, freq = torch.rand(dim, generator=g).cuda(), torch.rand(dim // 2, generator=g).cuda()
    pos = torch.randint(0, 5000, (batch, L), generator=g, dtype=torch.int32).cuda()
    dq, dk = (torch.randn(x.shape, generator=g).to(io).cuda() for x in (q, k))

    def run(q, k):
        return [*lr.qknorm_fwd(q, k, w, w, pos, freq), *lr.qknorm_bwd(q, k, w, w, dq, dk, pos, freq).values()]

    for a, b in zip(run(q, k), run(q.contiguous(), k.contiguous())):
        assert torch.equal(a, b)
    assert lr.get_last_error() == lr.SSCAN_OK
