"""Norms of queries and keys at the ends of what they take: no epsilon, against 64 bits.

Tolerances count roundings as in test_qknorm_gpu.py."""
import pytest
import torch

import lattn_reference as ref
from test_qknorm_gpu import DT, close, make, pair_size

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,rot", [(64, 32), (128, 64), (130, 65), (17, 8), (1, 0)])
@pytest.mark.parametrize("L", [1, 5, 31, 32, 33, 45, 200])
def test_no_epsilon(lr, dtype, dim, rot, L):
    """eps = 0: a norm of tokens that are there is finite, whatever lies behind the last of them."""
    q, k, qw, kw, pos, freq = make(dim + L, dtype, 2, 3, 1, dim, rot, L, offset=L % 3)
    io = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    c = 2.0 ** -24 * (dim + 16) + (2.0 ** -21 if rot else 0.0)
    out = lr.qknorm_fwd(q, k, qw, kw, pos, freq, eps=0.0)
    g = torch.Generator().manual_seed(L)
    do = [torch.randn(x.shape, generator=g).to(DT[dtype]).cuda() for x in (q, k)]
    got = lr.qknorm_bwd(q, k, qw, kw, *do, pos, freq, eps=0.0)
    for x, w, y, dy, name in ((q, qw, out[0], do[0], "dq"), (k, kw, out[1], do[1], "dk")):
        a, b = ref.d64(x).transpose(1, 2).unflatten(-1, (-1, dim)).requires_grad_(), ref.d64(w).requires_grad_()
        z = ref.heads_norm(a, b, ref.d64(pos), ref.d64(freq), 0.0).flatten(-2).transpose(1, 2)
        da, db = torch.autograd.grad(z, (a, b), ref.d64(dy))
        want = z.detach()
        assert want.isfinite().all() and db.isfinite().all()
        close(y, want, pair_size(want, dim, rot) * 2, io, c, "out")
        up = pair_size(ref.d64(dy), dim, rot).transpose(1, 2).unflatten(-1, (-1, dim))
        xs = a.detach()
        rstd = 1 / torch.sqrt((xs * xs).mean(-1, keepdim=True))
        n = (xs * rstd).abs()
        gw = up * b.detach().abs()
        mag = rstd * (gw + n * (gw * n).mean(-1, keepdim=True))
        close(got[name], da.flatten(-2).transpose(1, 2), mag.flatten(-2).transpose(1, 2), io, 4 * c, name)
        close(got[name + "_weight"], db, (up * n).sum((0, 1, 2)), 2.0 ** -24, 2 * c + 2.0 ** -24 * 256, name + "_weight")
    assert lr.get_last_error() == lr.SSCAN_OK
