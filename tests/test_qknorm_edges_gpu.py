"""Norms of queries and keys at the ends of what they take: no epsilon, against 64 bits, and angles of far positions
at large frequencies, against exact integers.

Tolerances count roundings as in test_qknorm_gpu.py."""
import math
from fractions import Fraction

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


# 1 / (2 pi) to 84 digits
PER_RADIAN = Fraction("0.159154943091895335768883763372514362034459645740456448747667344058896797634226535090")


def turned(freq, pos):
    """cos and sin of pos * freq, the angle modulo a turn in exact arithmetic."""
    turns = Fraction(freq) * pos * PER_RADIAN
    angle = float(turns - math.floor(turns + Fraction(1, 2))) * 2 * math.pi
    return math.cos(angle), math.sin(angle)


FREQUENCIES = [(1.0, 100.0, 1e4, -3.7), (1e6, 3e-5, -1e5, 0.5), (-1.0, -1e-3, 2.0 ** 30, 6.2831855), (1e-10, -2e-9, 123.456, 2.0 ** 44)]


# Angles are rounded to 2^-32 of a turn, then to fp32 (2^-24 of at most pi), cosines and sines are off by
# 2^-22, and the norm's four roundings come on top: 6e-7.
@pytest.mark.parametrize("freqs", FREQUENCIES, ids=str)
def test_angles_of_far_positions(lr, freqs):
    r, places = len(freqs), [0, 1, -1, 7, 12345, 500_000, 2 ** 30 + 1, 2 ** 31 - 1, -2 ** 31, -2 ** 31 + 3, 1_999_999_973]
    freq = torch.tensor(freqs, device="cuda")
    pos = torch.tensor(places, dtype=torch.int32, device="cuda")
    want = torch.zeros(2 * r, len(places), dtype=torch.float64)
    for i, f in enumerate(freq.tolist()):
        for t, p in enumerate(places):
            want[i, t], want[r + i, t] = turned(f, p)
    # heads of ones and zeros: what is turned by an angle is its cosine and sine
    q = torch.cat([torch.ones(r, len(places)), torch.zeros(r, len(places))]).cuda()
    w = torch.full((2 * r,), 0.5 ** 0.5, device="cuda")
    got, _ = lr.qknorm_fwd(q[None], None, w, None, pos[None], freq, eps=0.0)
    assert float((got[0].double().cpu() - want).abs().max()) <= 2.0 ** -20
    step, _ = lr.qknorm_step(q.t().contiguous(), None, w, None, pos, freq, eps=0.0)
    assert float((step.t().double().cpu() - want).abs().max()) <= 2.0 ** -20
    # upstream gradients are turned back: those of outputs along the turned heads lie along the heads, where the norm has none
    back = lr.qknorm_bwd(q[None], None, w, None, want.float().cuda()[None], None, pos[None], freq, eps=0.0)
    assert float(back["dq"][0, r:].abs().max()) <= 2.0 ** -19 and float(back["dq"][0, :r].abs().max()) <= 2.0 ** -19
