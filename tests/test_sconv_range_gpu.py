"""The short convolution at the ends of its types' range: sums c near the
largest values, whose sigmoid is 0 or 1, and infinities at a sequence's ends.

Tolerances are those of the convolution's other tests.  silu(c) is c or 0 here,
and its slope 1 or 0, both exact."""
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu
IO = {"f32": torch.float32, "bf16": torch.bfloat16}
LARGE = [-3.38e38, 3.38e38, -2.5e38, 2.5e38, -1e38, 1e38, -3e37]


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


def _large(dtype, batch, dim, L):
    """Ordinary inputs with the large ones among them, and at both ends of a row."""
    g = torch.Generator().manual_seed(L)
    x = torch.randn(batch, dim, L, generator=g)
    for i, v in enumerate(LARGE):
        x[..., i * 97 % L] = v
    x[..., -1] = LARGE[0]
    return x.to(IO[dtype]), g


def _near(got, want, dtype):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    tol = 2e-6 * (1 + want.abs()) + (want.abs() * 2.0 ** -8 if dtype == "bf16" else 0)
    assert bool(((got - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [5, 700, 701])
@pytest.mark.parametrize("width", [2, 4])
def test_sums_near_the_largest_values(lr, dtype, L, width):
    """One tap of weight one: c is x, as large as the type allows."""
    batch, dim = 2, 9
    x, g = _large(dtype, batch, dim, L)
    w = torch.zeros(dim, width)
    w[:, -1] = 1.0
    dy = torch.randn(batch, dim, L, generator=g).to(IO[dtype])
    y, _ = lr.sconv_fwd(x.cuda(), w.cuda())
    packed = lr.sconv_prompt(x[0].contiguous().cuda(), w.cuda(), cu_seqlens=torch.tensor([0, L], dtype=torch.int32).cuda(),
                             state=torch.zeros(1, dim, width - 1, dtype=IO[dtype]).cuda())
    got = lr.sconv_bwd(x.cuda(), w.cuda(), None, None, dy.cuda())
    assert lr.get_last_error() == 0
    c = ref.d64(x)
    s = 1 / (1 + torch.exp(-c))
    _near(y, c * s, dtype)
    _near(packed, (c * s)[0], dtype)
    _near(got["dx"], ref.d64(dy) * s * (1 + c * (1 - s)), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [3, 40, 700])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_value_that_is_not_finite_stays_in_its_taps(lr, dtype, L, value):
    """The last input meets the last tap alone, the one before the first all taps but the last."""
    g = torch.Generator().manual_seed(L)
    dim, width = 5, 4
    x = torch.randn(2, dim, L, generator=g).to(IO[dtype])
    x0 = torch.randn(2, dim, width - 1, generator=g).to(IO[dtype])
    w = torch.randn(dim, width, generator=g)
    dy = torch.randn(2, dim, L, generator=g).to(IO[dtype])
    for at, spoiled in (("last", [3]), ("before", [0, 1, 2])):
        xs, bs = x.clone(), x0.clone()
        (xs if at == "last" else bs)[0, :, -1] = value
        got = lr.sconv_bwd(xs.cuda(), w.cuda(), None, bs.cuda(), dy.cuda(), silu=False)["dweight"].double().cpu()
        line = torch.cat([ref.d64(bs), ref.d64(xs)], 2)
        want = torch.stack([(ref.d64(dy) * line[..., k:k + L]).sum((0, 2)) for k in range(width)], 1)
        size = torch.stack([(ref.d64(dy) * line[..., k:k + L]).abs().sum((0, 2)) for k in range(width)], 1)
        clean = [k for k in range(width) if k not in spoiled]
        assert torch.isfinite(want[:, clean]).all() and not torch.isfinite(want[:, spoiled]).any()
        assert bool(((got - want)[:, clean].abs() <= 1e-5 * size[:, clean] + 1e-7).all()), at
        assert not torch.isfinite(got[:, spoiled]).any()
