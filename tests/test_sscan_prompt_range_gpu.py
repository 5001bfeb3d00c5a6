"""The packed scan over values of very different sizes: what a split carries
over its borders, and what it leaves out.

Tolerances are those of the packed scan's other tests, 1e-4 (1 + |y|).  Outputs
are compared from where a large value has decayed by 2^-80 or more, so that
nothing of it is left in them."""
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


def _near(got, want, tol):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    err = float(((got - want).abs() / (1 + want.abs())).max())
    assert err <= tol, err


def _call(lr, x, cu, state, segments):
    c = {k: v.cuda() for k, v in x.items()}
    got = state.cuda()
    y = lr.sscan_prompt(c["u"], c["delta"], c["A"], c["B"], c["C"], cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
                        state=got, segments=segments)
    assert lr.get_last_error() == 0
    return y, got


def _want(x, cu, state):
    d = {k: ref.d64(v) for k, v in x.items()}
    y, after, _ = ref.scan_packed(d["u"], d["delta"], d["A"], d["B"], d["C"], None, cu, None, None, ref.d64(state))
    return y, after


def _inputs(dim, tokens, N, seed):
    g = torch.Generator().manual_seed(seed)
    return {"u": torch.randn(dim, tokens, generator=g), "delta": torch.full((dim, tokens), 0.5),
            "A": -torch.ones(dim, N), "B": torch.randn(N, tokens, generator=g), "C": torch.randn(N, tokens, generator=g)}


@pytest.mark.parametrize("segments", [1, 2, 4])
@pytest.mark.parametrize("tokens", [512, 515])
@pytest.mark.parametrize("N", [3, 16, 64])
def test_a_large_initial_state_decays_before_a_border(lr, segments, tokens, N):
    """Half a nat a token: an initial state of 1e12 is gone 128 tokens later, whatever the split."""
    x = _inputs(40, tokens, N, 1)
    state = torch.full((1, 40, N), 1e12)
    y, after = _call(lr, x, [0, tokens], state, segments)
    yr, ar = _want(x, [0, tokens], state)
    _near(y[:, 128:], yr[:, 128:], 1e-4)
    _near(after, ar, 1e-4)


@pytest.mark.parametrize("segments", [1, 4])
@pytest.mark.parametrize("tokens", [512, 515])
def test_a_large_input_decays_over_a_segment(lr, segments, tokens):
    """An input of 1e14 just before the first border, seen by fast states only; slow
    states beside them keep the composition of earlier segments going."""
    dim, N = 40, 16
    x = _inputs(dim, tokens, N, 2)
    x["A"][:, :4] = -1e-4
    x["u"][:, 120] = 1e14
    x["B"][:4, 120] = 0.0
    state = torch.zeros(1, dim, N)
    y, after = _call(lr, x, [0, tokens], state, segments)
    yr, ar = _want(x, [0, tokens], state)
    _near(y[:, 256:], yr[:, 256:], 1e-4)
    _near(after, ar, 1e-4)
