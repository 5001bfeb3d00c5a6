"""How exact linear attention is where its other tests allow much: by the norm of what is off.

Their bounds follow the sum of a chunk's exponents, or of all its terms' magnitudes.  Here inputs are
random, so that a sum of K terms of either sign is about sqrt(K) of one, and so is what their roundings add up
to: what a sum is off by, relative to it, is what a term is off by, whatever K."""
import pytest
import torch

import lattn_reference as ref
from test_lattn_gpu import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


def off(got, want):
    return float((got.detach().double().cpu() - want).norm() / want.norm())


def mixed_steps(kind, heads, L, g):
    """Rates and steps of which only differences between neighbours count, beside sums of hundreds."""
    if kind == "spread":  # steps from 0.02 to 3
        return -16.0, torch.exp(torch.rand(1, heads, L, generator=g) * 5.0106 - 3.912)
    steps = torch.full((1, heads, L), 0.02)
    steps[..., ::5] = 10.0
    return -8.0, steps


# The exponent is rounded three times, each by 2^-24 of itself, x e^-x at most 0.37; the exponent unit adds 2^-22 of a
# factor, the sums of 64 products and of 64 tokens some 2^-22: 2^-21 in all, twice that allowed.
@pytest.mark.parametrize("kind", ["spread", "long"])
@pytest.mark.parametrize("packed", [False, True], ids=["batch", "packed"])
def test_fp32_forward_of_fast_decays(lr, kind, packed):
    heads, value, key, L = 4, 32, 64, 333
    f = make(5, "f32", 1, heads, 1, value, key, L, D=False, s0=False)
    rate, steps = mixed_steps(kind, heads, L, torch.Generator().manual_seed(3))
    A, steps = torch.full((heads,), rate, device="cuda"), steps.cuda()
    cut = [0, 150, 333] if packed else [0, L]
    got, last = [], []
    if packed:
        state = torch.zeros(2, heads * value, key, device="cuda")
        o = lr.lattn_prompt(f["q"][0], f["k"][0], f["v"][0], A, steps[0], cu_seqlens=torch.tensor(cut, dtype=torch.int32, device="cuda"), state=state,
                            scale=0.125)[None]
        last = [state[:1], state[1:]]
    else:
        o, s = lr.lattn_fwd(f["q"], f["k"], f["v"], A, steps, scale=0.125)
        last = [s]
    for a, b, s in zip(cut, cut[1:], last):
        part = [x[..., a:b] for x in (f["q"], f["k"], f["v"])]
        want = ref.forward(*part, A, steps[..., a:b], None, None, 1, 0.125)
        got = o[..., a:b].unflatten(1, (heads, value))
        for h in range(heads):
            assert off(got[:, h], want[0].unflatten(1, (heads, value))[:, h]) <= 2.0 ** -20, ("o", h)
        assert off(s, want[1]) <= 2.0 ** -20, "state"
    assert lr.get_last_error() == lr.SSCAN_OK
