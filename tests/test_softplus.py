"""The softplus of the packed scan and the cached step.

Bound, relative to the result, for x < 0: the polynomial's coefficients 9.4e-8
(pinned below in 64 bits), nine fused steps and the product 2e-7, the
exponential unit 2^-22, and the exponent's rounding: x log2 e is off by 2^-24
of itself and log2 e in fp32 by 1.3e-8, which e = 2^t turns into 7.3e-8 |x|.
Together 6e-7 + 7.4e-8 |x|; above zero the result is larger still."""
import os
import re

import numpy as np
import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_recurrence_gb300", "csrc")


def _coefficients():
    with open(os.path.join(CSRC, "block_utils.cuh"), encoding="utf-8") as f:
        text = f.read()
    body = text[text.index("float softplus_f32"):]
    body = body[:body.index("return")]
    return [float(np.float32(v)) for v in re.findall(r"(-?\d+\.\d{8,})f\b", body)]


def test_polynomial_is_as_close_as_stated():
    c = _coefficients()
    assert len(c) == 9
    e = np.concatenate([np.logspace(-12, -3, 2000), np.linspace(1e-3, 1, 400001)])
    p = np.zeros_like(e)
    for k in c:
        p = p * e + k
    off = np.max(np.abs(p * e / np.log1p(e) - 1))
    assert 9.2e-8 < off < 9.4e-8, off


@pytest.mark.gpu
def test_steps_are_as_close_as_stated():
    """A state that starts at zero and forgets nothing holds the step size itself: y = h = dt."""
    import linear_recurrence_gb300 as lr
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.rand(4000, generator=g) * span + low for low, span in ((-80, 60), (-20, 20), (-1, 2), (0, 80))])
    n = x.numel()
    one, want = torch.ones(1, n), torch.log1p(torch.exp(-x.double().abs())) + x.double().clamp(min=0)
    bound = want * (6e-7 + 7.4e-8 * x.double().abs())
    y = lr.sscan_step(one.cuda(), x[None].cuda(), torch.zeros(n, 1).cuda(), torch.ones(1, 1).cuda(), torch.ones(1, 1).cuda(),
                      state=torch.zeros(1, n, 1).cuda(), delta_bias=torch.zeros(n).cuda(), delta_softplus=True)
    assert lr.get_last_error() == 0
    assert bool(((y[0].double().cpu() - want).abs() <= bound).all())
    state = torch.zeros(1, n, 1).cuda()
    y = lr.sscan_prompt(one.t().contiguous().cuda(), x[:, None].contiguous().cuda(), torch.zeros(n, 1).cuda(), torch.ones(1, 1).cuda(),
                        torch.ones(1, 1).cuda(), cu_seqlens=torch.tensor([0, 1], dtype=torch.int32).cuda(), state=state,
                        delta_softplus=True)
    assert lr.get_last_error() == 0
    assert bool(((y[:, 0].double().cpu() - want).abs() <= bound).all())
    assert torch.equal(state.view(-1), y[:, 0])
