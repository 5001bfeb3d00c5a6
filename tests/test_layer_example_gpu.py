"""The example layer: the operators together, trained and served.

Training has to lower the loss; serving in parts has to agree with whole
sequences, in fp32 within 1e-3 of the outputs' size (fp32 matrix products of
different shapes differ by about 1e-6 a layer, TF32 is off by default) and in
bf16 within 5% (each intermediate is rounded to 2^-9, and the two paths
round step sizes at different places).  The hand-written gradient chain is
checked against central differences of the layer's own fp32 forward."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-3), (torch.bfloat16, 5e-2)])
def test_trains_and_serves(dtype, tol):
    import layer as example
    m = example.Layer(width=64, inner=128, states=8, rank=8, dtype=dtype)
    losses = example.train(m)
    assert losses[-1] < 0.7 * losses[0], losses
    assert example.serve(m) <= tol


def test_gradients_of_the_whole_layer():
    import layer as example
    m = example.Layer(width=32, inner=64, states=4, rank=4, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, r, do, dr = (torch.randn(2, 19, 32, generator=g, device="cuda") for _ in range(4))
    _, _, saved = m.forward(x, r)
    grads, (dx, dres) = m.backward(saved, do, dr)

    def value(xv, rv):
        out, res, _ = m.forward(xv, rv)
        return float((out.double() * do.double()).sum() + (res.double() * dr.double()).sum())

    def slope_of(plus, minus, eps):
        return (plus - minus) / (2 * eps)

    eps = 1e-2  # fp32 forward: differences of this step carry about 1e-3 of noise
    for name, grad, at in (("x", dx, x), ("residual", dres, r)):
        way = torch.randn(at.shape, generator=g, device="cuda")
        way /= way.norm()
        ends = [value(x + s * eps * way, r) if name == "x" else value(x, r + s * eps * way) for s in (1, -1)]
        mine = float((grad.double() * way.double()).sum())
        assert abs(mine - slope_of(*ends, eps)) <= 2e-2 * (1 + abs(mine)), name
    for name, grad in grads.items():
        keep = m.w[name]
        way = torch.randn(keep.shape, generator=g, device="cuda")
        way /= way.norm()
        ends = []
        for s in (1, -1):
            m.w[name] = keep + s * eps * way
            ends.append(value(x, r))
        m.w[name] = keep
        mine = float((grad.double() * way.double()).sum())
        assert abs(mine - slope_of(*ends, eps)) <= 2e-2 * (1 + abs(mine)), name
