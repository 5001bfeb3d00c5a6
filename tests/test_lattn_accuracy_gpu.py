"""How exact linear attention is where its other tests allow much: by the norm of what is off.

Their bounds follow the sum of a chunk's exponents, or of all its terms' magnitudes.  Here inputs are
random, so that a sum of K terms of either sign is about sqrt(K) of one, and so is what their roundings add up
to: what a sum is off by, relative to it, is what a term is off by, whatever K."""
import pytest
import torch

import lattn_reference as ref
from test_lattn_gpu import fine, make, near

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


# Sums held in fp32: a term is off by 2^-21 (sums of at most 256 products, the exponential), and by 2^-16 where a state
# in two bf16 terms is a factor.  The steps' gradients are sums from the chunk's end in which neighbours cancel, down to a
# fraction of a term: 2^-13 leaves 2^3 for that in bf16, 2^8 in fp32.  ddelta in bf16 is rounded once more.  (A gradient of
# zeros is off by 1, one of the wrong sign by 2.)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["softplus", "steps", "fixed"])
@pytest.mark.parametrize("L", [65, 129, 333])
@pytest.mark.parametrize("ends", [False, True], ids=["alone", "states"])
@pytest.mark.parametrize("shape", [(4, 1, 64, 128), (2, 2, 64, 64), (2, 1, 200, 128), (3, 1, 17, 33), (6, 2, 48, 16)], ids=str)
def test_gradients_of_steps_and_rates(lr, dtype, kind, L, ends, shape):
    heads, groups, value, key = shape
    f = make(L + heads, dtype, 2, heads, groups, value, key, L, delta=kind != "fixed", options=kind == "softplus", D=ends, s0=ends)
    g = torch.Generator().manual_seed(L)
    do = torch.randn(2, heads * value, L, generator=g).to(f["q"].dtype).cuda()
    ds = torch.randn(2, heads * value, key, generator=g).cuda() if ends else None
    scale = key ** -0.5
    args = (f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], f["s0"], do, ds)
    got = lr.lattn_bwd(*args, groups=groups, scale=scale, delta_bias=f["bias"], delta_softplus=f["act"])
    want, _ = ref.backward(*args, groups, scale, f["bias"], f["act"])
    assert lr.get_last_error() == lr.SSCAN_OK
    assert off(got["dA"], want["dA"]) <= 2.0 ** -13, "dA"
    if f["bias"] is not None:
        assert off(got["ddelta_bias"], want["ddelta_bias"]) <= 2.0 ** -13, "ddelta_bias"
    if f["delta"] is not None:
        for h in range(heads):
            assert off(got["ddelta"][:, h], want["ddelta"][:, h]) <= 2.0 ** -13 + (2.0 ** -8 if dtype == "bf16" else 0.0), ("ddelta", h)
    if ends:  # from all tokens, each in fp32 (bf16: states' gradients pass through the chunks in fp32, too)
        assert off(got["dD"], want["dD"]) <= 2.0 ** -18, "dD"
        assert off(got["ds0"], want["ds0"]) <= 2.0 ** -18, "ds0"


# Fast decays leave a state to the first few tokens of a chunk alone: 2^-17 of a tenth of the sum and 2^-22 of the
# rest, 2^-20 in all; twice that allowed.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rate,bias", [(-16.0, 0.0), (-16.0, 2.0), (-4.0, 1.0)])
@pytest.mark.parametrize("value,key", [(64, 32), (128, 128)])
def test_rates_gradient_of_fast_decays_is_as_exact_as_a_state_allows(lr, dtype, rate, bias, value, key):
    heads, L = 4, 400
    f = make(18, dtype, 1, heads, 1, value, key, L, D=False, s0=False)
    f["A"], f["bias"] = torch.full((heads,), rate, device="cuda"), torch.full((heads,), bias, device="cuda")
    do = torch.randn(1, heads * value, L, generator=torch.Generator().manual_seed(2)).to(f["q"].dtype).cuda()
    args = (f["q"], f["k"], f["v"], f["A"], f["delta"], None, None, do, None)
    got = lr.lattn_bwd(*args, groups=1, scale=0.2, delta_bias=f["bias"], delta_softplus=True)
    want, _ = ref.backward(*args, 1, 0.2, f["bias"], True)
    assert off(got["dA"], want["dA"]) <= 2.0 ** -19


# D in 16 bits at least, and then the rounding of o: 2^-16 on top of what the rounded exact outputs are off by, whose
# norm is some 2^-9.3.
@pytest.mark.parametrize("packed", [False, True], ids=["batch", "packed"])
@pytest.mark.parametrize("value,key", [(64, 128), (128, 64), (40, 24)])
@pytest.mark.parametrize("L", [1, 130, 333])
def test_bf16_outputs_take_all_of_D(lr, packed, value, key, L):
    """Keys of zeros leave D v alone, and a D next to half a step of bf16 is off by as much where it is rounded."""
    heads = 6
    f = make(21, "bf16", 1, heads, 1, value, key, L, s0=False)
    D = torch.tensor([1.00390625, -1.0117, 0.3333333, 257.0, 1e-30, -3.003], device="cuda")
    k = torch.zeros_like(f["k"])
    options = dict(scale=0.1, delta_bias=f["bias"], delta_softplus=True)
    if packed:
        state = torch.zeros(2, heads * value, key, device="cuda")
        cu = torch.tensor([0, L // 3, L], dtype=torch.int32, device="cuda")
        o = lr.lattn_prompt(f["q"][0], k[0], f["v"][0], f["A"], f["delta"][0], D, cu_seqlens=cu, state=state, **options)[None]
    else:
        o, _ = lr.lattn_fwd(f["q"], k, f["v"], f["A"], f["delta"], D, **options)
    want = ref.d64(D).repeat_interleave(value)[None, :, None] * ref.d64(f["v"])
    least = (want.to(torch.bfloat16).double() - want).abs()
    assert bool(((o.double().cpu() - want).abs() <= least + 2.0 ** -15 * want.abs()).all())
    for h in range(heads):
        rows = slice(h * value, (h + 1) * value)
        assert off(o[:, rows], want[:, rows]) <= off(want[:, rows].to(torch.bfloat16), want[:, rows]) + 2.0 ** -15, h


# The bias' gradient term by term: a pair's weight is off by 2^-22 (the exponential) and its sums by as much, what cancels
# spans eight tokens of a block (8 * 2^-24), and a state in two bf16 terms (2^-17) counts for a few of a chunk's tokens: 2^-19.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("shape", [(8, 1, 64, 128, 128), (16, 2, 64, 64, 64), (8, 1, 128, 64, 333), (12, 4, 48, 40, 259)], ids=str)
def test_bias_gradient_by_terms(lr, dtype, softplus, shape):
    heads, groups, value, key, L = shape
    scale = key ** -0.5
    for seed in range(3):
        f = make(seed + L, dtype, 2, heads, groups, value, key, L, s0=False)
        if not softplus:  # steps as they are, the bias a small one
            f["delta"] = torch.nn.functional.softplus(f["delta"].float() - 2.5).to(f["q"].dtype)
            f["bias"], f["act"] = torch.full((heads,), 2.0 ** -6, device="cuda"), False
        do = torch.randn(2, heads * value, L, generator=torch.Generator().manual_seed(seed)).to(f["q"].dtype).cuda()
        args = (f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], None, do, None)
        got = lr.lattn_bwd(*args, groups=groups, scale=scale, delta_bias=f["bias"], delta_softplus=f["act"])
        want, _ = ref.backward(*args, groups, scale, f["bias"], f["act"])
        assert off(got["ddelta_bias"], want["ddelta_bias"]) <= 2.0 ** -19, seed


# Of few tokens dq and dk are few sums over the heads that share them.  Here the heads' terms cancel but for 2^-6 of
# them: c, the roundings in fp32, of the terms' magnitudes, and the rounding of the result.
@pytest.mark.parametrize("batch,groups,L", [(1, 1, 1), (2, 1, 1), (1, 2, 3), (3, 1, 5), (1, 1, 16), (2, 2, 4)])
@pytest.mark.parametrize("value,key", [(64, 128), (128, 16), (40, 40)])
@pytest.mark.parametrize("ends", [False, True], ids=["alone", "states"])
def test_bf16_gradients_of_few_tokens(lr, batch, groups, L, value, key, ends):
    heads = 8 * groups
    f = make(L, "bf16", batch, heads, groups, value, key, L, s0=ends, delta=False)
    f["A"] = f["A"][:1].expand(heads).contiguous()
    pairs = (f["v"].unflatten(1, (groups, 4, 2, value))[:, :, :, :1].expand(-1, -1, -1, 2, -1, -1)).flatten(1, 4)
    f["v"] = pairs.contiguous()
    g = torch.Generator().manual_seed(L)
    do = torch.randn(batch, groups, 4, 1, value, L, generator=g)
    do = torch.cat([do, -do * (1 + 2.0 ** -6 * torch.rand(do.shape, generator=g))], 3).flatten(1, 4).to(torch.bfloat16).cuda()
    ds = torch.randn(batch, heads * value, key, generator=g).cuda() if ends else None
    args = (f["q"], f["k"], f["v"], f["A"], None, f["D"], f["s0"], do, ds)
    got = lr.lattn_bwd(*args, groups=groups, scale=0.25)
    want, mag = ref.backward(*args, groups, 0.25)
    c = fine(f, key, L) + 2.0 ** -24 * (value + heads)
    for name in ("dq", "dk", "dv"):
        near(got[name], want[name], mag[name], (2.0 ** -8, c), name)
    assert lr.get_last_error() == lr.SSCAN_OK
