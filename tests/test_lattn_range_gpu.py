"""Offsets beyond 32 bits: caches, sequences and strides of more than 2^31 values."""
import pytest
import torch

import lattn_reference as ref
from test_lattn_gpu import coarse, fine, make, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


def test_rows_far_into_a_cache(lr):
    """Steps, short and long prompts and moves on the rows behind 2^31 values."""
    heads, value, key = 64, 256, 128  # 2^21 values a row
    rows = 1030
    state = torch.zeros(rows, heads * value, key, device="cuda")
    assert state[rows - 1].data_ptr() - state.data_ptr() > 2 ** 32
    f = make(3, "bf16", 1, heads, 1, value, key, 40, packed=True, s0=False)
    near_state = torch.zeros(4, heads * value, key, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    got = []
    for cache, slots in ((near_state, [0, 1, 2]), (state, [rows - 3, rows - 2, rows - 1])):
        out = []
        for cu in ([0, 5, 9, 40], [0, 2, 20, 40]):
            out.append(lr.lattn_prompt(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], cu_seqlens=torch.tensor(cu, **i32), state=cache,
                                       slots=torch.tensor(slots, **i32), scale=0.1, delta_bias=f["bias"], delta_softplus=True))
        one = [f[x][:, :3].t().contiguous() for x in ("q", "k", "v", "delta")]
        out.append(lr.lattn_step(*one[:3], f["A"], one[3], f["D"], state=cache, slots=torch.tensor(slots, **i32), scale=0.1,
                                 delta_bias=f["bias"], delta_softplus=True))
        out.append(cache[slots].clone())
        lr.state_move(cache, torch.tensor([slots[2], slots[0], -1], **i32), torch.tensor([slots[0], slots[2], slots[1]], **i32))
        out.append(cache[slots].clone())
        got.append(out)
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert got[0][3].any() and not got[0][4][1].any() and torch.equal(got[0][4][0], got[0][3][2])
    assert not state[:rows - 3].any()
    assert lr.get_last_error() == lr.SSCAN_OK


@pytest.mark.parametrize("tokens", [450_000, 450_001])
def test_rows_longer_than_32_bits_reach(lr, tokens):
    """5120 channels of 450,000 tokens: the last ones against the 64-bit form, from the state before them."""
    heads, value, key, tail = 80, 64, 16, 70
    g = torch.Generator(device="cuda").manual_seed(1)
    wide = torch.empty(heads * value + 2 * key, tokens, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    v, k, q = wide[:heads * value], wide[heads * value:heads * value + key], wide[heads * value + key:]
    assert v.numel() > 2 ** 31
    A = -torch.exp2(-1.0 - 6.0 * torch.arange(heads) / heads).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    state = torch.zeros(2, heads * value, key, device="cuda")
    cut = tokens - tail
    o = lr.lattn_prompt(q, k, v, A, cu_seqlens=torch.tensor([0, tokens], **i32), state=state, slots=torch.tensor([0], **i32), scale=0.25)
    lr.lattn_prompt(q[:, :cut], k[:, :cut], v[:, :cut], A, cu_seqlens=torch.tensor([0, cut], **i32), state=state,
                    slots=torch.tensor([1], **i32), scale=0.25)
    rest = [x[None, :, cut:] for x in (q, k, v)]
    want = ref.forward(*rest, A, None, None, state[1:2], 1, 0.25)
    f = dict(A=A, delta=None, bias=None, act=False)
    c = fine(f, key, tail)
    # both states carry the roundings of the tokens before, each c of the terms' magnitudes: decays of at
    # most 2^-1/128 a token leave some 400 tokens' terms, sqrt(400) of a value's size each
    before = 400 * c
    near(o[:, cut:], want[0][0], want[2][0] + 1, (2.0 ** -8, before + coarse("bf16")), "o")
    near(state[0], want[1][0], want[3][0] + 1, (2.0 ** -24, before), "state")
    turned, _ = lr.qknorm_fwd(v[None], None, torch.ones(value, device="cuda"), None)
    x = ref.d64(v[:, cut:]).t().unflatten(-1, (-1, value))
    want = ref.heads_norm(x, torch.ones(value, dtype=torch.float64), None, None, 1e-5).flatten(-2).t()
    off = (turned[0, :, cut:].double().cpu() - want).abs()
    assert float((off - 2.0 ** -8 * want.abs() - 2.0 ** -17).max()) <= 0
