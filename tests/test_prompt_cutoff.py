"""What a split of the packed scan leaves out: the figure that the header
promises is the one the kernels use, and they keep it.

An impulse of 2^20 (an input, or the initial state) decays by r bits up to a
border.  Where r < 26 all of it is carried: the state behind the border is
right to 1e-5 of itself (25.5 bits of decay round by 25.5 ln 2 2^-23, about
2e-6, and the steps after it add as much).  Where r > 26 the state may miss it, and is
off by no more than 2^-26 of 2^20, decayed on from the border."""
import math
import os
import re

import pytest
import torch

import block_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUT = 26


def _read(*path):
    with open(os.path.join(ROOT, *path), encoding="utf-8") as f:
        return f.read()


def test_header_and_kernels_name_one_figure():
    header = _read("include", "sscan.h")
    text = header[header.index("* sscan_prompt --"):header.index("int sscan_prompt(")]
    assert re.findall(r"2\^-(\d+)", text) == [str(CUT)] * 2
    code = _read("linear_recurrence_gb300", "csrc", "sscan_prompt.cuh")
    assert re.findall(r"kCutBits = (\d+)\.f", code) == [str(CUT)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens", [80, 83])  # whole 16-byte vectors and not; two segments of 48
@pytest.mark.parametrize("initial", [False, True])
def test_an_impulse_before_a_border(dtype, tokens, initial):
    import linear_recurrence_gb300 as lr
    border, at, dim, dt, size = 48, 17, 40, 2.0 ** -4, 2.0 ** 20
    bits = [4.0, 12.0, 20.0, 25.0, 25.5, 25.5, 25.5, 25.5, 26.5, 27.0, 28.0, 30.0, 40.0, 60.0, 100.0, 200.0]
    N = len(bits)
    # an input decays over the tokens after its own, an initial state over all of its request's
    steps = border - at if initial else border - at - 1
    A = -torch.tensor(bits)[None].repeat(dim, 1) * math.log(2) / (steps * dt)
    u, delta = torch.zeros(dim, tokens), torch.full((dim, tokens), dt)
    state = torch.zeros(2, dim, N)
    if initial:
        state[1] = size
    else:
        u[:, at] = size / dt
    B, C = torch.ones(N, tokens), torch.ones(N, tokens)
    cu = [0, at, tokens]
    got = state.cuda()
    lr.sscan_prompt(u.to(dtype).cuda(), delta.to(dtype).cuda(), A.cuda(), B.to(dtype).cuda(), C.to(dtype).cuda(),
                    cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), state=got, segments=2)
    assert lr.get_last_error() == 0 and lr.last_plan().endswith("segments=2 of 48")
    _, want, _ = ref.scan_packed(*(ref.d64(t) for t in (u, delta, A, B, C)), None, cu, None, None, ref.d64(state))
    off, want = (got.double().cpu() - want).abs()[1], want[1]
    kept = torch.tensor(bits) < CUT
    assert bool((off[:, kept] <= 1e-5 * want[:, kept]).all())
    decay = torch.exp(ref.d64(A) * dt * (tokens - border))
    assert bool((off <= 1e-5 * want + 2.0 ** -CUT * size * decay).all())
