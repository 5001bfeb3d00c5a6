"""Packed prompts and single tokens captured in a graph, as a server that decodes by graphs has them: kernels that
begin while the one before them ends, with scratch taken between them."""
import pytest
import torch

from test_lattn_gpu import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", [[5, 1, 300, 16, 0, 40, 2], [700, 333]], ids=["short", "long"])
@pytest.mark.parametrize("pieces", [0, 1, 3])
@pytest.mark.parametrize("offset", [0, 1])
def test_prompts_and_steps(lr, dtype, sizes, pieces, offset):
    heads, groups, value, key = 4, 2, 64, 64
    tokens, n = sum(sizes), len(sizes)
    f = make(3, dtype, 1, heads, groups, value, key, tokens, packed=True, s0=False, offset=offset)
    cu = torch.tensor([0] + sizes).cumsum(0).int().cuda()
    slots = torch.randperm(n + 2, generator=torch.Generator().manual_seed(n))[:n].int().cuda()
    has = torch.tensor([i % 2 == 0 for i in range(n)], device="cuda")
    first = torch.randn(n + 2, heads * value, key, device="cuda")
    one = {x: f[x].t()[:n].contiguous() for x in ("q", "k", "v", "delta")}
    qw = torch.rand(key, device="cuda")
    pos, freq = torch.arange(n, device="cuda", dtype=torch.int32), torch.rand(key // 2, device="cuda")
    options = dict(groups=groups, scale=0.125, delta_bias=f["bias"], delta_softplus=True)
    state = first.clone()

    def both():
        o = lr.lattn_prompt(f["q"], f["k"], f["v"], f["A"], f["delta"], f["D"], cu_seqlens=cu, state=state, slots=slots, has_state=has,
                            pieces=pieces, **options)
        q, k = lr.qknorm_step(one["q"], one["k"], qw, qw, pos, freq)
        return o, lr.lattn_step(q, k, one["v"], f["A"], one["delta"], f["D"], state=state, slots=slots, **options)

    want = []
    for _ in range(2):
        want.append([*(x.clone() for x in both()), state.clone()])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    state.copy_(first)
    for there in want:
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(there, (*outs, state)):
            assert torch.equal(a, b)
    assert lr.get_last_error() == lr.SSCAN_OK
