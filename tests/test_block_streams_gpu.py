"""The packed forms, which launch two kernels and take scratch memory, on
streams of the caller's, on two streams at once, and captured in a graph."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


def _problem(seed, dim, tokens, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    N, cu = 16, [0, tokens // 3, tokens // 3, tokens - 5, tokens]
    p = {"x": r(2 * dim, tokens).to(dtype)[:dim], "w": r(dim, 4), "delta": (r(dim, tokens) - 3).to(dtype), "z": r(dim, tokens).to(dtype),
         "A": -torch.rand(dim, N, generator=g, device="cuda") - 0.1, "B": r(N, tokens).to(dtype), "C": r(N, tokens).to(dtype), "D": r(dim),
         "nw": torch.ones(dim, device="cuda"), "cu": torch.tensor(cu, dtype=torch.int32, device="cuda"),
         "slots": torch.tensor([3, 0, -1, 2], dtype=torch.int32, device="cuda"),
         "has": torch.tensor([True, False, True, False], device="cuda"),
         "conv": r(5, dim, 3).to(dtype), "scan": r(5, dim, N)}
    return p


def _run(lr, p, conv, scan, outs=None):
    """The packed forms and the norm's gradients, caches advanced in place."""
    kw = dict(cu_seqlens=p["cu"], slots=p["slots"], has_state=p["has"])
    o = outs or {}
    u = lr.sconv_prompt(p["x"], p["w"], state=conv, out=o.get("u"), **kw)
    y = lr.sscan_prompt(u, p["delta"], p["A"], p["B"], p["C"], p["D"], state=scan, z=p["z"], delta_bias=p["nw"], delta_softplus=True,
                        segments=6, out=o.get("y"), **kw)
    g = lr.gatenorm_bwd(y[None], p["z"][None], p["nw"], u[None])
    return u, y, g["dy"], g["dz"], g["dweight"]


CASES = [(1, 600, 700, torch.bfloat16), (2, 320, 1003, torch.float32)]


def _alone(lr, p):
    conv, scan = p["conv"].clone(), p["scan"].clone()
    out = _run(lr, p, conv, scan)
    torch.cuda.synchronize()
    assert lr.get_last_error() == 0
    return (*out, conv, scan)


def test_two_streams_at_once(lr):
    ps = [_problem(*c) for c in CASES]
    want = [_alone(lr, p) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    caches = [[(p["conv"].clone(), p["scan"].clone()) for _ in range(20)] for p in ps]
    torch.cuda.synchronize()
    got = [[], []]
    for k in range(20):
        for i, p in enumerate(ps):
            with torch.cuda.stream(streams[i]):
                got[i].append((*_run(lr, p, *caches[i][k]), *caches[i][k]))
    torch.cuda.synchronize()
    assert lr.get_last_error() == 0
    for i in range(2):
        for tensors in got[i]:
            for a, b in zip(tensors, want[i]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("case", range(2))
def test_packed_forms_in_a_captured_graph(lr, case):
    """After one ordinary call; the scratch of a split belongs to the graph."""
    p = _problem(*CASES[case])
    want = _alone(lr, p)
    conv, scan = p["conv"].clone(), p["scan"].clone()
    outs = {"u": torch.empty_like(want[0]), "y": torch.empty_like(want[1])}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _run(lr, p, conv, scan, outs)
    for _ in range(3):
        conv.copy_(p["conv"])
        scan.copy_(p["scan"])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*got, conv, scan), want):
            assert torch.equal(a, b)
