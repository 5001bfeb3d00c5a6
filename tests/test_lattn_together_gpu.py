"""Norms of queries and keys, linear attention, the gated norm and moves of cache rows
in a run, as a layer uses them: packed prompts, a fork of one request's state, single
tokens; and a training step with its gradients.

Each operator is held against its 64-bit form on what it was given, so that its own
roundings are all that a tolerance counts; the training step in fp32 is held against
the 64-bit form of the whole."""
import pytest
import torch

import block_reference as block
import lattn_reference as ref
from test_lattn_gpu import coarse, fine, near
from test_qknorm_gpu import close, pair_size

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HEADS, GROUPS, VALUE, KEY, ROT = 4, 2, 64, 32, 16
EPS = 1e-5


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


def layer(seed):
    g = torch.Generator().manual_seed(seed)
    return dict(A=-(torch.rand(HEADS, generator=g) * 15 + 1).cuda(), D=torch.randn(HEADS, generator=g).cuda(),
                bias=(torch.randn(HEADS, generator=g) - 2).cuda(), qw=(1 + 0.1 * torch.randn(KEY, generator=g)).cuda(),
                kw=(1 + 0.1 * torch.randn(KEY, generator=g)).cuda(), ow=(1 + 0.1 * torch.randn(HEADS * VALUE, generator=g)).cuda(),
                freq=(10000.0 ** (-torch.arange(ROT, dtype=torch.float32) / ROT)).cuda())


def parts(x):
    """v, z, k, q, delta of the rows of one projection."""
    hp, gn = HEADS * VALUE, GROUPS * KEY
    return x.split([hp, hp, gn, gn, HEADS], 0)


CHANNELS = 2 * HEADS * VALUE + 2 * GROUPS * KEY + HEADS


def heads_form(x, w, pos, freq):
    """[channels, tokens] in 64 bits."""
    v = ref.d64(x).t().unflatten(-1, (-1, w.shape[0]))
    return ref.heads_norm(v, ref.d64(w), ref.d64(pos), ref.d64(freq), EPS).flatten(-2).t()


def check_norms(dtype, x, w, pos, freq, got):
    want = heads_form(x, w, pos, freq)
    close(got, want, pair_size(want[None], KEY, ROT)[0] * 2, 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24,
          2.0 ** -24 * (KEY + 16) + 2.0 ** -20, "norms")


def check_gate(dtype, y, z, w, got):
    want = block.gatenorm(ref.d64(y)[None], ref.d64(z)[None], ref.d64(w), HEADS, False, EPS)[0]
    close(got, want, want.abs(), 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24, 1e-5, "gate")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompts_fork_and_steps(lr, dtype):
    p = layer(1)
    sizes, rows = [37, 1, 150], 7
    cu = torch.tensor([0] + sizes).cumsum(0).int()
    tokens = int(cu[-1])
    g = torch.Generator().manual_seed(2)
    wide = torch.randn(CHANNELS, tokens, generator=g).to(DT[dtype]).cuda()
    v, z, k, q, delta = parts(wide)
    pos = torch.cat([torch.arange(n) for n in sizes]).int().cuda()
    slots = [4, 0, 2]
    before = torch.randn(rows, HEADS * VALUE, KEY, generator=g)
    state = before.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    options = dict(groups=GROUPS, scale=KEY ** -0.5, delta_bias=p["bias"], delta_softplus=True)
    qn, kn = (t[0] for t in lr.qknorm_fwd(q[None], k[None], p["qw"], p["kw"], pos[None], p["freq"], eps=EPS))
    o = lr.lattn_prompt(qn, kn, v, p["A"], delta, p["D"], cu_seqlens=cu.cuda(), state=state, slots=torch.tensor(slots, **i32),
                        has_state=torch.tensor([False, True, False], device="cuda"), **options)
    out = lr.gatenorm_fwd(o[None], z[None], p["ow"], groups=HEADS, eps=EPS)[0]
    check_norms(dtype, q, p["qw"], pos, p["freq"], qn)
    check_norms(dtype, k, p["kw"], pos, p["freq"], kn)
    want = ref.packed(qn, kn, v, p["A"], delta, p["D"], cu.tolist(), slots, [False, True, False], before, GROUPS, KEY ** -0.5, p["bias"], True)
    f = dict(A=p["A"], delta=delta, bias=p["bias"], act=True)
    c = fine(f, KEY, tokens)
    io = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    near(o, want[0], want[2], (io, c + coarse(dtype)), "o")
    near(state[slots], want[1][slots], want[3][slots], (2.0 ** -24, c), "state")
    check_gate(dtype, o, z, p["ow"], out)
    # request 0 goes on in two ways, request 1 ends, and its row takes request 2's state
    held = state.clone()
    lr.state_move(state, torch.tensor([4, 4, 2, -1], **i32), torch.tensor([1, 6, 0, 2], **i32))
    assert torch.equal(state[[1, 6, 4]], held[[4, 4, 4]]) and torch.equal(state[0], held[2]) and not state[2].any()
    now, at = [1, 6, 0], [37, 37, 150]
    for step in range(3):
        first = state.cpu()
        one = torch.randn(3, CHANNELS, generator=g).to(DT[dtype]).cuda()
        one_v, one_z, one_k, one_q, one_d = (x.t() for x in parts(one.t()))
        here = torch.tensor([x + step for x in at], **i32)
        qs, ks = lr.qknorm_step(one_q, one_k, p["qw"], p["kw"], here, p["freq"], eps=EPS)
        os = lr.lattn_step(qs, ks, one_v, p["A"], one_d, p["D"], state=state, slots=torch.tensor(now, **i32), **options)
        outs = lr.gatenorm_step(os, one_z, p["ow"], groups=HEADS, eps=EPS)
        check_norms(dtype, one_q.t(), p["qw"], here, p["freq"], qs.t())
        check_norms(dtype, one_k.t(), p["kw"], here, p["freq"], ks.t())
        cut = [x[..., None] for x in (qs, ks, one_v, one_d)]
        want = ref.forward(*cut[:3], p["A"], cut[3], p["D"], first[now], GROUPS, KEY ** -0.5, p["bias"], True)
        c = fine(dict(A=p["A"], delta=cut[3], bias=p["bias"], act=True), KEY, 1)
        near(os, want[0][..., 0], want[2][..., 0], (io, c), "step")
        near(state[now], want[1], want[3], (2.0 ** -24, c), "state")
        check_gate(dtype, os.t(), one_z.t(), p["ow"], outs.t())
    others = [2, 3, 4, 5]
    assert torch.equal(state[others].cpu(), first[others]) and torch.equal(state[[3, 5]].cpu(), before[[3, 5]])
    assert lr.get_last_error() == lr.SSCAN_OK


@pytest.mark.parametrize("L", [130, 67])
def test_training_step(lr, L):
    """Gradients through the norms and linear attention.  The roundings of its gradients, c of their
    terms' magnitudes, pass through the norm's Jacobian, whose entries' magnitudes are at most
    rstd |w| (1 + |n| mean |n|) over a pair that turns."""
    p = layer(3)
    g = torch.Generator().manual_seed(L)
    x = torch.randn(2, CHANNELS, L, generator=g).cuda()
    hp, gn = HEADS * VALUE, GROUPS * KEY
    v, _, k, q, delta = x.split([hp, hp, gn, gn, HEADS], 1)
    pos = torch.arange(L, dtype=torch.int32).expand(2, L).contiguous().cuda()
    do = torch.randn(2, hp, L, generator=g).cuda()
    options = dict(groups=GROUPS, scale=KEY ** -0.5, delta_bias=p["bias"], delta_softplus=True)
    qn, kn = lr.qknorm_fwd(q, k, p["qw"], p["kw"], pos, p["freq"], eps=EPS)
    lr.lattn_fwd(qn, kn, v, p["A"], delta, p["D"], **options)
    a = lr.lattn_bwd(qn, kn, v, p["A"], delta, p["D"], None, do, **options)
    b = lr.qknorm_bwd(q, k, p["qw"], p["kw"], a["dq"], a["dk"], pos, p["freq"], eps=EPS)
    exact = {}
    leaves = {}
    for name, t, w in (("q", q, p["qw"]), ("k", k, p["kw"])):
        leaf = ref.d64(t).transpose(1, 2).unflatten(-1, (-1, KEY)).requires_grad_()
        weight = ref.d64(w).requires_grad_()
        leaves[name] = (leaf, weight)
        exact[name] = ref.heads_norm(leaf, weight, ref.d64(pos), ref.d64(p["freq"]), EPS).flatten(-2).transpose(1, 2)
    want, mag = ref.backward(exact["q"].detach(), exact["k"].detach(), v, p["A"], delta, p["D"], None, do, None, GROUPS, KEY ** -0.5,
                             p["bias"], True)
    c = 4 * fine(dict(A=p["A"], delta=delta, bias=p["bias"], act=True), KEY, L) + 2.0 ** -24 * (KEY + 16) * 4 + 2.0 ** -19
    near(a["dv"], want["dv"], mag["dv"], (2.0 ** -24, c), "dv")
    for name in ("q", "k"):
        leaf, weight = leaves[name]
        dx, dw = torch.autograd.grad(exact[name], (leaf, weight), want["d" + name])
        xs = leaf.detach()
        rstd = 1 / torch.sqrt((xs * xs).mean(-1, keepdim=True) + EPS)
        n = (xs * rstd).abs()
        up = pair_size(mag["d" + name], KEY, ROT).transpose(1, 2).unflatten(-1, (-1, KEY))
        gw = up * weight.detach().abs()
        size = rstd * (gw + n * (gw * n).mean(-1, keepdim=True))
        close(b["d" + name], dx.flatten(-2).transpose(1, 2), size.flatten(-2).transpose(1, 2), 2.0 ** -24, 2 * c, "d" + name)
        close(b["d" + name + "_weight"], dw, (up * n).sum((0, 1, 2)), 2.0 ** -24, 2 * c + 2.0 ** -16, "d" + name + "_weight")
    assert lr.get_last_error() == lr.SSCAN_OK
