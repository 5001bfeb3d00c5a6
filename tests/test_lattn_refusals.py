"""What linear attention, the norms of its queries and keys and the moves of cache rows refuse,
before anything is launched: the C ABI on sizes, flags and missing pointers, the binding on tensors."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails first
S8 = (ctypes.c_int64 * 8)(64, 8, 64, 8, 64, 8, 16, 8)
S4 = (ctypes.c_int64 * 4)(64, 8, 64, 8)
NEG8 = (ctypes.c_int64 * 8)(64, 8, 64, 8, 64, -8, 16, 8)
NEG4 = (ctypes.c_int64 * 4)(64, 8, 64, -8)

IN = dict(q=FAKE, k=FAKE, v=FAKE, A=FAKE, delta=None, D=None, bias=None)
FWD = dict(**IN, s0=None, o=FAKE, final=None, batch=1, heads=4, groups=2, key=8, value=8, len=8, strides=S8, scale=1.0, dtype=0,
           flags=0, pieces=0, stream=None)
BWD = dict(**IN, s0=None, dout=FAKE, dfinal=None, dq=FAKE, dk=FAKE, dv=FAKE, ddelta=None, dA=FAKE, dD=None, dbias=None, ds0=None,
           batch=1, heads=4, groups=2, key=8, value=8, len=8, strides=S8, scale=1.0, dtype=0, flags=0, stream=None)
PROMPT = dict(**IN, cu=FAKE, slots=None, has=None, state=FAKE, o=FAKE, requests=1, rows=1, heads=4, groups=2, key=8, value=8, tokens=8,
              strides=S8, scale=1.0, dtype=0, flags=0, pieces=0, stream=None)
STEP = dict(**IN, slots=None, state=FAKE, o=FAKE, batch=1, rows=1, heads=4, groups=2, key=8, value=8, qs=16, ks=16, vs=32, ts=4,
            scale=1.0, dtype=0, flags=0, stream=None)
QK = dict(q=FAKE, k=FAKE, qw=FAKE, kw=FAKE, pos=FAKE, freq=FAKE)
QKF = dict(**QK, qo=FAKE, ko=FAKE, batch=1, qh=2, kh=1, dim=8, len=8, rot=4, strides=S4, eps=1e-5, dtype=0, stream=None)
QKB = dict(**QK, dqo=FAKE, dko=FAKE, dq=FAKE, dk=FAKE, dqw=FAKE, dkw=FAKE, batch=1, qh=2, kh=1, dim=8, len=8, rot=4, strides=S4, eps=1e-5,
           dtype=0, stream=None)
QKS = dict(**QK, qo=FAKE, ko=FAKE, batch=1, qh=2, kh=1, dim=8, rot=4, qs=16, ks=8, eps=1e-5, dtype=0, stream=None)
MOVE = dict(cache=FAKE, src=FAKE, dst=FAKE, moves=2, layers=1, rows=4, bytes=64, stream=None)

SHARED = (dict(q=None), dict(k=None), dict(v=None), dict(A=None), dict(key=0), dict(key=129), dict(value=0), dict(value=257),
          dict(groups=0), dict(groups=3), dict(heads=-1), dict(heads=65536), dict(dtype=2), dict(flags=2), dict(flags=3))
BAD = [("lattn_fwd", FWD, c) for c in SHARED + (
    dict(o=None), dict(batch=-1), dict(batch=65536), dict(len=-1), dict(len=1 << 31), dict(strides=None), dict(strides=NEG8), dict(pieces=-1))]
BAD += [("lattn_bwd", BWD, c) for c in SHARED + (
    dict(dout=None), dict(dq=None), dict(dk=None), dict(dv=None), dict(dA=None), dict(delta=FAKE), dict(strides=None), dict(len=-1))]
BAD += [("lattn_prompt", PROMPT, c) for c in SHARED + (
    dict(cu=None), dict(state=None), dict(o=None), dict(requests=2), dict(requests=-1), dict(tokens=1 << 31), dict(rows=-1),
    dict(rows=1 << 31), dict(strides=NEG8), dict(pieces=-2))]
BAD += [("lattn_step", STEP, c) for c in SHARED + (
    dict(state=None), dict(o=None), dict(batch=2), dict(batch=-1), dict(qs=-1), dict(ts=-1), dict(rows=-1), dict(batch=1 << 29, rows=1 << 29))]
QBAD = (dict(q=None), dict(k=None), dict(qw=None), dict(kw=None), dict(pos=None), dict(freq=None), dict(dim=0), dict(dim=257),
        dict(rot=5), dict(rot=-1), dict(qh=-1), dict(kh=1 << 21), dict(batch=-1), dict(dtype=3))
BAD += [("qknorm_fwd", QKF, c) for c in QBAD + (dict(qo=None), dict(ko=None), dict(strides=None), dict(strides=NEG4), dict(len=1 << 31))]
BAD += [("qknorm_bwd", QKB, c) for c in QBAD + (dict(dq=None), dict(dk=None), dict(dqw=None), dict(dkw=None), dict(dqo=None), dict(strides=NEG4))]
BAD += [("qknorm_step", QKS, c) for c in QBAD + (dict(qo=None), dict(qs=-1), dict(ks=-1))]
BAD += [("state_move", MOVE, c) for c in (
    dict(cache=None), dict(src=None), dict(dst=None), dict(moves=-1), dict(moves=8193), dict(layers=-1), dict(rows=-1), dict(bytes=-1),
    dict(rows=1 << 31), dict(bytes=1 << 35), dict(layers=1 << 20, rows=1 << 20, bytes=1 << 20))]


@pytest.mark.parametrize("name,base,change", BAD,
                         ids=[f"{n}-{'-'.join(k if k == 'strides' else f'{k}={v}' for k, v in c.items())}" for n, _, c in BAD])
def test_abi_refuses(lr, name, base, change):
    args = dict(base)
    args.update(change)
    assert getattr(lr.lib(), name)(*args.values()) == lr.SSCAN_ERR_INVALID
    assert lr.last_launch_count() == 0 and lr.last_plan() == "rejected"


@pytest.mark.parametrize("name,base,change", [
    ("lattn_fwd", FWD, dict(batch=0)), ("lattn_fwd", FWD, dict(len=0)), ("lattn_fwd", FWD, dict(heads=0)), ("lattn_bwd", BWD, dict(heads=0)),
    ("lattn_prompt", PROMPT, dict(heads=0)), ("lattn_prompt", PROMPT, dict(requests=0, tokens=0)), ("lattn_step", STEP, dict(batch=0)),
    ("qknorm_fwd", QKF, dict(len=0)), ("qknorm_fwd", QKF, dict(qh=0, kh=0)), ("qknorm_step", QKS, dict(batch=0)),
    ("state_move", MOVE, dict(moves=0)), ("state_move", MOVE, dict(bytes=0)), ("state_move", MOVE, dict(layers=0))])
def test_abi_takes_empty_problems(lr, name, base, change):
    args = dict(base)
    args.update(change)
    assert getattr(lr.lib(), name)(*args.values()) == lr.SSCAN_OK
    assert lr.last_launch_count() == 0 and lr.last_plan() == "empty"


def calls(lr, dev):
    """Calls of wrong shapes, types or strides; on the CPU every call is one."""
    z = lambda *s: torch.zeros(*s, device=dev)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    q, v, A = z(1, 8, 16), z(1, 32, 16), z(4)
    s = z(2, 32, 8)
    cu = i32(2)
    return [
        lambda: lr.lattn_fwd(q, q, v.half(), A), lambda: lr.lattn_fwd(q[0], q, v, A), lambda: lr.lattn_fwd(q, q[:, :4], v, A),
        lambda: lr.lattn_fwd(q, q, v, z(5)), lambda: lr.lattn_fwd(q, q, v, A.double()), lambda: lr.lattn_fwd(q, q, v, A, groups=3),
        lambda: lr.lattn_fwd(q, q, v, A, z(1, 3, 16)), lambda: lr.lattn_fwd(q, q, v, A, delta_bias=A),
        lambda: lr.lattn_fwd(q, q, v.transpose(1, 2).contiguous().transpose(1, 2), A), lambda: lr.lattn_fwd(q, q.bfloat16(), v, A),
        lambda: lr.lattn_fwd(q, q, v, A, None, None, z(1, 32, 9)), lambda: lr.lattn_fwd(z(1, 129, 16), z(1, 129, 16), v, A),
        lambda: lr.lattn_fwd(q, q, z(1, 257, 16), z(1)), lambda: lr.lattn_fwd(q, q, v, A, out=z(1, 32, 15)),
        lambda: lr.lattn_bwd(q, q, v, A, None, None, None, v[:, :16]), lambda: lr.lattn_bwd(q, q, v, A, None, None, None, v, z(1, 32, 9)),
        lambda: lr.lattn_bwd(q, q, v, A, None, z(3), None, v),
        lambda: lr.lattn_prompt(q[0], q[0], v[0], A, cu_seqlens=cu, state=z(1, 32, 9)),
        lambda: lr.lattn_prompt(q[0], q[0], v[0], A, cu_seqlens=cu.long(), state=s),
        lambda: lr.lattn_prompt(q[0], q[0], v[0], A, cu_seqlens=i32(4), state=s),
        lambda: lr.lattn_prompt(q[0], q[0], v[0], A, cu_seqlens=cu, state=s.bfloat16()),
        lambda: lr.lattn_prompt(q, q, v, A, cu_seqlens=cu, state=s),
        lambda: lr.lattn_step(z(3, 8), z(3, 8), z(3, 32), A, state=s), lambda: lr.lattn_step(z(2, 8), z(2, 9), z(2, 32), A, state=s),
        lambda: lr.lattn_step(z(2, 8), z(2, 8), z(2, 32), A, state=s, slots=i32(3)),
        lambda: lr.lattn_step(z(2, 8), z(2, 8), z(2, 32), A, z(2, 5), state=s),
        lambda: lr.qknorm_fwd(q, q, z(3), z(3)), lambda: lr.qknorm_fwd(q, None, z(8), z(8)), lambda: lr.qknorm_fwd(q, q, z(8), z(4)),
        lambda: lr.qknorm_fwd(q, q, z(8), z(8), i32(1, 16)), lambda: lr.qknorm_fwd(q, q, z(8), z(8), i32(1, 15), z(4)),
        lambda: lr.qknorm_fwd(q, q, z(8), z(8), i32(1, 16), z(5)), lambda: lr.qknorm_fwd(q, q, z(8), z(8), i32(1, 16).long(), z(4)),
        lambda: lr.qknorm_fwd(z(1, 257, 16), None, z(257), None), lambda: lr.qknorm_fwd(q, q, z(8), z(8), out=(q, None)),
        lambda: lr.qknorm_bwd(q, q, z(8), z(8), q, None), lambda: lr.qknorm_bwd(q, q, z(8), z(8), q[:, :, :8], q),
        lambda: lr.qknorm_step(q, q, z(8), z(8)), lambda: lr.qknorm_step(z(2, 8), z(2, 8), z(8), z(8), i32(3), z(4)),
        lambda: lr.state_move(s.transpose(1, 2), i32(1), i32(1)), lambda: lr.state_move(s, i32(2), i32(1)),
        lambda: lr.state_move(s, i32(1).long(), i32(1)), lambda: lr.state_move(s, i32(8193), i32(8193)),
        lambda: lr.state_move(z(4), i32(1), i32(1), layers=True)]


def test_binding_refuses_cpu_tensors(lr):
    q, v, A, s = torch.zeros(1, 8, 16), torch.zeros(1, 32, 16), torch.zeros(4), torch.zeros(2, 32, 8)
    i = torch.zeros(2, dtype=torch.int32)
    right = [lambda: lr.lattn_fwd(q, q, v, A), lambda: lr.lattn_bwd(q, q, v, A, None, None, None, v),
             lambda: lr.lattn_prompt(q[0], q[0], v[0], A, cu_seqlens=i, state=s),
             lambda: lr.lattn_step(q[0, :, :2].t(), q[0, :, :2].t(), v[0, :, :2].t(), A, state=s),
             lambda: lr.qknorm_fwd(q, q, torch.zeros(8), torch.zeros(8)), lambda: lr.qknorm_bwd(q, q, torch.zeros(8), torch.zeros(8), q, q),
             lambda: lr.qknorm_step(q[0], q[0], torch.zeros(16), torch.zeros(16)), lambda: lr.state_move(s, i, i)]
    for call in right + calls(lr, "cpu"):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu(lr):
    for n, call in enumerate(calls(lr, "cuda")):
        with pytest.raises(ValueError):
            call()
            print("not refused:", n)
