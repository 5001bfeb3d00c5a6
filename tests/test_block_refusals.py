"""What the operators around the scan refuse, before anything is launched: the
binding on tensors, the C ABI on sizes, flags and missing pointers."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails first


def _call(lr, name, base, **change):
    args = dict(base)
    args.update(change)
    return getattr(lr.lib(), name)(*args.values())


SCONV_FWD = dict(x=FAKE, weight=FAKE, bias=None, x0=None, y=FAKE, final=None, batch=1, dim=4, len=8, width=4, bs=32, ds=8,
                 dtype=0, flags=1, stream=None)
SCONV_BWD = dict(x=FAKE, weight=FAKE, bias=None, x0=None, dy=FAKE, dfinal=None, dx=FAKE, dweight=FAKE, dbias=None, dx0=None,
                 batch=1, dim=4, len=8, width=4, bs=32, ds=8, dtype=0, flags=1, stream=None)
SCONV_PROMPT = dict(x=FAKE, weight=FAKE, bias=None, cu=FAKE, slots=None, has=None, state=FAKE, y=FAKE, requests=1, rows=1,
                    dim=4, tokens=8, width=4, ds=8, dtype=0, flags=1, stream=None)
SCONV_STEP = dict(x=FAKE, weight=FAKE, bias=None, slots=None, state=FAKE, y=FAKE, batch=1, rows=1, dim=4, width=4, xs=4,
                  dtype=0, flags=1, stream=None)
SSCAN_PROMPT = dict(u=FAKE, delta=FAKE, A=FAKE, B=FAKE, C=FAKE, D=None, z=None, bias=None, cu=FAKE, slots=None, has=None,
                    state=FAKE, out=FAKE, requests=1, rows=1, dim=4, tokens=8, N=16, dtype=0, flags=0, segments=0, stream=None)
SSCAN_STEP = dict(u=FAKE, delta=FAKE, A=FAKE, B=FAKE, C=FAKE, D=None, z=None, bias=None, slots=None, state=FAKE, out=FAKE,
                  batch=1, rows=1, dim=4, N=16, zs=4, dtype=0, flags=0, stream=None)
ADD_FWD = dict(x=FAKE, residual=None, weight=FAKE, y=FAKE, r=FAKE, rows=1, width=8, scale=1.0, eps=1e-5, dtype=0, stream=None)
ADD_BWD = dict(r=FAKE, weight=FAKE, dy=FAKE, dr=None, dx=FAKE, dres=None, dweight=FAKE, rows=1, width=8, scale=1.0, eps=1e-5,
               dtype=0, stream=None)
GATE_FWD = dict(y=FAKE, z=FAKE, weight=FAKE, out=FAKE, batch=1, dim=8, len=4, groups=1, bs=32, ds=4, eps=1e-5, dtype=0,
                flags=0, stream=None)
GATE_BWD = dict(y=FAKE, z=FAKE, weight=FAKE, dout=FAKE, dy=FAKE, dz=FAKE, dweight=FAKE, batch=1, dim=8, len=4, groups=1,
                bs=32, ds=4, eps=1e-5, dtype=0, flags=0, stream=None)
GATE_STEP = dict(y=FAKE, z=FAKE, weight=FAKE, out=FAKE, rows=1, dim=8, groups=1, zs=8, eps=1e-5, dtype=0, flags=0, stream=None)

BAD = [("sconv_fwd", SCONV_FWD, c) for c in (
    dict(x=None), dict(weight=None), dict(y=None), dict(width=1), dict(width=5), dict(dtype=2), dict(flags=2), dict(batch=-1),
    dict(len=-1), dict(bs=-1), dict(dim=1 << 39, len=1 << 20), dict(dim=1 << 31))]
BAD += [("sconv_bwd", SCONV_BWD, c) for c in (dict(dy=None), dict(dx=None), dict(dweight=None), dict(width=0), dict(flags=8))]
BAD += [("sconv_prompt", SCONV_PROMPT, c) for c in (
    dict(cu=None), dict(state=None), dict(requests=2), dict(requests=-1), dict(tokens=1 << 31), dict(x=None), dict(width=6))]
BAD += [("sconv_step", SCONV_STEP, c) for c in (dict(batch=2), dict(state=None), dict(y=None), dict(xs=-4), dict(dtype=7))]
BAD += [("sscan_prompt", SSCAN_PROMPT, c) for c in (
    dict(u=None), dict(A=None), dict(cu=None), dict(state=None), dict(N=0), dict(N=65), dict(flags=2), dict(segments=-1),
    dict(requests=2), dict(tokens=1 << 31), dict(dtype=-1))]
BAD += [("sscan_step_slots", SSCAN_STEP, c) for c in (
    dict(u=None), dict(state=None), dict(N=65), dict(flags=2), dict(batch=2), dict(zs=-1), dict(batch=-1))]
BAD += [("addnorm_fwd", ADD_FWD, c) for c in (dict(x=None), dict(r=None), dict(width=0), dict(width=16385), dict(rows=-1), dict(dtype=2))]
BAD += [("addnorm_bwd", ADD_BWD, c) for c in (dict(dweight=None), dict(dx=None), dict(width=16385), dict(dtype=2))]
BAD += [("gatenorm_fwd", GATE_FWD, c) for c in (dict(y=None), dict(groups=3), dict(groups=0), dict(flags=2), dict(bs=-1), dict(dtype=2))]
BAD += [("gatenorm_bwd", GATE_BWD, c) for c in (dict(dout=None), dict(dweight=None), dict(groups=3), dict(flags=4))]
BAD += [("gatenorm_step", GATE_STEP, c) for c in (dict(z=None), dict(dim=16392), dict(groups=5), dict(zs=-1))]


@pytest.mark.parametrize("name,base,change", BAD, ids=[f"{n}-{'-'.join(f'{k}={v}' for k, v in c.items())}" for n, _, c in BAD])
def test_abi_refuses(lr, name, base, change):
    assert _call(lr, name, base, **change) == lr.SSCAN_ERR_INVALID
    assert lr.last_launch_count() == 0 and lr.last_plan() == "rejected"


@pytest.mark.parametrize("name,base,change", [
    ("sconv_fwd", SCONV_FWD, dict(batch=0)), ("sconv_bwd", SCONV_BWD, dict(dim=0)), ("sconv_step", SCONV_STEP, dict(batch=0)),
    ("sconv_prompt", SCONV_PROMPT, dict(dim=0)), ("sscan_prompt", SSCAN_PROMPT, dict(requests=0, tokens=0)),
    ("sscan_step_slots", SSCAN_STEP, dict(batch=0)), ("addnorm_fwd", ADD_FWD, dict(rows=0)),
    ("gatenorm_fwd", GATE_FWD, dict(len=0)), ("gatenorm_bwd", GATE_BWD, dict(dim=0)), ("gatenorm_step", GATE_STEP, dict(rows=0))])
def test_abi_takes_empty_problems(lr, name, base, change):
    assert _call(lr, name, base, **change) == lr.SSCAN_OK
    assert lr.last_launch_count() == 0 and lr.last_plan() == "empty"


def test_binding_refuses_cpu_tensors_and_wrong_shapes(lr):
    x3, x2, w = torch.zeros(1, 4, 8), torch.zeros(4, 8), torch.zeros(4, 4)
    cu = torch.tensor([0, 8], dtype=torch.int32)
    for call in (lambda: lr.sconv_fwd(x3, w), lambda: lr.sconv_bwd(x3, w, None, None, x3),
                 lambda: lr.sconv_prompt(x2, w, cu_seqlens=cu, state=torch.zeros(1, 4, 3)),
                 lambda: lr.sconv_step(x2, w, state=torch.zeros(4, 8, 3)),
                 lambda: lr.sscan_prompt(x2, x2, w, x2, x2, cu_seqlens=cu, state=torch.zeros(1, 4, 4)),
                 lambda: lr.addnorm_fwd(x2, None, torch.zeros(8)), lambda: lr.addnorm_bwd(x2, torch.zeros(8), x2),
                 lambda: lr.gatenorm_fwd(x3, x3, torch.zeros(4)), lambda: lr.gatenorm_bwd(x3, x3, torch.zeros(4), x3),
                 lambda: lr.gatenorm_step(x2, x2, torch.zeros(8)),
                 lambda: lr.sconv_fwd(x2, w), lambda: lr.addnorm_fwd(x3, None, torch.zeros(8))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu(lr):
    dev = "cuda"
    x, w = torch.zeros(1, 4, 8, device=dev), torch.zeros(4, 4, device=dev)
    x2 = x[0]
    cu = torch.tensor([0, 8], dtype=torch.int32, device=dev)
    bad = [lambda: lr.sconv_fwd(x.half(), w), lambda: lr.sconv_fwd(x, torch.zeros(4, 5, device=dev)),
           lambda: lr.sconv_fwd(x, w.double()), lambda: lr.sconv_fwd(x.transpose(1, 2), torch.zeros(8, 4, device=dev)),
           lambda: lr.sconv_fwd(x, w, None, torch.zeros(1, 4, 2, device=dev)),
           lambda: lr.sconv_prompt(x2, w, cu_seqlens=cu.long(), state=torch.zeros(1, 4, 3, device=dev)),
           lambda: lr.sconv_prompt(x2, w, cu_seqlens=cu, state=torch.zeros(0, 4, 3, device=dev)),
           lambda: lr.sconv_prompt(x2, w, cu_seqlens=cu, state=torch.zeros(1, 4, 3, device=dev), has_state=cu[:1]),
           lambda: lr.sconv_step(x2, torch.zeros(8, 4, device=dev), state=torch.zeros(3, 8, 3, device=dev)),
           lambda: lr.sscan_prompt(x2, x2, w, x2[:3], x2, cu_seqlens=cu, state=torch.zeros(1, 4, 4, device=dev)),
           lambda: lr.sscan_prompt(x2, x2, w, x2, x2, cu_seqlens=cu, state=torch.zeros(1, 4, 4, device=dev).bfloat16()),
           lambda: lr.sscan_step(x2, x2, torch.zeros(8, 4, device=dev), w, w, state=torch.zeros(9, 8, 4, device=dev),
                                 slots=torch.zeros(3, dtype=torch.int32, device=dev)),
           lambda: lr.addnorm_fwd(x2, x2.bfloat16(), torch.zeros(8, device=dev)),
           lambda: lr.addnorm_fwd(x2.t(), None, torch.zeros(4, device=dev)),
           lambda: lr.gatenorm_fwd(x, x, torch.zeros(4, device=dev), groups=3),
           lambda: lr.gatenorm_bwd(x, x.bfloat16(), torch.zeros(4, device=dev), x),
           lambda: lr.gatenorm_step(x2, x2[:, :4], torch.zeros(8, device=dev))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(lr.SscanError):
        lr.addnorm_fwd(torch.zeros(1, 16385, device=dev), None, torch.zeros(16385, device=dev))
