"""Host-only checks of the linear attention and norm-with-rotation entry points:
bad arguments are refused synchronously (every call below returns before any
CUDA runtime call), and the workspace sizes are pure functions."""
import ctypes

import pytest

import gated_deltanet_04_b200 as gdn
from gated_deltanet_04_b200 import build as gdn_build

P, MIS = 0x10000, 0x10008  # fake device addresses, the second misaligned
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    gdn_build.build()
    return gdn.library()


def prefill(lib, **kw):
    a = dict(q=P, k=P + 16, v=P + 32, dt=0, g=P + 48, scale=1.0, s0=None, cu=None, N=1, T=64, Hqk=16,
             Hv=48, Dk=128, Dv=128, o=P + 64, sT=None, ws=P + 80, wsb=1 << 40, err=None, st=None)
    a.update(kw)
    return lib.gdn_linear_prefill(*a.values())


BAD = [(dict(q=None), INVALID), (dict(g=None), INVALID), (dict(o=None), INVALID), (dict(k=MIS), INVALID),
       (dict(dt=3), INVALID), (dict(N=-1), INVALID), (dict(T=-1), INVALID), (dict(Hv=47), INVALID),
       (dict(Hqk=0), INVALID), (dict(N=2), INVALID), (dict(N=0), INVALID), (dict(Dk=96), UNSUPPORTED),
       (dict(Dv=256), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", BAD + [
    (dict(o=P), INVALID), (dict(s0=P + 64), INVALID), (dict(sT=P + 32), INVALID), (dict(sT=MIS), INVALID),
    (dict(ws=None, T=1 << 20), INVALID), (dict(wsb=16, T=1 << 20), INVALID), (dict(ws=P + 64), INVALID)])
def test_prefill_refuses(lib, kw, code):
    assert prefill(lib, **kw) == code


def slots(lib, **kw):
    a = dict(q=P, k=P + 16, v=P + 32, dt=0, g=P + 48, scale=1.0, pool=P + 96, num=4, idx=P + 112,
             reset=None, cu=None, N=1, T=64, Hqk=16, Hv=48, Dk=128, Dv=128, o=P + 64, ws=P + 80,
             wsb=1 << 40, err=None, st=None)
    a.update(kw)
    return lib.gdn_linear_prefill_slots(*a.values())


@pytest.mark.parametrize("kw,code", BAD + [
    (dict(pool=None), INVALID), (dict(idx=None), INVALID), (dict(num=0), INVALID), (dict(pool=P), INVALID),
    (dict(reset=MIS), INVALID), (dict(T=0, pool=None), INVALID)])
def test_prefill_slots_refuses(lib, kw, code):
    assert slots(lib, **kw) == code


def backward(lib, **kw):
    a = dict(o=P + 128, q=P, k=P + 16, v=P + 32, dt=0, g=P + 48, scale=1.0, s0=None, dsT=None, cu=None, N=1,
             T=64, Hqk=16, Hv=48, Dk=128, Dv=128, dq=P + 64, dk=P + 144, dv=P + 160, ds0=None, ws=P + 80,
             wsb=1 << 40, err=None, st=None)
    a.update(kw)
    return lib.gdn_linear_prefill_backward(*a.values())


@pytest.mark.parametrize("kw,code", BAD + [
    (dict(dq=None), INVALID), (dict(dk=P + 64), INVALID), (dict(dv=P), INVALID), (dict(ds0=MIS), INVALID),
    (dict(ws=None), INVALID), (dict(wsb=1000), INVALID), (dict(dsT=P + 160), INVALID),
    (dict(s0=P + 64), INVALID), (dict(ds0=P + 48), INVALID)])
def test_backward_refuses(lib, kw, code):
    assert backward(lib, **kw) == code


def decode(lib, **kw):
    a = dict(q=P, k=P + 16, v=P + 32, dt=0, g=P + 48, scale=1.0, state=P + 96, N=4, Hqk=16, Hv=48, Dk=128,
             Dv=128, o=P + 64, err=None, st=None)
    a.update(kw)
    return lib.gdn_linear_decode_step(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(g=None), INVALID), (dict(state=None), INVALID), (dict(o=None), INVALID),
    (dict(state=P), INVALID), (dict(o=P + 96), INVALID), (dict(k=MIS), INVALID), (dict(dt=2), INVALID),
    (dict(N=-1), INVALID), (dict(Hv=40), INVALID), (dict(Dv=0), INVALID), (dict(Dk=24), UNSUPPORTED),
    (dict(N=1 << 30), UNSUPPORTED)])
def test_decode_refuses(lib, kw, code):
    assert decode(lib, **kw) == code


def test_decode_slots_refuses(lib):
    f = lambda pool=P + 96, num=4, idx=P + 112, N=4: lib.gdn_linear_decode_step_slots(
        P, P + 16, P + 32, 0, P + 48, 1.0, pool, num, idx, None, N, 16, 48, 128, 128, P + 64, None, None)
    assert f(pool=None) == f(num=0) == f(idx=None) == f(idx=MIS) == f(N=-1) == INVALID


def test_nothing_to_do_is_ok(lib):
    assert prefill(lib, N=0, T=0, cu=P + 128) == 0
    assert prefill(lib, T=0, q=None, k=None, v=None, o=None, g=None, ws=None, wsb=0) == 0
    assert backward(lib, T=0, o=None, q=None, k=None, v=None, dq=None, dk=None, dv=None, ws=None, wsb=0) == 0
    assert decode(lib, N=0, q=None, k=None, v=None, state=None, o=None) == 0
    assert rope(lib, T=0, xq=None, xk=None, q=None, k=None) == 0


def test_workspace_bytes(lib):
    f, b = lib.gdn_linear_prefill_workspace_bytes, lib.gdn_linear_prefill_backward_workspace_bytes
    for args in ((1, 65536, 16, 48, 128, 128, 0), (3, 5000, 2, 4, 64, 32, 1), (1, 1, 1, 1, 16, 16, 1)):
        assert f(*args) == f(*args) and b(*args) >= 0
    for bad in ((-1, 10, 1, 1, 64, 64, 0), (1, -1, 1, 1, 64, 64, 0), (1, 10, 2, 3, 64, 64, 0),
                (1, 10, 1, 1, 65, 64, 0), (1, 10, 1, 1, 64, 64, 9), (1, 0, 1, 1, 64, 64, 0)):
        assert f(*bad) == 0 and b(*bad) == 0


def rope(lib, backward=False, **kw):
    a = dict(xq=P, xk=P + 16, dt=0, sq=24 * 256, sk=4 * 256, wq=None, wk=None, eps=1e-6, pos=P + 32, axes=1,
             sections=None, f=P + 48, rot=64, inter=0, T=8, Hq=24, Hk=4, D=256)
    out = dict(dxq=P + 64, dxk=P + 80, dsq=24 * 256, dsk=4 * 256, dwq=P + 96, dwk=P + 112, ws=P + 128,
               wsb=1 << 30) if backward else dict(q=P + 64, k=P + 80)
    for k, v in kw.items():
        (a if k in a else out)[k] = v
    if a["sections"] is not None:
        a["sections"] = (ctypes.c_int32 * len(a["sections"]))(*a["sections"])
    if backward:
        dz = [kw.get("dq", P + 144), kw.get("dk", P + 160)]
        out = {k: v for k, v in out.items() if k not in ("dq", "dk")}
        return lib.gdn_qk_norm_rope_backward(*dz, *a.values(), *out.values(), None)
    return lib.gdn_qk_norm_rope(*a.values(), *out.values(), None)


ROPE_BAD = [(dict(xq=None), INVALID), (dict(xk=None), INVALID), (dict(xq=MIS), INVALID), (dict(dt=9), INVALID),
            (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(pos=None), INVALID),
            (dict(f=None), INVALID), (dict(axes=0), INVALID), (dict(axes=2), INVALID),
            (dict(axes=2, sections=[16, 15]), INVALID), (dict(axes=2, sections=[-1, 33]), INVALID),
            (dict(axes=5, sections=[8, 8, 8, 4, 4]), UNSUPPORTED), (dict(rot=-16), INVALID),
            (dict(rot=272), INVALID), (dict(rot=24), UNSUPPORTED), (dict(inter=2), INVALID),
            (dict(sq=24 * 256 - 8), INVALID), (dict(sq=24 * 256 + 4), INVALID), (dict(Hq=0), INVALID),
            (dict(Hk=-1), INVALID), (dict(D=96, rot=96), UNSUPPORTED), (dict(T=-1), INVALID),
            (dict(Hq=32768, sq=32768 * 256), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", ROPE_BAD + [(dict(q=None), INVALID), (dict(k=None), INVALID),
                                                (dict(q=P), INVALID), (dict(k=P + 64), INVALID)])
def test_rope_refuses(lib, kw, code):
    assert rope(lib, **kw) == code


@pytest.mark.parametrize("kw,code", ROPE_BAD + [
    (dict(dq=None), INVALID), (dict(dxq=None), INVALID), (dict(dxk=P + 64), INVALID), (dict(dsq=8), INVALID),
    (dict(ws=None), INVALID), (dict(wsb=64), INVALID), (dict(dwq=P), INVALID)])
def test_rope_backward_refuses(lib, kw, code):
    assert rope(lib, backward=True, **kw) == code


def test_python_refuses_before_the_library():
    import torch

    x = torch.zeros(4, 2, 64)
    g = torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_linear_prefill(x, x, x, g)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_linear_decode_step(x, x, x, g, torch.zeros(4, 2, 64, 64))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_qk_norm_rope(x)
