"""GPU parity of gdn_qk_norm_rope and its backward pass against the fp64 oracle.

Tolerances, from the arithmetic, with u = 2^-24 (half a step of fp32) and a row
of D elements: the mean of squares is within (D + 2) u, its inverse root
(rsqrtf, 2 ulp) and the products add a few more; an angle is within 2^-24 turns
after the fp64 reduction, which turns a pair of length L by 2 pi 2^-24 L, and
sincospif adds 2 ulp.  So every output is within (D + 64) u of its pair's (row's)
largest magnitude, plus half a step of the output type.  Weight gradients are
fp32 sums of T H products each within (D + 64) u of its terms.
"""
import numpy as np
import pytest
import torch

import gated_deltanet_04_b200 as gdn
import oracle
from tests.helpers import Guarded

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gated_deltanet_04_b200 import build
    build.build()


def make(T, Hq, Hk, D, R, dt, axes=1, seed=0, far=True, weights=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    pos = torch.randint(-5, 1 << 20 if far else 50, (axes, T), generator=gen, dtype=torch.int32)
    cut = [R // 2 // axes] * (axes - 1)
    return dict(xq=r(T, Hq, D).to(dt), xk=r(T, Hk, D).to(dt) if Hk else None, dq=r(T, Hq, D).to(dt),
                dk=r(T, Hk, D).to(dt) if Hk else None, wq=1 + 0.3 * r(D) if weights else None,
                wk=1 + 0.3 * r(D) if weights else None, pos=pos if R else None,
                f=(1e6 ** (-torch.arange(0, R, 2).double() / max(R, 1))).float() if R else None,
                sections=cut + [R // 2 - sum(cut)] if axes > 1 else None, dt=dt, D=D)


def dev(x):
    return None if x is None else x.to(DEV).contiguous()


def close(x, ref, dt, D, what):
    x = x.detach().cpu().double().numpy()
    row = np.max(np.abs(ref), axis=-1, keepdims=True)
    tol = (D + 64) * 2.0 ** -24
    lim = tol * 2 * row + torch.finfo(dt).eps / 2 * (np.abs(ref) + 2 * tol * row) + 1e-37
    worst = float(np.max(np.abs(x - ref) / lim)) if x.size else 0.0
    assert worst <= 1, f"{what}: {worst:.3g} times the bound"


def kw(c, interleaved):
    return dict(sections=c["sections"], interleaved=interleaved)


def check(c, interleaved=False, eps=1e-6):
    T, Hq, D = c["xq"].shape
    pos = None if c["pos"] is None else dev(c["pos"] if c["sections"] else c["pos"][0])
    outs = [None if x is None else Guarded(tuple(x.shape), c["dt"], DEV) for x in (c["xq"], c["xk"])]
    t = lambda g: None if g is None else g.t
    q, k = gdn.gdn_qk_norm_rope(dev(c["xq"]), dev(c["xk"]), pos, dev(c["f"]), wq=dev(c["wq"]), wk=dev(c["wk"]),
                                eps=eps, q=t(outs[0]), k=t(outs[1]), **kw(c, interleaved))
    dxq, dxk, dwq, dwk = gdn.gdn_qk_norm_rope_backward(
        dev(c["dq"]), dev(c["dk"]), dev(c["xq"]), dev(c["xk"]), pos, dev(c["f"]), wq=dev(c["wq"]),
        wk=dev(c["wk"]), eps=eps, **kw(c, interleaved))
    torch.cuda.synchronize()
    for x, z, w, dz, dx, dw, g in ((c["xq"], q, c["wq"], c["dq"], dxq, dwq, outs[0]),
                                   (c["xk"], k, c["wk"], c["dk"], dxk, dwk, outs[1])):
        if x is None:
            assert z is None and dx is None and dw is None
            continue
        g.check()
        ref = oracle.qk_norm_rope(x, w, eps, c["pos"], c["f"], **kw(c, interleaved))
        close(z, ref, c["dt"], D, "out")
        rdx, rdw = oracle.qk_norm_rope_backward(dz, x, w, eps, c["pos"], c["f"], **kw(c, interleaved))
        close(dx, rdx, c["dt"], D, "dx")
        # every product dy n of the sum, in absolute values
        n = oracle.qk_norm_rope(x, None, eps, None, None)
        dy = oracle.qk_norm_rope(dz, None, eps, c["pos"], c["f"], inverse=True, norm=False, **kw(c, interleaved))
        row = np.max(np.abs(dy), axis=-1, keepdims=True)
        A = np.sum(row * np.abs(n), axis=(0, 1))
        lim = (T + D + 64) * 2.0 ** -23 * A + 1e-37
        assert np.all(np.abs(dw.cpu().double().numpy() - rdw) <= lim), "dw"


@pytest.mark.parametrize("dt", [F32, BF], ids=str)
@pytest.mark.parametrize("T,Hq,Hk,D,R", [(1, 1, 1, 16, 16), (3, 2, 1, 32, 16), (17, 5, 3, 64, 48), (130, 3, 3, 64, 64),
                                         (33, 6, 2, 128, 128), (64, 4, 1, 128, 80), (21, 24, 4, 256, 64),
                                         (9, 2, 2, 256, 256), (50, 1, 0, 128, 32), (12, 3, 1, 128, 0)])
def test_matches_oracle(T, Hq, Hk, D, R, dt):
    check(make(T, Hq, Hk, D, R, dt, seed=T + D))


@pytest.mark.parametrize("dt", [F32, BF], ids=str)
def test_interleaved_pairs(dt):
    for T, D, R in ((40, 64, 64), (7, 128, 48), (5, 16, 16)):
        check(make(T, 4, 2, D, R, dt, seed=T), interleaved=True)


@pytest.mark.parametrize("axes", [2, 3, 4])
def test_position_axes(axes):
    check(make(45, 4, 2, 128, 96, F32, axes=axes, seed=axes))
    check(make(45, 4, 2, 64, 32, BF, axes=axes, seed=axes), interleaved=True)
    c = make(20, 2, 2, 64, 32, F32, axes=2)
    c["sections"] = [0, 16]
    check(c)
    c["sections"] = [16, 0]
    check(c)


def test_many_rows():
    """Enough rows for the kernels' four-row form, a ragged end, and no weights."""
    check(make(3001, 24, 1, 64, 64, BF, seed=3, weights=False))
    check(make(2001, 13, 3, 256, 64, F32, seed=4))
    check(make(40001, 1, 1, 16, 16, F32, seed=5))


def test_zero_and_large_rows():
    c = make(6, 2, 1, 64, 32, F32, seed=9)
    c["xq"][2] = 0
    c["xk"][3] = 0
    check(c, eps=1e-5)
    c["xq"][1] *= 1e15
    c["xk"][0] *= 1e-15
    check(c, eps=1e-5)


def test_far_positions_keep_the_angle():
    """Relative positions: rotating q at p + d and k at p gives the same product
    at any p, 2^31 - 1 included, to the angles' accuracy."""
    D = 128
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(2, 1, 1, D, generator=gen).to(DEV)
    f = (1e7 ** (-torch.arange(0, D, 2).double() / D)).float().to(DEV)
    dots = []
    for p in (0, 1000, 262143, (1 << 31) - 8):
        pos = [torch.tensor([p + d], dtype=torch.int32, device=DEV) for d in (7, 0)]
        q, _ = gdn.gdn_qk_norm_rope(x[0], None, pos[0], f)
        k, _ = gdn.gdn_qk_norm_rope(x[1], None, pos[1], f)
        dots.append(float((q.double() * k.double()).sum()))
    # 64 pairs of length ~ sqrt(2) each, turned to 2^-22 of a turn at the farthest
    assert max(dots) - min(dots) <= 64 * 2 * 2 * np.pi * 2.0 ** -21


def test_strided_parts_of_a_projection():
    T, Hq, Hk, D = 37, 6, 2, 128
    for dt in (BF, F32):
        c = make(T, Hq, Hk, D, 64, dt, seed=6)
        W = (Hq + 2 * Hk) * D
        x = torch.randn(T, W, generator=torch.Generator().manual_seed(1)).to(dt).to(DEV)
        part = lambda t: (t[:, :Hq * D].unflatten(1, (Hq, D)), t[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)))
        xq, xk = part(x)
        a = dict(wq=dev(c["wq"]), wk=dev(c["wk"]))
        pos, f = dev(c["pos"][0]), dev(c["f"])
        got = gdn.gdn_qk_norm_rope(xq, xk, pos, f, **a)
        want = gdn.gdn_qk_norm_rope(xq.contiguous(), xk.contiguous(), pos, f, **a)
        assert all(torch.equal(g, w) for g, w in zip(got, want))
        dx = torch.full_like(x, 3.0)
        dxq, dxk = part(dx)
        got = gdn.gdn_qk_norm_rope_backward(dev(c["dq"]), dev(c["dk"]), xq, xk, pos, f, dxq=dxq, dxk=dxk, **a)
        want = gdn.gdn_qk_norm_rope_backward(dev(c["dq"]), dev(c["dk"]), xq.contiguous(), xk.contiguous(), pos,
                                             f, **a)
        assert all(torch.equal(g, w) for g, w in zip(got, want))
        assert bool((dx[:, (Hq + Hk) * D:] == 3).all())


def test_no_rows():
    z = torch.empty(0, 2, 64, dtype=BF, device=DEV)
    f = torch.ones(16, device=DEV)
    pos = torch.empty(0, dtype=torch.int32, device=DEV)
    q, k = gdn.gdn_qk_norm_rope(z, z, pos, f)
    assert q.shape == k.shape == (0, 2, 64)
    dxq, dxk, dwq, dwk = gdn.gdn_qk_norm_rope_backward(z, z, z, z, pos, f)
    assert dxq.numel() == dxk.numel() == 0 and not bool(dwq.any()) and not bool(dwk.any())


def test_repeatable_side_stream_and_graph():
    c = make(2100, 12, 4, 128, 64, BF, seed=8)
    a = [dev(c[x]) for x in ("dq", "dk", "xq", "xk")] + [dev(c["pos"][0]), dev(c["f"])]
    w = dict(wq=dev(c["wq"]), wk=dev(c["wk"]))
    first = gdn.gdn_qk_norm_rope(*a[2:], **w) + gdn.gdn_qk_norm_rope_backward(*a, **w)
    again = gdn.gdn_qk_norm_rope(*a[2:], **w) + gdn.gdn_qk_norm_rope_backward(*a, **w)
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    side = torch.cuda.Stream(DEV)
    torch.cuda.synchronize()
    other = gdn.gdn_qk_norm_rope(*a[2:], **w, stream=side) + gdn.gdn_qk_norm_rope_backward(*a, **w, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gdn.gdn_qk_norm_rope(*a[2:], **w) + gdn.gdn_qk_norm_rope_backward(*a, **w)
    a[2].copy_(a[2].flip(0))
    graph.replay()
    want = gdn.gdn_qk_norm_rope(*a[2:], **w) + gdn.gdn_qk_norm_rope_backward(*a, **w)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert not torch.equal(got[0], first[0])
