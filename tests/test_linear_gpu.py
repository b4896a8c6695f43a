"""GPU parity of linear attention with a decay per head (gdn_linear_*) against
the fp64 oracle.

Tolerances, element by element, from the arithmetic.  Let A be the same
quantity computed from absolute values (the sum of the absolute terms; the
oracle on |q|, |k|, |v|, ...).
* An fp32 sum of n products in any order is within (n + 4) 2^-24 A.  A decay
  applied once per token adds one rounding per token, so the recurrent kernels
  are within (2 len + D + 8) 2^-24 A.
* The tensor-core kernels round the score (or state) operand to bf16, half a
  step, 2^-8, of each term, plus sums of at most a chunk's products and one
  rounding per chunk: within (2^-8 + 2^-10) A.  In the gradients the rows that
  meet a state are scaled by their decay and rounded as well, a second half
  step of those terms: within (2 2^-8 + 2^-10) A.  Their fp32 states take the
  value operand as two bf16 parts, 2^-16 of each term: within 2^-15 A.
* An output is rounded once: half a step of its type, 2^-8 for bf16.
"""
import numpy as np
import pytest
import torch

import gated_deltanet_04_b200 as gdn
import oracle
from gated_deltanet_04_b200 import inputs
from tests.helpers import Guarded

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gated_deltanet_04_b200 import build
    build.build()


def tensor_core(dt, Dk, Dv):
    return dt == BF and Dk == 128 and Dv == 128


def decays(Hv, kind):
    h = torch.arange(1, Hv + 1, dtype=torch.float64)
    return {"slopes": -(2.0 ** (-8.0 * h / Hv)), "none": 0 * h, "slow": -1e-4 * h,
            "strong": -6.0 * h / Hv, "mixed": torch.where(h % 2 == 0, -0.0 * h, -20.0 / h)}[kind].float()


def make(lens, Hqk, Hv, Dk, Dv, dt, seed, decay="slopes", state=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    T, N = sum(lens), len(lens)
    return dict(q=r(T, Hqk, Dk).to(dt), k=r(T, Hqk, Dk).to(dt), v=r(T, Hv, Dv).to(dt),
                do=r(T, Hv, Dv).to(dt), g=decays(Hv, decay), lens=lens, dt=dt,
                s0=r(N, Hv, Dv, Dk) if state else None, dsT=r(N, Hv, Dv, Dk) if state else None,
                cu=inputs.cu_from_lengths(lens).to(torch.int32), scale=Dk ** -0.5)


def dev(x):
    return None if x is None else x.to(DEV).contiguous()


def absd(c):
    return {k: (x.abs() if isinstance(x, torch.Tensor) and x.is_floating_point() and k != "g" else x)
            for k, x in c.items()}


def ulp_half(dt):
    return torch.finfo(dt).eps / 2


def slack(c, Dk, Dv, state=False, roundings=1):
    n = max(c["lens"]) if c["lens"] else 0
    if tensor_core(c["dt"], Dk, Dv):
        return 2.0 ** -15 if state else roundings * 2.0 ** -8 + 2.0 ** -10
    return (2 * n + max(Dk, Dv) + 8) * 2.0 ** -24


def close(x, ref, A, tol, dt, what):
    x = x.detach().cpu().double().numpy()
    err = np.abs(x - ref)
    lim = tol * A + ulp_half(dt) * (np.abs(ref) + tol * A) + 1e-37
    assert np.isfinite(x).all() == np.isfinite(ref).all(), what
    worst = float(np.max(err / lim)) if x.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"


def run_prefill(c, **kw):
    flag = torch.zeros(4, dtype=torch.int32, device=DEV)
    T, Hv, Dv = c["v"].shape
    o = Guarded((T, Hv, Dv), c["dt"], DEV)
    sT = Guarded((len(c["lens"]), Hv, Dv, c["q"].shape[2]), F32, DEV)
    gdn.gdn_linear_prefill(dev(c["q"]), dev(c["k"]), dev(c["v"]), dev(c["g"]), dev(c["s0"]), dev(c["cu"]),
                           scale=c["scale"], o=o.t, final_state=sT.t, error_flag=flag, **kw)
    torch.cuda.synchronize()
    assert int(flag[0]) == 0
    o.check("o")
    sT.check("final_state")
    return o.t, sT.t


def check_prefill(c, o, sT):
    Dk, Dv = c["q"].shape[2], c["v"].shape[2]
    args = lambda x: (x["q"], x["k"], x["v"], c["g"], x["s0"], c["cu"])
    o_ref, s_ref = oracle.linear_recurrent(*args(c), scale=c["scale"])
    o_abs, s_abs = oracle.linear_recurrent(*args(absd(c)), scale=c["scale"])
    close(o, o_ref, o_abs, slack(c, Dk, Dv), c["dt"], "o")
    close(sT, s_ref, s_abs, slack(c, Dk, Dv, True), F32, "final_state")


SHAPES = [  # (Hqk, Hv, Dk, Dv, dtype)
    (1, 1, 16, 16, F32), (2, 4, 64, 64, F32), (1, 3, 32, 128, F32), (2, 2, 128, 16, BF), (1, 2, 64, 64, BF),
    (1, 2, 128, 128, F32), (2, 6, 128, 128, BF), (3, 3, 128, 128, BF),
]
LENS = [[1], [127], [128], [129], [300], [0, 1, 2, 0, 257, 64, 0], [5, 130, 128, 260]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_prefill_matches_oracle(shape, lens):
    c = make(lens, *shape, seed=100 + sum(lens))
    check_prefill(c, *run_prefill(c))


@pytest.mark.parametrize("decay", ["none", "slow", "strong", "mixed"])
@pytest.mark.parametrize("shape", [(1, 2, 64, 32, F32), (1, 2, 128, 128, BF)], ids=str)
def test_prefill_decays(shape, decay):
    c = make([300, 1, 140], *shape, seed=7, decay=decay)
    check_prefill(c, *run_prefill(c))


def test_prefill_many_chunks_and_segments():
    """Long enough that the sequence is cut into segments (both kernel families)."""
    for shape in [(1, 1, 32, 32, F32), (1, 2, 128, 128, BF)]:
        c = make([3000, 17, 1200], *shape, seed=11, decay="slow")
        check_prefill(c, *run_prefill(c))


def test_prefill_without_cu_or_state_and_in_place():
    for shape in [(2, 4, 32, 64, F32), (1, 3, 128, 128, BF)]:
        c = make([513], *shape, seed=13)
        o1, s1 = run_prefill(c)
        st = dev(c["s0"]).clone()
        o2, s2 = gdn.gdn_linear_prefill(dev(c["q"]), dev(c["k"]), dev(c["v"]), dev(c["g"]), st, None,
                                        scale=c["scale"], final_state=st)
        assert s2 is st and torch.equal(o1, o2) and torch.equal(s1, st)
        c["s0"] = None
        check_prefill(c, *run_prefill(c))


def test_prefill_split_and_carry():
    """Splitting a sequence anywhere and carrying the state gives the one-shot
    result to the tolerance of one more state rounding."""
    for shape in [(1, 2, 64, 64, F32), (1, 2, 128, 128, BF)]:
        c = make([400], *shape, seed=17)
        _, s_ref = oracle.linear_recurrent(c["q"], c["k"], c["v"], c["g"], c["s0"], c["cu"], scale=c["scale"])
        a = absd(c)
        _, s_abs = oracle.linear_recurrent(a["q"], a["k"], a["v"], c["g"], a["s0"], c["cu"], scale=c["scale"])
        for cut in (1, 127, 128, 200, 399):
            st = dev(c["s0"])
            for lo, hi in ((0, cut), (cut, 400)):
                part = [dev(c[x][lo:hi]) for x in "qkv"]
                _, st = gdn.gdn_linear_prefill(*part, dev(c["g"]), st, scale=c["scale"])
            close(st, s_ref, s_abs, 2 * slack(c, shape[2], shape[3], True), F32, f"cut {cut}")


def test_prefill_no_tokens():
    for dt in (F32, BF):
        s0 = torch.randn(2, 3, 128, 128, device=DEV)
        z = torch.empty(0, 3, 128, dtype=dt, device=DEV)
        g = decays(3, "slopes").to(DEV)
        o, sT = gdn.gdn_linear_prefill(z, z, z, g, s0, torch.zeros(3, dtype=torch.int32, device=DEV))
        assert o.shape == (0, 3, 128) and torch.equal(sT, s0)
        dq, dk, dv, ds0 = gdn.gdn_linear_prefill_backward(
            z, z, z, z, g, s0, torch.zeros(3, dtype=torch.int32, device=DEV), dfinal_state=s0,
            output_dinitial_state=True)
        assert dq.numel() == dk.numel() == dv.numel() == 0 and torch.equal(ds0, s0)


def test_other_rows_do_not_leak_into_a_sequence():
    """NaN and infinities in one sequence's inputs leave its neighbours' results
    as they are, to the bit."""
    for shape in [(1, 2, 64, 64, F32), (1, 2, 128, 128, BF)]:
        c = make([70, 90, 130], *shape, seed=19)
        o1, s1 = run_prefill(c)
        g1 = run_backward(c)
        bad = dict(c)
        for x, val in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("do", float("-inf"))):
            bad[x] = c[x].clone()
            bad[x][70:160] = val
        o2, s2 = run_prefill(bad)
        g2 = run_backward(bad)
        keep = [i for i in range(290) if not 70 <= i < 160]
        assert torch.equal(o1[keep], o2[keep])
        assert torch.equal(s1[[0, 2]], s2[[0, 2]])
        for x, y in zip(g1[:3], g2[:3]):
            assert torch.equal(x[keep], y[keep])
        assert torch.equal(g1[3][[0, 2]], g2[3][[0, 2]])


def run_backward(c, **kw):
    flag = torch.zeros(4, dtype=torch.int32, device=DEV)
    outs = [Guarded(tuple(c[x].shape), c["dt"], DEV) for x in "qkv"]
    ds0 = Guarded((len(c["lens"]), c["v"].shape[1], c["v"].shape[2], c["q"].shape[2]), F32, DEV)
    gdn.gdn_linear_prefill_backward(dev(c["do"]), dev(c["q"]), dev(c["k"]), dev(c["v"]), dev(c["g"]),
                                    dev(c["s0"]), dev(c["cu"]), dfinal_state=dev(c["dsT"]),
                                    scale=c["scale"], dq=outs[0].t, dk=outs[1].t, dv=outs[2].t,
                                    dinitial_state=ds0.t, error_flag=flag, **kw)
    torch.cuda.synchronize()
    assert int(flag[0]) == 0
    for x, name in zip(outs + [ds0], ("dq", "dk", "dv", "dinitial_state")):
        x.check(name)
    return [x.t for x in outs] + [ds0.t]


def check_backward(c, got):
    Dk, Dv = c["q"].shape[2], c["v"].shape[2]
    f = lambda x: oracle.linear_backward(x["do"], x["q"], x["k"], x["v"], c["g"], x["s0"], c["cu"],
                                         dsT=x["dsT"], scale=c["scale"])
    G = c["v"].shape[1] // c["q"].shape[1]
    for name, x, ref, A in zip(("dq", "dk", "dv", "ds0"), got, f(c), f(absd(c))):
        st = name == "ds0"
        # a group's heads add G further roundings to fp32 sums
        close(x, ref, A, slack(c, Dk, Dv, st, roundings=2) + G * 2.0 ** -24, F32 if st else c["dt"], name)


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward_matches_oracle(shape, lens):
    c = make(lens, *shape, seed=200 + sum(lens))
    check_backward(c, run_backward(c))


@pytest.mark.parametrize("decay", ["none", "slow", "strong", "mixed"])
@pytest.mark.parametrize("shape", [(1, 2, 64, 32, F32), (1, 2, 128, 128, BF)], ids=str)
def test_backward_decays(shape, decay):
    c = make([300, 1, 140], *shape, seed=23, decay=decay)
    check_backward(c, run_backward(c))


def test_backward_segments_and_groups():
    for shape in [(1, 2, 32, 32, F32), (1, 5, 128, 128, BF)]:
        c = make([2300, 17, 900], *shape, seed=29, decay="slow")
        check_backward(c, run_backward(c))


@pytest.mark.parametrize("lens", [[2], [3], [4, 3, 0, 5], [9, 1] * 12], ids=str)
def test_backward_of_short_sequences(lens):
    c = make(lens, 2, 6, 128, 128, BF, seed=33 + sum(lens))
    check_backward(c, run_backward(c))


def test_backward_without_states_and_in_place():
    for shape in [(2, 4, 32, 64, F32), (1, 3, 128, 128, BF)]:
        c = make([513], *shape, seed=31)
        full = run_backward(c)
        g = dev(c["dsT"]).clone()
        got = gdn.gdn_linear_prefill_backward(dev(c["do"]), dev(c["q"]), dev(c["k"]), dev(c["v"]), dev(c["g"]),
                                              dev(c["s0"]), None, dfinal_state=g, scale=c["scale"],
                                              dinitial_state=g)
        assert got[3] is g and all(torch.equal(x, y) for x, y in zip(full, got))
        c["s0"] = c["dsT"] = None
        check_backward(c, run_backward(c))


def test_backward_against_differences():
    """fp32 gradients against central differences of the forward call's own
    loss, in directions of all inputs at once: the forward's fp32 error e of the
    loss leaves 2 e / (2 h) in the quotient, the third order of the trilinear
    form h^2 of the loss's own cubic term."""
    c = make([37, 0, 70], 2, 4, 32, 32, F32, seed=37)
    dq, dk, dv, ds0 = run_backward(c)
    gen = torch.Generator().manual_seed(38)
    w, wT = c["do"].double(), c["dsT"].double()

    def loss(h, d):
        x = dict(c)
        for name in ("q", "k", "v", "s0"):
            x[name] = (c[name] + h * d[name]).float()
        o, sT = run_prefill(x)
        return float((o.cpu().double() * w).sum() + (sT.cpu().double() * wT).sum())

    for _ in range(4):
        d = {n: torch.randn(c[n].shape, generator=gen) for n in ("q", "k", "v", "s0")}
        want = sum(float((g.cpu().double() * d[n].double()).sum())
                   for n, g in (("q", dq), ("k", dk), ("v", dv), ("s0", ds0)))
        h = 1e-2
        got = (loss(h, d) - loss(-h, d)) / (2 * h)
        # the cubic term, from a second step length, bounds the truncation
        got2 = (loss(2 * h, d) - loss(-2 * h, d)) / (4 * h)
        assert abs(got - want) <= abs(got2 - got) + 2e-4 * (abs(want) + float(w.abs().sum()))


def test_slots_prefill_then_decode():
    """Prefill into pool slots and single-token steps from them, with new
    requests: the oracle's recurrence over the same tokens."""
    for shape in [(1, 2, 64, 64, F32), (2, 4, 128, 128, BF), (1, 1, 16, 128, BF)]:
        Hqk, Hv, Dk, Dv, dt = shape
        c = make([40, 1, 150], *shape, seed=41)
        step = make([1, 1, 1], *shape, seed=42)
        pool = torch.randn(6, Hv, Dv, Dk)
        slots = torch.tensor([4, 0, 2], dtype=torch.int32)
        reset = torch.tensor([0, 1, 0], dtype=torch.int32)
        s0 = torch.stack([torch.zeros_like(pool[0]) if r else pool[s] for s, r in zip(slots, reset)])
        p = pool.to(DEV)
        flag = torch.zeros(4, dtype=torch.int32, device=DEV)
        o = gdn.gdn_linear_prefill_slots(dev(c["q"]), dev(c["k"]), dev(c["v"]), dev(c["g"]), p, dev(slots),
                                         dev(reset), dev(c["cu"]), scale=c["scale"], error_flag=flag)
        c["s0"] = s0
        check_prefill(c, o, p[slots.long().to(DEV)])
        others = [1, 3, 5]
        assert torch.equal(p[others].cpu(), pool[others])
        before = p[slots.long().to(DEV)].cpu()
        o = gdn.gdn_linear_decode_step_slots(dev(step["q"]), dev(step["k"]), dev(step["v"]), dev(c["g"]), p,
                                             dev(slots), dev(reset), scale=c["scale"], error_flag=flag)
        assert int(flag[0]) == 0
        step["s0"] = torch.where(reset.bool()[:, None, None, None], 0.0, before)
        step["g"] = c["g"]
        check_step(step, o, p[slots.long().to(DEV)])
        assert torch.equal(p[others].cpu(), pool[others])


def check_step(c, o, sT):
    D = c["q"].shape[2]
    f = lambda x: oracle.linear_recurrent(x["q"], x["k"], x["v"], c["g"], x["s0"],
                                          inputs.cu_from_lengths([1] * len(x["q"])), scale=c["scale"])
    (o_ref, s_ref), (o_abs, s_abs) = f(c), f(absd(c))
    close(o, o_ref, o_abs, (D + 8) * 2.0 ** -24, c["dt"], "o")
    close(sT, s_ref, s_abs, 4 * 2.0 ** -24, F32, "state")


@pytest.mark.parametrize("shape", [(1, 1, 16, 1, F32), (2, 4, 32, 7, BF), (1, 3, 64, 100, F32),
                                   (2, 6, 128, 128, BF), (2, 2, 128, 128, F32), (1, 1, 128, 130, BF)], ids=str)
@pytest.mark.parametrize("N", [1, 2, 67])
def test_decode_step(shape, N):
    c = make([1] * N, *shape, seed=300 + N)
    st = Guarded(tuple(c["s0"].shape), F32, DEV, fill=c["s0"].to(DEV))
    o = Guarded(tuple(c["v"].shape), c["dt"], DEV)
    gdn.gdn_linear_decode_step(dev(c["q"]), dev(c["k"]), dev(c["v"]), dev(c["g"]), st.t, scale=c["scale"],
                               o=o.t)
    torch.cuda.synchronize()
    st.check("state")
    o.check("o")
    check_step(c, o.t, st.t)


def at_16(t):
    """A copy of t at an address that is a multiple of 16 but not of 32."""
    if t is None:
        return None
    n = t.numel() * t.element_size()
    buf = torch.empty(n + 64, dtype=torch.uint8, device=DEV)
    off = 16 if buf.data_ptr() % 32 == 0 else 0
    view = buf[off:off + n].view(t.dtype).view(t.shape)
    assert view.data_ptr() % 32 == 16
    return view.copy_(t)


def test_arrays_aligned_to_16_bytes_only():
    for shape in [(1, 2, 64, 64, F32), (2, 6, 128, 128, BF)]:
        c = make([300, 5, 129], *shape, seed=71)
        want, wantg = run_prefill(c), run_backward(c)
        a = [at_16(c[x].to(DEV)) for x in ("q", "k", "v", "g", "s0")]
        cu, do, dsT = at_16(c["cu"].to(DEV)), at_16(c["do"].to(DEV)), at_16(c["dsT"].to(DEV))
        N, T = len(c["lens"]), sum(c["lens"])
        size = (N, T, *shape[:4])
        f, b = gdn.gdn_linear_prefill_workspace_bytes, gdn.gdn_linear_prefill_backward_workspace_bytes
        ws = [at_16(torch.zeros(max(x(*size, dtype=shape[4]), 16), dtype=torch.uint8, device=DEV)) for x in (f, b)]
        o, sT = at_16(want[0]), at_16(want[1])
        gdn.gdn_linear_prefill(*a, cu, scale=c["scale"], o=o.zero_(), final_state=sT.zero_(), workspace=ws[0])
        assert torch.equal(o, want[0]) and torch.equal(sT, want[1])
        outs = [at_16(x).zero_() for x in wantg]
        gdn.gdn_linear_prefill_backward(do, *a, cu, dfinal_state=dsT, scale=c["scale"], dq=outs[0], dk=outs[1],
                                        dv=outs[2], dinitial_state=outs[3], workspace=ws[1])
        assert all(torch.equal(x, y) for x, y in zip(outs, wantg))
        st = at_16(c["s0"].to(DEV))
        o = gdn.gdn_linear_decode_step(*[at_16(x[:3]) for x in a[:3]], a[3], st, scale=c["scale"])
        st2 = dev(c["s0"])
        assert torch.equal(o, gdn.gdn_linear_decode_step(*[x[:3].contiguous() for x in a[:3]], a[3], st2,
                                                         scale=c["scale"]))
        assert torch.equal(st, st2)


def test_a_new_request_does_not_read_its_slot():
    """reset: whatever the slot held, NaN included, the result is that of zeros."""
    for shape in [(1, 2, 64, 64, F32), (1, 2, 128, 128, BF)]:
        c = make([40, 130], *shape, seed=73)
        pool = torch.full((3, *c["s0"].shape[1:]), float("nan"), device=DEV)
        slots, reset = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([2, 0], [1, 1]))
        a = [dev(c[x]) for x in ("q", "k", "v", "g")]
        o = gdn.gdn_linear_prefill_slots(*a, pool, slots, reset, dev(c["cu"]), scale=c["scale"])
        c["s0"] = None
        check_prefill(c, o, pool[[2, 0]])
        pool.fill_(float("nan"))
        o = gdn.gdn_linear_decode_step_slots(*[x[:2].contiguous() for x in a[:3]], a[3], pool, slots, reset)
        assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(pool[[2, 0]]).all())


def test_extreme_decays_and_scales():
    """Decays of fp32's whole finite range and a zero scale give finite results
    equal to the oracle's."""
    for shape in [(1, 4, 64, 64, F32), (1, 4, 128, 128, BF)]:
        c = make([260, 33], *shape, seed=79)
        c["g"] = torch.tensor([-3.4e38, -90.0, -1e-30, 0.0])
        check_prefill(c, *run_prefill(c))
        check_backward(c, run_backward(c))
        c["scale"] = 0.0
        o, _ = run_prefill(c)
        assert not bool(o.any())
        assert not bool(run_backward(c)[0].any())


def test_more_than_2_to_31_elements():
    """v of 400,000 tokens and 48 heads has more than 2^31 elements: the last
    tokens' results are those of a run over the last 2,048, before which the
    decay (at most e^-0.5 a token) leaves nothing in fp32."""
    T, Hqk, Hv, D, tail = 400_000, 1, 48, 128, 2048
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    gen = torch.Generator(device=DEV).manual_seed(83)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV, dtype=BF)
    q, k, v, do = r(T, Hqk, D), r(T, Hqk, D), r(T, Hv, D), r(T, Hv, D)
    assert v.numel() > 1 << 31
    g = torch.full((Hv,), -0.5, device=DEV)
    o, sT = gdn.gdn_linear_prefill(q, k, v, g, scale=D ** -0.5)
    # chunks of 128 tokens from the sequence's start: the tail starts on one
    t0 = (T - tail) // 128 * 128
    o2, s2 = gdn.gdn_linear_prefill(q[t0:], k[t0:], v[t0:], g, scale=D ** -0.5)
    half = t0 + 1024
    assert torch.equal(o[half:], o2[1024:])
    assert float((sT - s2).abs().max()) <= 2.0 ** -20 * float(s2.abs().max())
    del o, o2
    dq, dk, dv, _ = gdn.gdn_linear_prefill_backward(do, q, k, v, g, scale=D ** -0.5)
    gq, gk, gv, _ = gdn.gdn_linear_prefill_backward(do[t0:], q[t0:], k[t0:], v[t0:], g, scale=D ** -0.5)
    for x, y in ((dq, gq), (dk, gk), (dv, gv)):
        assert torch.equal(x[half:], y[1024:])


def test_bad_slots_are_reported_and_write_nothing():
    for shape in [(1, 2, 64, 64, F32), (1, 2, 128, 128, BF)]:
        Hqk, Hv, Dk, Dv, dt = shape
        c = make([30, 140], *shape, seed=43)
        pool = torch.randn(3, Hv, Dv, Dk)
        for bad in (-1, 3):
            slots = torch.tensor([bad, 1], dtype=torch.int32)
            p, flag = pool.to(DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
            gdn.gdn_linear_prefill_slots(dev(c["q"]), dev(c["k"]), dev(c["v"]), dev(c["g"]), p, dev(slots),
                                         None, dev(c["cu"]), scale=c["scale"], error_flag=flag)
            assert int(flag[0]) == 6 and torch.equal(p[[0, 2]].cpu(), pool[[0, 2]])
            p, flag = pool.to(DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
            o = torch.full((2, Hv, Dv), 7.0, dtype=dt, device=DEV)
            gdn.gdn_linear_decode_step_slots(dev(c["q"][:2]), dev(c["k"][:2]), dev(c["v"][:2]), dev(c["g"]),
                                             p, dev(slots), scale=c["scale"], o=o, error_flag=flag)
            assert int(flag[0]) == 6 and torch.equal(p[[0, 2]].cpu(), pool[[0, 2]])
            assert bool((o[0] == 7).all()) and not bool((o[1] == 7).all())


@pytest.mark.parametrize("cu", [[0, 90, 60, 100], [0, 30, 120, 100], [5, 30, 60, 100], [0, 30, 60, 90],
                                [0, -5, 60, 100]], ids=str)
def test_bad_cu_seqlens_is_reported_and_stays_inside(cu):
    for shape in [(1, 2, 64, 64, F32), (1, 2, 128, 128, BF)]:
        c = make([30, 30, 40], *shape, seed=47)
        o, sT = (Guarded(tuple(c["v"].shape), c["dt"], DEV), Guarded(tuple(c["s0"].shape), F32, DEV))
        flag = torch.zeros(4, dtype=torch.int32, device=DEV)
        bad = torch.tensor(cu, dtype=torch.int32, device=DEV)
        gdn.gdn_linear_prefill(dev(c["q"]), dev(c["k"]), dev(c["v"]), dev(c["g"]), dev(c["s0"]), bad,
                               o=o.t, final_state=sT.t, error_flag=flag)
        torch.cuda.synchronize()
        o.check()
        sT.check()
        assert int(flag[0]) == 5
        flag.zero_()
        outs = [Guarded(tuple(c[x].shape), c["dt"], DEV) for x in "qkv"]
        gdn.gdn_linear_prefill_backward(dev(c["do"]), dev(c["q"]), dev(c["k"]), dev(c["v"]), dev(c["g"]),
                                        dev(c["s0"]), bad, dfinal_state=dev(c["dsT"]), dq=outs[0].t,
                                        dk=outs[1].t, dv=outs[2].t, error_flag=flag)
        torch.cuda.synchronize()
        for x in outs:
            x.check()
        assert int(flag[0]) == 5


def test_repeatable_on_another_stream_and_in_a_graph():
    """Two runs give the same bits; so do a side stream and a replayed graph of
    prefill, backward and decode with new inputs copied into its buffers."""
    for shape in [(1, 2, 64, 64, F32), (2, 6, 128, 128, BF)]:
        c = make([300, 5, 129], *shape, seed=53)
        first, grads = run_prefill(c), run_backward(c)
        assert all(torch.equal(x, y) for x, y in zip(first, run_prefill(c)))
        assert all(torch.equal(x, y) for x, y in zip(grads, run_backward(c)))
        side = torch.cuda.Stream(DEV)
        a = [dev(c[x]) for x in ("q", "k", "v", "g", "s0", "cu", "do", "dsT")]
        torch.cuda.synchronize()
        o, sT = gdn.gdn_linear_prefill(*a[:6], scale=c["scale"], stream=side)
        side.synchronize()
        assert torch.equal(o, first[0]) and torch.equal(sT, first[1])
        graph = torch.cuda.CUDAGraph()
        st = a[4].clone()
        with torch.cuda.graph(graph):
            o, sT = gdn.gdn_linear_prefill(*a[:6], scale=c["scale"])
            got = gdn.gdn_linear_prefill_backward(a[6], *a[:6], dfinal_state=a[7], scale=c["scale"],
                                                  output_dinitial_state=True)
            od = gdn.gdn_linear_decode_step(a[0][:3], a[1][:3], a[2][:3], a[3], st, scale=c["scale"])
        for seed in (53, 54):
            n = make([300, 5, 129], *shape, seed=seed)
            for x, name in zip(a, ("q", "k", "v", "g", "s0", "cu", "do", "dsT")):
                x.copy_(n[name])
            st.copy_(n["s0"])
            graph.replay()
            torch.cuda.synchronize()
            want, wantg = run_prefill(n), run_backward(n)
            assert torch.equal(o, want[0]) and torch.equal(sT, want[1])
            assert all(torch.equal(x, y) for x, y in zip(got, wantg))
            st2 = dev(n["s0"])
            assert torch.equal(od, gdn.gdn_linear_decode_step(dev(n["q"][:3]), dev(n["k"][:3]), dev(n["v"][:3]),
                                                              dev(n["g"]), st2, scale=c["scale"]))
            assert torch.equal(st, st2)


def test_calls_in_a_row_share_a_workspace():
    """A call's kernels may start before the ones ahead of them end; the next call's
    must not touch a workspace, or inputs, that this one still reads."""
    for shape, lens in [((1, 2, 128, 128, BF), [4096]), ((2, 6, 128, 128, BF), [700, 5, 900]),
                        ((1, 2, 64, 64, F32), [1500, 40])]:
        cs = [make(lens, *shape, seed=s) for s in (81, 82)]
        want = [(run_prefill(c), run_backward(c)) for c in cs]
        size = (len(lens), sum(lens), *shape[:4])
        need = max(f(*size, dtype=shape[4]) for f in (gdn.gdn_linear_prefill_workspace_bytes,
                                                      gdn.gdn_linear_prefill_backward_workspace_bytes))
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
        a = [[dev(c[x]) for x in ("q", "k", "v", "g", "s0", "cu", "do", "dsT")] for c in cs]
        live = [torch.empty_like(x) for x in a[0]]
        got = []
        torch.cuda.synchronize()
        for _ in range(3):
            for b in a:
                for x, y in zip(live, b):
                    x.copy_(y)
                f = gdn.gdn_linear_prefill(*live[:6], scale=cs[0]["scale"], workspace=ws)
                g = gdn.gdn_linear_prefill_backward(live[6], *live[:6], dfinal_state=live[7], scale=cs[0]["scale"],
                                                    output_dinitial_state=True, workspace=ws)
                got.append((f, g))
        torch.cuda.synchronize()
        for i, (f, g) in enumerate(got):
            assert all(torch.equal(x, y) for x, y in zip(f, want[i % 2][0]))
            assert all(torch.equal(x, y) for x, y in zip(g, want[i % 2][1]))


def test_layer_run_norm_prefill_decode_and_gradients():
    """As a layer uses them: norm and rotation of a projection's queries and
    keys, linear prefill into states, decode steps, and the gradients of both."""
    T, Hqk, Hv, D = 200, 2, 6, 128
    gen = torch.Generator().manual_seed(61)
    r = lambda *s: torch.randn(*s, generator=gen)
    qkv = r(T + 2, (2 * Hqk + Hv) * D).to(BF)
    w = 1 + 0.2 * r(2, D)
    f = (1e4 ** (-torch.arange(0, 64, 2).double() / 64)).float()
    pos = torch.arange(1000, 1000 + T + 2, dtype=torch.int32)
    g, scale = decays(Hv, "slopes"), D ** -0.5
    x = qkv.to(DEV)
    xq, xk = (x[:, i * Hqk * D:(i + 1) * Hqk * D].unflatten(1, (Hqk, D)) for i in (0, 1))
    v = x[:, 2 * Hqk * D:].unflatten(1, (Hv, D)).contiguous()
    rope = dict(wq=dev(w[0]), wk=dev(w[1]))
    q, k = gdn.gdn_qk_norm_rope(xq, xk, dev(pos), dev(f), **rope)
    o, st = gdn.gdn_linear_prefill(q[:T], k[:T], v[:T], dev(g), scale=scale)
    steps = [gdn.gdn_linear_decode_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], dev(g), st, scale=scale)
             for t in (T, T + 1)]
    got = torch.cat([o] + steps)
    c = dict(q=q.cpu(), k=k.cpu(), v=v.cpu(), g=g, s0=None, dsT=None, cu=None, lens=[T + 2], dt=BF,
             scale=scale, do=r(T + 2, Hv, D).to(BF))
    check_prefill(c, got, st)
    do = dev(c["do"])
    dq, dk, dv, _ = gdn.gdn_linear_prefill_backward(do, q, k, v, dev(g), scale=scale)
    dx = torch.zeros_like(x)
    dxq, dxk = (dx[:, i * Hqk * D:(i + 1) * Hqk * D].unflatten(1, (Hqk, D)) for i in (0, 1))
    _, _, dwq, dwk = gdn.gdn_qk_norm_rope_backward(dq, dk, xq, xk, dev(pos), dev(f), dxq=dxq, dxk=dxk, **rope)
    check_backward(c, [dq, dk, dv])
    for dz, xx, ww, dxx, dww in ((dq, xq, w[0], dxq, dwq), (dk, xk, w[1], dxk, dwk)):
        ref, dref = oracle.qk_norm_rope_backward(dz.cpu(), xx.cpu(), ww, 1e-6, pos, f)
        scale_ = np.abs(ref).max()
        assert np.abs(dxx.cpu().double().numpy() - ref).max() <= 2.0 ** -8 * scale_ + 1e-5 * scale_
        assert np.abs(dww.cpu().double().numpy() - dref).max() <= 1e-5 * np.abs(dref).max()
    assert not bool(dx[:, 2 * Hqk * D:].any())
