"""How far a value that is not finite spreads in linear attention: forward in time and
down its own sums everywhere; on tensor cores also to the other tokens of its 128-token
chunk where the formula masks it; never to other heads' sums, earlier (in the gradients
that run backwards, later) chunks, or other sequences."""
import pytest
import torch

import gated_deltanet_04_b200 as gdn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")
T, AT = 500, 200  # the odd token out, in the second chunk of 128


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gated_deltanet_04_b200 import build
    build.build()


def make(dt, D):
    gen = torch.Generator(device=DEV).manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(dt)
    return dict(q=r(T, 2, D), k=r(T, 2, D), v=r(T, 4, D), do=r(T, 4, D)), torch.tensor([-0.01, -0.1, 0.0, -1.0],
                                                                                       device=DEV)


def run(x, g):
    o, S = gdn.gdn_linear_prefill(x["q"], x["k"], x["v"], g, scale=0.1)
    dq, dk, dv, ds = gdn.gdn_linear_prefill_backward(x["do"], x["q"], x["k"], x["v"], g, scale=0.1,
                                                     output_dinitial_state=True)
    return dict(o=o, S=S[0], dq=dq, dk=dk, dv=dv, ds=ds[0])


def same(a, b, where):
    return torch.equal(a[where], b[where])


@pytest.mark.parametrize("bad", [NAN, INF, -INF], ids=str)
@pytest.mark.parametrize("dt,D", [(F32, 64), (BF, 64), (BF, 128)], ids=str)
def test_a_value_or_its_gradient(dt, D, bad):
    """v or do of one token, head 1 (q/k head 0) and column 5."""
    chunks = dt == BF and D == 128
    first, last = (128, 255) if chunks else (AT, AT)  # tokens that may be touched, from and to
    x, g = make(dt, D)
    want = run(x, g)
    for name in ("v", "do"):
        y = dict(x)
        y[name] = x[name].clone()
        y[name][AT, 1, 5] = bad
        got = run(y, g)
        cols = [c for c in range(D) if c != 5]
        others = [0, 2, 3]
        for z in ("o", "dv"):
            assert same(got[z], want[z], (slice(None), others)), z
            assert same(got[z], want[z], (slice(None), 1, cols)), z
        for z in ("dq", "dk"):
            assert same(got[z], want[z], (slice(None), 1)), z
        assert same(got["S"], want["S"], others) and same(got["ds"], want["ds"], others)
        assert same(got["S"][1], want["S"][1], cols) and same(got["ds"][1], want["ds"][1], cols)
        if name == "v":  # S and o forward in time; dq forward (through S), dk at the token itself
            assert same(got["o"], want["o"], slice(0, first)) and same(got["dq"], want["dq"], slice(0, first))
            assert same(got["dk"], want["dk"], slice(0, AT)) and same(got["dk"], want["dk"], slice(AT + 1, T))
            assert torch.equal(got["dv"], want["dv"]) and torch.equal(got["ds"], want["ds"])
            assert not torch.isfinite(got["o"][AT:, 1, 5]).any() and not torch.isfinite(got["S"][1, 5]).any()
        else:  # G backward in time: dk, dv and the entering state's; dq at the token itself
            assert torch.equal(got["o"], want["o"]) and torch.equal(got["S"], want["S"])
            assert same(got["dq"], want["dq"], slice(0, AT)) and same(got["dq"], want["dq"], slice(AT + 1, T))
            assert same(got["dk"], want["dk"], slice(last + 1, T))
            assert same(got["dv"], want["dv"], slice(last + 1, T))
            assert not torch.isfinite(got["dv"][:AT + 1, 1, 5]).any() and not torch.isfinite(got["ds"][1, 5]).any()


@pytest.mark.parametrize("dt,D", [(F32, 64), (BF, 64), (BF, 128)], ids=str)
def test_a_query_or_key(dt, D):
    """q and k of one token and q/k head 0 (v-heads 0 and 1), all columns."""
    chunks = dt == BF and D == 128
    first, last = (128, 255) if chunks else (AT, AT)
    x, g = make(dt, D)
    want = run(x, g)
    y = dict(x, q=x["q"].clone())
    y["q"][AT, 0] = NAN
    got = run(y, g)
    rest = [t for t in range(T) if t != AT]
    assert same(got["o"], want["o"], rest) and same(got["o"], want["o"], (slice(None), [2, 3]))
    assert torch.equal(got["S"], want["S"]) and not torch.isfinite(got["o"][AT, :2]).any()
    assert same(got["dk"], want["dk"], slice(last + 1, T)) and same(got["dk"], want["dk"], (slice(None), 1))
    assert same(got["dv"], want["dv"], slice(AT + 1, T)) and torch.equal(got["dq"], want["dq"])
    y = dict(x, k=x["k"].clone())
    y["k"][AT, 0] = NAN
    got = run(y, g)
    assert same(got["o"], want["o"], slice(0, AT)) and same(got["o"], want["o"], (slice(None), [2, 3]))
    assert same(got["S"], want["S"], [2, 3]) and not torch.isfinite(got["o"][AT:, :2]).any()
    assert same(got["dq"], want["dq"], slice(0, first)) and same(got["dq"], want["dq"], (slice(None), 1))
    assert same(got["dv"], want["dv"], slice(0, AT)) and same(got["dv"], want["dv"], slice(AT + 1, T))
    assert torch.equal(got["dk"], want["dk"]) and torch.equal(got["ds"], want["ds"])
