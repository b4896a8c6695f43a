"""Tensor-core linear attention against the fp64 oracle chunk by chunk, by the
bounds of linear_checks.py: a chunk that is lost, reads a stale state or loses a
part of its values is seen, which bounds that grow with the sequence would let pass."""
import pytest
import torch

import gated_deltanet_04_b200 as gdn
import oracle
from gated_deltanet_04_b200 import inputs
from tests.linear_checks import CHUNK, OUT_BOUND, state_bound, worst_chunk, worst_state

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
D = 128


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gated_deltanet_04_b200 import build
    build.build()


# (lengths, Hqk, Hv): one chunk, whole ones, ragged ones, a chain of 24 chunks in segments,
# several sequences in segments, and 40 heads of which the tensor cores take one segment each
CASES = [([100], 1, 2), ([256], 2, 2), ([300, 16, 0, 129 + 64], 2, 6), ([3000], 1, 2), ([2300, 17, 900], 1, 5),
         ([700, 660], 8, 40)]


@pytest.mark.parametrize("decay", [0.0, -1e-4, -0.02, -0.5])
@pytest.mark.parametrize("lens,Hqk,Hv", CASES, ids=lambda x: str(x).replace(" ", ""))
def test_every_chunk(lens, Hqk, Hv, decay):
    gen = torch.Generator().manual_seed(sum(lens) + Hv)
    r = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16)
    T, N = sum(lens), len(lens)
    q, k, v, do = r(T, Hqk, D), r(T, Hqk, D), r(T, Hv, D), r(T, Hv, D)
    g = decay * (1 + torch.arange(Hv) / Hv)
    cu, scale = inputs.cu_from_lengths(lens).to(torch.int32), D ** -0.5
    dev = [x.to(DEV) for x in (q, k, v, g)]
    # without states: what every chunk passes on is all there is
    o, sT = gdn.gdn_linear_prefill(*dev, None, cu.to(DEV), scale=scale)
    dq, dk, dv, ds0 = gdn.gdn_linear_prefill_backward(do.to(DEV), *dev, None, cu.to(DEV), scale=scale,
                                                      output_dinitial_state=True)
    o_ref, s_ref = oracle.linear_recurrent(q, k, v, g, None, cu, scale=scale)
    refs = oracle.linear_backward(do, q, k, v, g, None, cu, scale=scale)
    f = lambda x: x.detach().cpu().double().numpy()
    for name, x, ref in (("o", o, o_ref), ("dq", dq, refs[0]), ("dk", dk, refs[1]), ("dv", dv, refs[2])):
        worst = worst_chunk(f(x), ref, lens)
        assert worst <= OUT_BOUND, f"{name}: {worst:.3g}, allowed {OUT_BOUND:.3g}"
    some = [n for n in range(N) if lens[n]]
    allowed = state_bound(-(-max(lens) // CHUNK))
    for name, x, ref in (("final_state", sT, s_ref), ("dinitial_state", ds0, refs[3])):
        worst = worst_state(f(x)[some], ref[some])
        assert worst <= allowed, f"{name}: {worst:.3g}, allowed {allowed:.3g}"
        assert not x[[n for n in range(N) if not lens[n]]].any()
