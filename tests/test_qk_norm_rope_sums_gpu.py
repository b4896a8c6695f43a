"""The weights' gradients of gdn_qk_norm_rope_backward against float64, by a bound that
a single lost row of many thousands passes (linear_checks.py)."""
import numpy as np
import pytest
import torch

import gated_deltanet_04_b200 as gdn
import oracle
from tests.linear_checks import dw_bound

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gated_deltanet_04_b200 import build
    build.build()


# one CTA's rows; several blocks a CTA; several turns of the persistent grid, both types and
# every head size; one key head beside many query heads
@pytest.mark.parametrize("T,Hq,Hk,D,R,dt", [
    (5, 2, 1, 64, 32, F32), (700, 6, 2, 128, 128, BF), (3001, 24, 1, 64, 64, BF), (6001, 24, 4, 256, 64, BF),
    (4003, 13, 3, 256, 256, F32), (40001, 1, 1, 16, 16, F32), (9001, 5, 5, 32, 16, BF), (5003, 16, 16, 128, 64, F32)],
    ids=str)
def test_weight_gradients(T, Hq, Hk, D, R, dt):
    gen = torch.Generator().manual_seed(T + D)
    r = lambda *s: torch.randn(*s, generator=gen)
    xq, xk, dq, dk = (r(T, h, D).to(dt) for h in (Hq, Hk, Hq, Hk))
    w = 1 + 0.3 * r(2, D)
    pos = torch.randint(0, 1 << 18, (T,), generator=gen, dtype=torch.int32)
    f = (1e6 ** (-torch.arange(0, R, 2).double() / R)).float()
    d = lambda x: x.to(DEV).contiguous()
    _, _, dwq, dwk = gdn.gdn_qk_norm_rope_backward(d(dq), d(dk), d(xq), d(xk), d(pos), d(f), wq=d(w[0]), wk=d(w[1]))
    for x, dz, dw in ((xq, dq, dwq), (xk, dk, dwk)):
        n = oracle.qk_norm_rope(x, None, 1e-6, None, None)
        dy = oracle.qk_norm_rope(dz, None, 1e-6, pos, f, inverse=True, norm=False)
        off = np.abs(dw.cpu().double().numpy() - (dy * n).sum((0, 1))) / dw_bound(dy, n)
        assert off.max() <= 1, f"{off.max():.3g} times the bound"
