"""What the fp32 states of linear attention keep (gdn_linear_prefill and its
backward pass), against sums in float64.

Bounds are relative L2 errors per head, from the arithmetic with u = 2^-24 (half a
step of fp32, relative): roundings that are independent of one another add in
quadrature, each u / sqrt(3) on average; those that may all have one sign add as
they are.
* A state carried over n chunks (segments, tokens) is rounded twice at each, so
  it is off by sqrt(2 n / 3) u where its size stays about the same; twice that is
  allowed.
* A chunk's own sum of 128 products is at most 24 accumulations of 16 (three
  parts), each off by u in one direction, and its weights by 2 u: 26 u of it.
"""
import pytest
import torch

import gated_deltanet_04_b200 as gdn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gated_deltanet_04_b200 import build
    build.build()


def rel_per_head(x, ref):
    """Relative L2 error of each head of [H, Dv, Dk]."""
    err = (x.double() - ref).flatten(1).norm(dim=1)
    return err / ref.flatten(1).norm(dim=1)


def state_after(x, y, g, s0, weight):
    """exp(g T) s0 + sum_t exp(g weight[t]) x_t y_t^T of one sequence in float64,
    [H, Dx, Dy]: x [T,H,Dx], y [T,Hy,Dy]."""
    T, H, _ = x.shape
    out = torch.empty(H, x.shape[2], y.shape[2], dtype=torch.float64, device=DEV)
    for h in range(H):
        w = torch.exp(g[h].double() * weight)[:, None]
        out[h] = torch.exp(g[h].double() * T) * s0[h].double() + (w * x[:, h].double()).T @ \
            y[:, h // (H // y.shape[1])].double()
    return out


# (lengths, Hqk, Hv, D, dtype, chunks or segments one after another): one chain of 513
# chunks (48 heads of 16 sequences, 15 of them empty, leave no reason for segments), 129
# segments of 4 chunks, and 1,024 segments of 64 tokens in the token recurrence
SLOW = [([0] * 15 + [65536], 1, 48, 128, BF, 513), ([65536], 1, 6, 128, BF, 133), ([65536], 1, 1, 16, F32, 1088)]


@pytest.mark.parametrize("lens,Hqk,Hv,D,dt,n", SLOW, ids=["chain", "segments", "tokens"])
def test_a_slow_decay_keeps_its_24_bits(lens, Hqk, Hv, D, dt, n):
    """Decays near -1e-6: the factor of a chunk is so near 1 that its rounding, the same
    every time, must not compound.  The entering state, 4 times the size of what
    comes in, is most of the result."""
    T, N = sum(lens), len(lens)
    gen = torch.Generator(device=DEV).manual_seed(91)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)
    q, k = r(T, Hqk, D).to(dt), r(T, Hqk, D).to(dt)
    v, do = (r(T, Hv, D) * 2.0 ** -10).to(dt), (r(T, Hv, D) * 2.0 ** -10).to(dt)
    s0, dsT = r(N, Hv, D, D), r(N, Hv, D, D)
    cu = torch.tensor([0] * N + [T], dtype=torch.int32, device=DEV)
    bound = (2 * (2 * n / 3) ** 0.5 + 26 * 0.3 + 2) * U
    t = torch.arange(T, dtype=torch.float64, device=DEV)
    for shift in range(1 if Hv > 1 else 6):
        g = -1e-6 * (1 + 0.37 * (shift + torch.arange(Hv, device=DEV, dtype=F32)))
        _, sT = gdn.gdn_linear_prefill(q, k, v, g, s0, cu)
        worst = rel_per_head(sT[-1], state_after(v, k, g, s0[-1], T - 1 - t)).max()
        assert worst <= bound, f"final state: {worst:.3g}, allowed {bound:.3g}"
        assert torch.equal(sT[:-1], s0[:-1])
        ds0 = gdn.gdn_linear_prefill_backward(do, q, k, v, g, s0, cu, dfinal_state=dsT,
                                              output_dinitial_state=True)[3]
        worst = rel_per_head(ds0[-1], state_after(do, q, g, dsT[-1], t + 1)).max()
        assert worst <= bound, f"dinitial_state: {worst:.3g}, allowed {bound:.3g}"
