"""Host-only checks: sizes past what the linear attention and norm-with-rotation
kernels can index are refused as unsupported before anything is launched,
the largest 32- and 64-bit values among them."""
import pytest

import gated_deltanet_04_b200 as gdn
from gated_deltanet_04_b200 import build as gdn_build

P = 0x10000  # a fake device address
UNSUPPORTED = 2
I31 = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib():
    gdn_build.build()
    return gdn.library()


def decode(lib, N, Hv, Dk, Dv):
    return lib.gdn_linear_decode_step(P, P + 16, P + 32, 1, P + 48, 1.0, P + 64, N, 1, Hv, Dk, Dv, P + 80, None, None)


@pytest.mark.parametrize("N,Hv,Dk,Dv", [(1 << 25, 48, 128, 1024), (1 << 24, 127, 128, 129), (1, 1, 16, I31),
                                        (1, 1, 128, I31), (I31, I31, 64, 1)])
def test_decode_grids(lib, N, Hv, Dk, Dv):
    assert decode(lib, N, Hv, Dk, Dv) == UNSUPPORTED


def prefill(lib, N, T, Hv, D):
    return lib.gdn_linear_prefill(P, P + 16, P + 32, 1, P + 48, 1.0, None, P + 64, N, T, 1, Hv, D, D, P + 80, None,
                                  P + 96, 1 << 60, None, None)


def backward(lib, N, T, Hv, D):
    return lib.gdn_linear_prefill_backward(P, P + 16, P + 32, P + 48, 1, P + 64, 1.0, None, None, P + 80, N, T, 1,
                                           Hv, D, D, P + 96, P + 112, P + 128, None, P + 144, 1 << 60, None, None)


@pytest.mark.parametrize("N,T,Hv,D", [
    (I31, 64, I31, 64), (I31, I31, I31, 128),       # the product of all sizes passes 64 bits
    ((1 << 24) - 1, 64, 32, 128),                   # one grid slot past the limit
    (1, 1 << 31, 1, 64), (1, 1 << 62, 1, 64)])
def test_prefill_and_backward_grids(lib, N, T, Hv, D):
    assert prefill(lib, N, T, Hv, D) == UNSUPPORTED
    assert backward(lib, N, T, Hv, D) == UNSUPPORTED
    for dt in (0, 1):
        assert lib.gdn_linear_prefill_workspace_bytes(N, T, 1, Hv, D, D, dt) == 0
        assert lib.gdn_linear_prefill_backward_workspace_bytes(N, T, 1, Hv, D, D, dt) == 0


@pytest.mark.parametrize("T,Hq,Hk", [(1 << 62, 24, 4), (1 << 61, 4, 4), ((1 << 33) // 7 + 1, 6, 1),
                                     ((1 << 63) - 1, 32767, 1)])
def test_rotation_rows(lib, T, Hq, Hk):
    D = 64
    head = (P, P + 16, 1, Hq * D, Hk * D, None, None, 1e-6, P + 32, 1, None, P + 48, 32, 0, T, Hq, Hk, D)
    assert lib.gdn_qk_norm_rope(*head, P + 64, P + 80, None) == UNSUPPORTED
    assert lib.gdn_qk_norm_rope_backward(P + 96, P + 112, *head, P + 64, P + 80, Hq * D, Hk * D, None, None, None, 0,
                                         None) == UNSUPPORTED


@pytest.mark.parametrize("stride", [1 << 30, 1 << 62, (1 << 63) - 4])
def test_rotation_strides(lib, stride):
    head = lambda sq: (P, None, 1, sq, 0, None, None, 1e-6, None, 0, None, None, 0, 0, 4, 2, 0, 64)
    assert lib.gdn_qk_norm_rope(*head(stride), P + 64, None, None) == UNSUPPORTED
    assert lib.gdn_qk_norm_rope_backward(P + 96, None, *head(128), P + 64, None, stride, 0, None, None, None, 0,
                                         None) == UNSUPPORTED
