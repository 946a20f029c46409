"""What the feed-forward calls accept at the edges of their documentation, and what they say of their
workspaces, without a GPU: through the C ABI on invented addresses and through the binding."""
import pytest
import torch

from bitwise_reproducible_int8_gb300 import build_lib, repro


class Device(torch.Tensor):                  # host memory that passes for a device's
    is_cuda = property(lambda self: True)


def d(*shape, dt=torch.float32):
    return torch.zeros(shape, dtype=dt).as_subclass(Device)


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return repro.lib()


def test_selftest_holds_a_pair_s_whole_tile(L):
    """The exactness check runs a product of 256 x 256 over three slices of 512 terms: two outputs (the exact
    one and a path's), both operands' codes and their copies in 16 bits."""
    assert L.repro_selftest_ws_bytes() >= 2 * 256 * 256 * 4 + 2 * 256 * 1025 * (1 + 2)


@pytest.mark.parametrize("M,N", [(0, 0), (0, 5), (3, 0), (200, 0)])
@pytest.mark.parametrize("K", [0, 7])
@pytest.mark.parametrize("ta,tb", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_products_without_outputs(L, M, N, K, ta, tb, accumulate):
    """No tokens or no channels: nothing to do, whichever side is empty."""
    a, b = d(*((K, M) if ta else (M, K)), dt=torch.int8), d(*((K, N) if tb else (N, K)), dt=torch.int8)
    repro.repro_matmul_i8(a, b, d(M, N), d(M), d(N), ta, tb, accumulate, stream=0)
    if M != N:
        with pytest.raises(ValueError):
            repro.repro_matmul_i8(a, b, d(N, M), d(M), d(N), ta, tb, accumulate, stream=0)
