"""What the feed-forward calls accept at the edges of their documentation, and what they say of their
workspaces, without a GPU: through the C ABI on invented addresses and through the binding."""
import pytest
import torch

from bitwise_reproducible_int8_gb300 import build_lib, repro
from test_boundary_blocks import B, BAD, INF, NAN, call
from test_boundary_ffn import NORM


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


@pytest.mark.parametrize("alpha,beta", [(NAN, 1.0), (1.0, -INF), (INF, NAN)])
def test_a_norm_alone_takes_any_residual_scales(L, alpha, beta):
    """Without a block's output alpha and beta are not looked at; with one they are finite."""
    scales = dict(alpha=alpha, beta=beta)
    assert call(L.repro_block_norm_fwd, NORM, **scales) == -1
    assert call(L.repro_block_norm_fwd, NORM, y=None, h=None, **scales) not in BAD
    ok = dict(dh=B, dh_ld=64, du=2 * B, u_type=0, du_ld=64, h=3 * B, h_ld=64, y=None, y_ld=0, type=0, gate=None, gate_ld=0,
              gain_post=None, gain_pre=None, stats=6 * B, alpha=1.0, beta=1.0, n=10, D=64, flags=0, dx=7 * B, dx_ld=64, dy=None,
              dy_ld=0, dgate=None, dgate_ld=0, dgain_post=None, dgain_pre=None, ws=None, ws_bytes=0, stream=None)
    assert call(L.repro_block_norm_bwd, ok, **scales) not in BAD
    assert call(L.repro_block_norm_bwd, ok, y=4 * B, y_ld=64, dy=8 * B, dy_ld=64, **scales) == -1
