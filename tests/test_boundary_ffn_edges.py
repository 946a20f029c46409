"""What the feed-forward calls accept at the edges of their documentation, and what they say of their
workspaces, without a GPU: through the C ABI on invented addresses and through the binding."""
import pytest

from bitwise_reproducible_int8_gb300 import build_lib, repro


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return repro.lib()


def test_selftest_holds_a_pair_s_whole_tile(L):
    """The exactness check runs a product of 256 x 256 over three slices of 512 terms: two outputs (the exact
    one and a path's), both operands' codes and their copies in 16 bits."""
    assert L.repro_selftest_ws_bytes() >= 2 * 256 * 256 * 4 + 2 * 256 * 1025 * (1 + 2)
