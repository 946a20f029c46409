"""GPU: the product of codes for up to 16 tokens whose rows lie on any byte, against exact integers:
every length up to several groups of codes, every place of either row within a word."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import bitwise_reproducible_int8_gb300 as R  # noqa: E402
import test_gpu_ffn as T  # noqa: E402
from gpu_helpers import dev, host  # noqa: E402
from test_gpu_blocks import same, strided  # noqa: E402

pytestmark = pytest.mark.gpu


def check(M, N, K, pa, oa, pb, ob, accumulate=False, kind=T.F32):
    a, b, sa, sb = T.mm_case(M, N, K)
    old = np.linspace(-1, 1, M * N, dtype=np.float32).reshape(M, N)
    y = dev(old).to(kind)
    R.repro_matmul_i8(strided(a, pa, oa, torch.int8), strided(b, pb, ob, torch.int8), y, dev(sa), dev(sb), accumulate=accumulate)
    e = (a.astype(np.int64) @ b.astype(np.int64).T).astype(np.float32) * sa[:, None] * sb
    e = old + e if accumulate else e
    same(host(y.float()), T.bf(e) if kind is T.BF else e)


@pytest.mark.parametrize("K", list(range(1, 34)) + [127, 128, 129, 515, 516, 517, 520, 523, 1036])
@pytest.mark.parametrize("M", [1, 3, 8, 11, 16])
def test_lengths(K, M):
    check(M, 9, K, 0, 0, 0, 0)
    check(M, 9, K, 5, 1, 3, 2)


@pytest.mark.parametrize("oa", range(4))
@pytest.mark.parametrize("ob", range(4))
@pytest.mark.parametrize("pa,pb", [(0, 0), (1, 0), (2, 3), (16, 1)])
@pytest.mark.parametrize("K", [12, 528, 1101])
def test_places(oa, ob, pa, pb, K):
    check(1, 5, K, pa, oa, pb, ob)
    check(10, 7, K, pa, oa, pb, ob, accumulate=True)
    check(4, 6, K, pa, oa, pb, ob, kind=T.BF)


@pytest.mark.parametrize("M,N,K", [(16, 700, 133143), (2, 4099, 2049), (16, 1001, 5633), (7, 1, 133142)])
def test_long(M, N, K):
    check(M, N, K, 0, 0, 0, 0)
    check(M, N, K, 1, 3, 2, 1)
