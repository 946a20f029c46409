"""The oracle's distillation loss where a row's values are not ordinary: teacher
values that are no numbers beside empty entries, masks of the type's lowest value,
weights of zero, log-probabilities that are none."""
import numpy as np
import pytest

import ops64 as F
from test_oracle_blocks import case

LOWEST = np.finfo(np.float32).min
FULL = dict(tau=1.0, w_kd=1.0, w_ce=0.0, w_z=0.0, logprobs=False)


def both(orc, z, idx, tl, lab, **hp):
    """(loss, stats, gradient for an upstream gradient of 1)."""
    hp = {**FULL, **hp}
    loss, stats = orc.distill_fwd(z, idx, tl, lab, **hp)
    hp.pop("logprobs")
    return loss, stats, orc.distill_bwd(z, idx, stats, np.ones(1, dtype=np.float32), lab, **hp)


def nonfinite_teachers():
    """Rows with a live teacher value that is no number beside empty entries and
    entries out of range; the last row is ordinary."""
    V, K = 300, 6
    z, idx, tl, lab = case(11, 6, V, K)
    idx[:] = np.arange(K) * 31 + 2
    idx[:, [1, 4]] = -1
    idx[2:4, 2] = V
    idx[3, 1] = 1 << 36
    for row, bad in enumerate((np.nan, np.inf, np.nan, np.inf, -np.inf)):
        tl[row, 0] = bad
    return z, idx, tl, lab


@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0])
@pytest.mark.parametrize("logprobs", [False, True])
def test_empty_entries_weigh_nothing(orc, tau, logprobs):
    """Whatever the others are, an empty entry's weight is +0 and its column is not read."""
    z, idx, tl, lab = nonfinite_teachers()
    if logprobs:
        tl = np.where(tl == np.inf, np.float32(np.nan), tl - 9).astype(np.float32)
    V = z.shape[1]
    loss, stats, dz = both(orc, z, idx, tl, lab, tau=tau, logprobs=logprobs)
    p, empty = stats[:, orc.DISTILL_STATS:], (idx < 0) | (idx >= V)
    assert np.all(p[empty].view(np.uint32) == 0)
    assert np.isnan(p[[0, 2], 0]).all() and np.isfinite(p[4:]).all()
    assert np.isfinite(loss[4:]).all() and not np.isfinite(loss[:4]).any()
    assert np.isfinite(dz[4:]).all() and not np.isfinite(dz[:4]).all(1).any()


MIXES = [dict(), dict(w_kd=0.7, w_ce=0.3), dict(w_kd=0.5, w_ce=0.5, w_z=1e-3)]


def masked_rows():
    """Rows masked by the lowest values of binary32 and bf16: a tail, a whole block and
    more, all but one logit.  Teacher and label keep to what is left."""
    V, K = 3000, 5
    z, idx, tl, lab = case(12, 6, V, K)
    idx[:] = np.arange(K)
    idx[::2, 3] = -1
    lab[:] = 2
    lab[4] = -1
    bf_lowest = np.float32(-(2.0 - 2.0 ** -7) * 2.0 ** 127)
    for row, low in enumerate((LOWEST, bf_lowest) * 3):
        z[row, (60, 1024, 5)[row // 2]:None if row < 4 else 2999] = low
    z[2:4, 2500:] = 1.0
    return z, idx, tl, lab


@pytest.mark.parametrize("tau", [1e-4, 0.5, 0.9, 1.0, 2.0])
@pytest.mark.parametrize("mix", MIXES)
def test_lowest_value_masks_like_minus_infinity(orc, tau, mix):
    """A product by 1 / tau that overflows makes no NaN: the same bits as with -infinity."""
    z, idx, tl, lab = masked_rows()
    if tau < 0.1:
        z, tl = np.where(z > -1e30, z * np.float32(1e-3), z), tl * np.float32(1e-3)
    got = both(orc, z, idx, tl, lab, tau=tau, **mix)
    exp = both(orc, np.where(z < -1e30, np.float32(-np.inf), z), idx, tl, lab, tau=tau, **mix)
    for a, b in zip(got, exp):
        assert np.isfinite(b).all()
        assert np.array_equal(a.view(np.uint32), b.view(np.uint32))


def overflowing_rows():
    """(rows, the same with 0 for each row's largest and -infinity for the rest): logits and
    teacher values whose products by 1 / tau overflow."""
    V, K = 2100, 4
    z, idx, tl, lab = case(13, 4, V, K)
    idx[:] = np.arange(K) * 500
    lab[:] = 1500
    z[0] = LOWEST                               # nothing but the mask
    z[1, :] = -3e38
    z[1, [500, 1500, 2099]] = 3e38
    tl[2] = LOWEST
    tl[3] = (3e38, LOWEST, 3e38, 0)
    plain_z, plain_t = z.copy(), tl.copy()
    plain_z[0] = 0
    plain_z[1] = np.where(z[1] > 0, 0, -np.inf)
    plain_t[2] = 0
    plain_t[3] = (0, -np.inf, 0, -np.inf)
    return (z, tl), (plain_z, plain_t), idx, lab


@pytest.mark.parametrize("tau", [0.01, 0.5, 0.9])
@pytest.mark.parametrize("mix", MIXES[:2])
def test_overflowing_products(orc, tau, mix):
    """Softmax and gradient depend on differences alone, whatever the products do."""
    (z, tl), (plain_z, plain_t), idx, lab = overflowing_rows()
    _, s, dz = both(orc, z, idx, tl, lab, tau=tau, **mix)
    _, es, ez = both(orc, plain_z, idx, plain_t, lab, tau=tau, **mix)
    assert np.array_equal(s[:, [1, 3]], es[:, [1, 3]])                       # the sums
    assert np.array_equal(s[:, orc.DISTILL_STATS:], es[:, orc.DISTILL_STATS:])
    assert np.isfinite(dz).all() and np.array_equal(dz, ez)
