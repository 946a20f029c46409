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


def far_rows():
    """(rows, the same moved to zero): logits and teacher values so far from zero that 64 bits
    cannot hold their sums with a logarithm.  Softmax depends on differences, so each pair has
    one loss; the differences here are exact."""
    V, K = 2100, 6
    z, idx, tl, lab = case(14, 7, V, K)
    idx[:] = np.arange(K) * 301
    idx[1::2, 2] = -1
    lab[:] = 2 * 301
    tl = np.round(tl * 4).astype(np.float32)
    plain_z, plain_t = z.copy(), tl.copy()
    z[0], plain_z[0] = LOWEST, 0                # a row that its mask leaves nothing of
    z[1], plain_z[1] = -(2.0 - 2.0 ** -7) * 2.0 ** 127, 0
    plain_z[2] = np.where(np.arange(V) % 301 == 0, 2.0 ** 20, 0) - 2.0 ** 20
    z[2] = plain_z[2] + 2.0 ** 40
    tl[3], plain_t[3] = LOWEST, 0               # a teacher that its mask leaves nothing of
    tl[4], plain_t[4] = 2.0 ** 100, 0
    z[4], plain_z[4] = 2.0 ** 100, 0
    z[5], plain_z[5] = LOWEST, 0
    tl[5], plain_t[5] = LOWEST, 0
    return (z, tl), (plain_z, plain_t), idx, lab


@pytest.mark.parametrize("tau", [0.01, 0.5, 0.9, 1.0, 1.5, 2.0, 4.0])
@pytest.mark.parametrize("mix", [dict(), dict(w_kd=0.0, w_ce=1.0), dict(w_kd=0.7, w_ce=0.3)])
def test_loss_of_rows_far_from_zero(orc, tau, mix):
    """A row masked by the lowest value throughout is uniform: its cross entropy is ln V."""
    (z, tl), (plain_z, plain_t), idx, lab = far_rows()
    loss, _, dz = both(orc, z, idx, tl, lab, tau=tau, **mix)
    el, bound, ez, zb = F.distill_rows(plain_z, idx, plain_t, lab, **{**FULL, "tau": tau, **mix})
    assert np.all(np.abs(loss - el) <= bound)
    assert np.all(np.abs(dz - ez) <= zb)


def test_loss_of_masked_row_with_logprobs(orc):
    (z, tl), (plain_z, plain_t), idx, lab = far_rows()
    lp = (plain_t - 12).astype(np.float32)
    loss = both(orc, z, idx, lp, lab, logprobs=True)[0]
    el, bound, _, _ = F.distill_rows(plain_z, idx, lp, lab, **{**FULL, "logprobs": True})
    assert np.all(np.abs(loss - el) <= bound)


def test_loss_of_infinite_columns(orc):
    """Teacher weight on a masked logit costs without end; a mask that is large and finite costs
    its weight."""
    z, idx, tl, lab = case(15, 4, 300, 3)
    idx[:] = (1, 2, 3)
    tl[:] = 0.0
    z[0, 2] = -np.inf
    z[1, 1:4] = -np.inf
    z[2, 2] = LOWEST
    z[3, 1:4] = LOWEST
    for tau in (0.5, 1.0, 2.0):
        loss = both(orc, z, idx, tl, lab, tau=tau)[0]
        assert np.all(loss[:2] == np.inf)
        exp = tau * np.float64(-LOWEST) * np.float64([1 / 3, 1])
        rows = 2 if tau < 1 else 1                          # (the other's loss is past binary32)
        assert np.all(np.abs(loss[2:2 + rows] / exp[:rows] - 1) < 4 * F.U)


@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0])
def test_teacher_without_weight_is_not_looked_at(orc, tau):
    """w_kd 0: whatever the teacher's values are, loss and gradient are those of an ordinary one."""
    z, idx, tl, lab = case(16, 4, 300, 5)
    idx[:, 0] = 7
    lab[:] = (3, -1, 7, 299)
    bad = tl.copy()
    bad[0, 0], bad[1, 0], bad[2, 0] = np.nan, np.inf, -np.inf
    for g in (1.0, -0.5):
        hp = dict(tau=tau, w_kd=0.0, w_ce=1.0)
        got, exp = (orc.distill_fwd(z, idx, t, lab, **hp) for t in (bad, tl))
        assert np.array_equal(got[0], exp[0]) and np.isfinite(got[0]).all()
        got, exp = (orc.distill_bwd(z, idx, s, np.float32([g]), lab, **hp) for s in (got[1], exp[1]))
        assert np.isfinite(got).all() and np.array_equal(got.view(np.uint32), exp.view(np.uint32))


def positive_logprobs():
    """Values that are no log-probabilities: one a row, beside ordinary ones."""
    big = [0.0, 1e-6, 0.02, 20.0, 88.0, 88.5, 89.5, 100.0, 1e4, 1e30, np.inf]
    z, idx, tl, lab = case(17, len(big), 300, 4)
    idx[:] = (5, 60, 7, 8)
    tl = (tl - 9).astype(np.float32)
    tl[:, 1] = big
    return z, idx, tl, lab


def test_logprobs_above_zero(orc):
    """Rounding may leave a log-probability above 0; from 88 on the weight is infinite instead of
    some number that binary32 exponents wrap around to."""
    z, idx, tl, lab = positive_logprobs()
    loss, stats, dz = both(orc, z, idx, tl, lab, logprobs=True)
    p = stats[:, orc.DISTILL_STATS + 1]
    exp = np.exp(tl[:5, 1].astype(np.float64))
    assert np.all(np.abs(p[:5] / exp - 1) <= (2 * tl[:5, 1] + 5) * F.U)   # t's two roundings, e's four
    assert np.all(p[5:] == np.inf) and np.all(stats[5:, 7] == np.inf)
    assert np.isfinite(loss[:4]).all() and not np.isfinite(loss[5:]).any()
    assert not np.isfinite(dz[5:]).all(1).any()
