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
