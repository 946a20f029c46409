"""GPU: the distillation loss bit for bit against the oracle where a row's values are
not ordinary."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import bitwise_reproducible_int8_gb300 as R  # noqa: E402
from gpu_helpers import dev  # noqa: E402
from test_gpu_blocks import BF, bf, run_distill, same  # noqa: E402
from test_oracle_blocks import case  # noqa: E402
from test_oracle_distill_edges import (LOWEST, MIXES, both, far_rows, masked_rows, nonfinite_teachers,  # noqa: E402
                                       overflowing_rows, positive_logprobs)

pytestmark = pytest.mark.gpu


def check(orc, z, idx, tl, lab, status=0, copies=1, wide=True, **hp):
    """The device's loss, stats and gradient against the oracle's; `copies` of the rows, so
    that CTAs own their rows."""
    z, idx, tl, lab = (np.concatenate([a] * copies) for a in (z, idx, tl, lab))
    if not wide:
        z, tl = bf(z), bf(tl)
    el, es, ez = both(orc, z, idx, tl, lab, **hp)
    t = torch.float32 if wide else BF
    loss, stats, dz = run_distill(z, idx, tl, lab, np.ones(1, dtype=np.float32), hp, dev(z).to(t), t, np.int64)
    same(stats, es, "stats")
    same(loss, el, "loss")
    same(dz, ez if wide else bf(ez), "dz")
    assert R.repro_device_check() == status
    return loss, stats, dz


@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0])
@pytest.mark.parametrize("logprobs", [False, True])
@pytest.mark.parametrize("copies", [1, 900])
def test_empty_entries_weigh_nothing(orc, tau, logprobs, copies):
    z, idx, tl, lab = nonfinite_teachers()
    if logprobs:
        tl = np.where(tl == np.inf, np.float32(np.nan), tl - 9).astype(np.float32)
    _, stats, _ = check(orc, z, idx, tl, lab, R.REPRO_ERR_INDEX, copies, tau=tau, logprobs=logprobs)
    p = stats[:, R.REPRO_DISTILL_STATS:].reshape(copies, 6, 6)
    assert np.all(p[:, :, [1, 4]].view(np.uint32) == 0) and np.all(p[:, 2:4, 2].view(np.uint32) == 0)


@pytest.mark.parametrize("tau", [1e-4, 0.5, 0.9, 1.0, 2.0])
@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("copies,wide", [(1, True), (1, False), (300, True)])
def test_lowest_value_masks(orc, tau, mix, copies, wide):
    z, idx, tl, lab = masked_rows()
    if tau < 0.1:
        z, tl = np.where(z > -1e30, z * np.float32(1e-3), z), tl * np.float32(1e-3)
    loss, stats, dz = check(orc, z, idx, tl, lab, 0, copies, wide, tau=tau, **mix)
    assert np.isfinite(loss).all() and np.isfinite(dz).all() and np.all(dz[0, 60:] == 0)


@pytest.mark.parametrize("tau", [0.01, 0.5, 0.9])
@pytest.mark.parametrize("mix", MIXES[:2])
@pytest.mark.parametrize("copies,wide", [(1, True), (1, False), (400, True)])
def test_overflowing_products(orc, tau, mix, copies, wide):
    (z, tl), _, idx, lab = overflowing_rows()
    check(orc, z, idx, tl, lab, 0, copies, wide, tau=tau, **mix)


@pytest.mark.parametrize("tau", [0.01, 0.5, 0.9, 1.0, 1.5, 2.0, 4.0])
@pytest.mark.parametrize("mix", [dict(), dict(w_kd=0.0, w_ce=1.0), dict(w_kd=0.7, w_ce=0.3)])
@pytest.mark.parametrize("copies,wide", [(1, True), (1, False), (250, True)])
def test_loss_of_rows_far_from_zero(orc, tau, mix, copies, wide):
    (z, tl), _, idx, lab = far_rows()
    loss, _, dz = check(orc, z, idx, tl, lab, 0, copies, wide, tau=tau, **mix)
    if wide:                                   # (bf16 has -infinity for the lowest value)
        assert np.isfinite(loss).all() and np.isfinite(dz).all()


def test_loss_of_masked_row_with_logprobs(orc):
    (z, _), (_, tl), idx, lab = far_rows()
    check(orc, z, idx, (tl - 12).astype(np.float32), lab, logprobs=True)


@pytest.mark.parametrize("tau", [0.5, 1.0, 2.0])
def test_loss_of_infinite_columns(orc, tau):
    z, idx, tl, lab = case(15, 4, 300, 40)
    idx[:] = np.arange(40) + 1
    tl[:] = 0.0
    z[0, 2], z[1, 1:41], z[2, 2], z[3, 1:41] = -np.inf, -np.inf, LOWEST, LOWEST
    loss, _, _ = check(orc, z, idx, tl, lab, tau=tau)
    assert np.all(loss[:2] == np.inf)


@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0])
@pytest.mark.parametrize("K", [5, 80])
@pytest.mark.parametrize("wide", [True, False])
def test_teacher_without_weight_is_not_looked_at(orc, tau, K, wide):
    z, idx, tl, lab = case(16, 4, 300, K)
    idx[:, 0] = 7
    lab[:] = (3, -1, 7, 299)
    tl[0, 0], tl[1, 0], tl[2, 0] = np.nan, np.inf, -np.inf
    loss, _, dz = check(orc, z, idx, tl, lab, wide=wide, tau=tau, w_kd=0.0, w_ce=1.0)
    assert np.isfinite(loss).all() and np.isfinite(dz).all()


@pytest.mark.parametrize("copies,wide", [(1, True), (1, False), (500, True)])
@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_logprobs_above_zero(orc, copies, wide, tau):
    check(orc, *positive_logprobs(), 0, copies, wide, tau=tau, logprobs=True)
