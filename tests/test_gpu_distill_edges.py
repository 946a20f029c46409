"""GPU: the distillation loss bit for bit against the oracle where a row's values are
not ordinary."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import bitwise_reproducible_int8_gb300 as R  # noqa: E402
from gpu_helpers import dev  # noqa: E402
from test_gpu_blocks import BF, bf, run_distill, same  # noqa: E402
from test_oracle_distill_edges import MIXES, both, masked_rows, nonfinite_teachers, overflowing_rows  # noqa: E402

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
