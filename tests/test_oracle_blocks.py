"""The oracle's embedding, per-head norm with rotation and distillation loss
against 64-bit plain forms (bounds that count roundings), hand-worked orders, and
gradients against differences."""
import math

import numpy as np
import pytest

import ops64 as F

rng = np.random.default_rng


def rope_table(P, R, theta=500000.0):
    ang = np.arange(P)[:, None] * theta ** (-2.0 * np.arange(R // 2) / max(R, 1))[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


@pytest.mark.parametrize("n,V,D,scale,pad", [(1, 1, 1, 1.0, -1), (7, 5, 3, 2.5, 2), (200, 3, 4, 0.3, -1),
                                             (5000, 40, 2, 1.0, 0)])
def test_embed(orc, n, V, D, scale, pad):
    g = rng(n)
    tok = g.integers(0, V, n)
    W = g.standard_normal((V, D)).astype(np.float32)
    exp = F.embed_fwd(W, tok, scale, None, pad)
    assert np.all(np.abs(orc.embed_fwd(W, tok, scale, pad=pad) - exp) <= F.U * np.abs(exp))
    q = g.integers(-127, 128, (V, D)).astype(np.int8)
    exp = F.embed_fwd(q, tok, scale, np.float32(0.013), pad)
    assert np.all(np.abs(orc.embed_fwd(q, tok, scale, 0.013, pad) - exp) <= 2.01 * F.U * np.abs(exp))
    dout = g.standard_normal((n, D)).astype(np.float32)
    for acc in (None, g.standard_normal((V, D)).astype(np.float32)):
        exp, bound = F.embed_bwd(dout, tok, V, scale, pad, acc)
        assert np.all(np.abs(orc.embed_bwd(dout, tok, V, scale, pad, acc) - exp) <= bound)


def test_embed_gradient_order(orc):
    """Positions ascending in chunks of 64, then the pairwise tree: 2^24 absorbs
    the ones that follow it in its chunk, and only those."""
    n = 200
    d = np.ones((n, 1), dtype=np.float32)
    d[0] = 2.0 ** 24
    got = orc.embed_bwd(d, np.zeros(n, dtype=np.int64), 1)
    # chunk sums 2^24, 64, 64, 8; (2^24 + 64) + (64 + 8)
    assert got[0, 0] == 2.0 ** 24 + 136
    got = orc.embed_bwd(d, np.zeros(n, dtype=np.int64), 1, scale=0.5, acc=np.ones((1, 1), dtype=np.float32))
    assert got[0, 0] == 2.0 ** 23 + 68 + 1


SHAPES = [(3, 2, 1, 0), (2, 1, 2, 2), (5, 3, 6, 4), (4, 2, 33, 10), (3, 4, 80, 40), (2, 2, 128, 128), (1, 3, 512, 512)]


@pytest.mark.parametrize("n,H,D,R", SHAPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("with_gain", [False, True])
def test_qk(orc, n, H, D, R, inter, with_gain):
    g = rng(D + n)
    x = g.standard_normal((n, H, D)).astype(np.float32)
    x[0, 0] = 0.0
    do = g.standard_normal((n, H, D)).astype(np.float32)
    gain = (1 + 0.1 * g.standard_normal(D)).astype(np.float32) if with_gain else None
    rope, pos = rope_table(50, R), g.integers(0, 50, n)
    exp, bound = F.qk_fwd(x, rope, pos, gain, 1e-6, inter)
    assert np.all(np.abs(orc.qk_fwd(x, rope, pos, gain, 1e-6, inter) - exp) <= bound)
    dx, bx, dg, bg = F.qk_bwd(do, x, rope, pos, gain, 1e-6, inter)
    got, got_g = orc.qk_bwd(do, x, rope, pos, gain, 1e-6, inter)
    assert np.all(np.abs(got - dx) <= bx)
    if with_gain:
        assert np.all(np.abs(got_g - dg) <= bg)


def test_qk_plain_gradient_matches_differences():
    g = rng(3)
    n, H, D, R = 2, 2, 10, 6
    x, do = g.standard_normal((n, H, D)), g.standard_normal((n, H, D))
    gain, rope, pos = 1 + 0.2 * g.standard_normal(D), rope_table(9, R).astype(np.float64), np.array([3, 7])
    f = lambda x, gain: np.sum(F.qk_fwd(x, rope, pos, gain, 1e-5, True)[0] * do)  # noqa: E731
    dx, _, dg, _ = F.qk_bwd(do, x, rope, pos, gain, 1e-5, True)
    h = 1e-5
    for i in [(0, 0, 0), (1, 1, 9), (0, 1, 5)]:
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, gain) - f(x - e, gain)) / (2 * h) - dx[i]) < 1e-7
    for d in (0, 5, 9):
        e = np.zeros(D)
        e[d] = h
        assert abs((f(x, gain + e) - f(x, gain - e)) / (2 * h) - dg[d]) < 1e-7


def test_qk_norm_order(orc):
    """Groups of 4 left to right, then the pairwise tree (adjacent groups first)."""
    x = np.zeros((1, 1, 16), dtype=np.float32)
    x[0, 0, :] = 1.0
    x[0, 0, 0] = 2.0 ** 12                   # its square absorbs single ones of its group
    S = np.float32(np.float32(2.0 ** 24 + 4) + np.float32(8))
    r = np.float32(1) / np.sqrt(np.float32(S / np.float32(16)) + np.float32(0))
    got = orc.qk_fwd(x, np.zeros((1, 0), dtype=np.float32), [0], None, 0.0)
    assert got[0, 0, 1] == r and got[0, 0, 0] == np.float32(2.0 ** 12) * r


def test_exp2_and_ln(orc):
    t = np.concatenate([np.linspace(-125, 0, 20001), -np.logspace(-30, 2, 500)]).astype(np.float32)
    got = np.array([orc.exp2_neg(v) for v in t], dtype=np.float64)
    exp = np.exp2(t.astype(np.float64))
    # the polynomial's 5.4e-8 (0.9 U), the table entry's rounding, those of the polynomial's
    # last sum (on a value of at least 0.989: 1.02 U) and of the product, and the small ones of
    # the terms below them (|f| <= 1/64: 0.04 U)
    assert np.all(np.abs(got - exp) <= 4 * F.U * exp)
    assert orc.exp2_neg(0.0) == 1.0 and orc.exp2_neg(-126.0) == 0.0 and orc.exp2_neg(-math.inf) == 0.0
    assert math.isnan(orc.exp2_neg(math.nan))
    x = np.concatenate([np.logspace(-30, 30, 3001), 1 + np.linspace(-0.5, 1, 3001)]).astype(np.float32)
    got = np.array([orc.ln(v) for v in x])
    exp = np.log(x.astype(np.float64))
    # k ln 2 rounded twice and the series' last steps, in 64 bits
    assert np.all(np.abs(got - exp) <= 4 * 2.0 ** -53 * np.maximum(np.abs(exp), 1.0))


def case(seed, n, V, K):
    g = rng(seed)
    z = (2 * g.standard_normal((n, V))).astype(np.float32)
    idx = np.stack([g.permutation(V)[:K] if V >= K else g.integers(0, V, K) for _ in range(n)]).reshape(n, K)
    tl = (2 * g.standard_normal((n, K)) + 3).astype(np.float32)
    idx[g.random((n, K)) < 0.1] = -1
    lab = g.integers(0, V, n)
    lab[::3] = -100
    return z, idx, tl, lab


HP = [dict(), dict(tau=2.0), dict(tau=2.0, w_kd=0.7, w_ce=0.3, w_z=1e-3), dict(w_kd=0.5, w_ce=0.5, w_z=1e-4),
      dict(w_kd=0.0, w_ce=1.0), dict(tau=0.5, logprobs=True), dict(tau=4.0, w_kd=0.5, w_ce=0.5),
      dict(tau=1.5, w_kd=0.5, w_ce=0.5, w_z=1e-4)]


@pytest.mark.parametrize("n,V,K", [(2, 1, 1), (3, 130, 0), (4, 1025, 17), (2, 3000, 70)])
@pytest.mark.parametrize("hp", HP)
def test_distill(orc, n, V, K, hp):
    z, idx, tl, lab = case(V, n, V, K)
    if hp.get("logprobs"):
        tl = (tl - 6).astype(np.float32)
    full = dict(tau=1.0, w_kd=1.0, w_ce=0.0, w_z=0.0, logprobs=False)
    full.update(hp)
    loss, stats = orc.distill_fwd(z, idx, tl, lab, **full)
    el, bl, ez, bz = F.distill_rows(z, idx, tl, lab, **full)
    assert np.all(np.abs(loss - el) <= bl)
    back = {k: v for k, v in full.items() if k != "logprobs"}
    got = orc.distill_bwd(z, idx, stats, np.ones(1, dtype=np.float32), lab, **back)
    assert np.all(np.abs(got - ez) <= bz)


def test_distill_plain_gradient_matches_differences():
    z, idx, tl, lab = case(5, 2, 40, 6)
    hp = dict(tau=1.7, w_kd=0.7, w_ce=0.3, w_z=0.01, logprobs=False)
    hp["tau"] = float(np.float32(1.7))
    _, _, dz, _ = F.distill_rows(z, idx, tl, lab, **hp)
    h = 1e-5
    for r, j in [(0, 0), (1, 39), (0, int(idx[0].max())), (1, int(lab[1]))]:
        e = np.zeros(z.shape)
        e[r, j] = h
        up, dn = F.distill_rows(z + e, idx, tl, lab, **hp)[0], F.distill_rows(z - e, idx, tl, lab, **hp)[0]
        assert abs((up[r] - dn[r]) / (2 * h) - dz[r, j]) < 1e-7


def test_distill_masked_rows(orc):
    """Masked logits, rows that their mask leaves empty, the type's lowest value,
    teachers without weight, repeated entries, NaN."""
    V, K = 300, 4
    z, idx, tl, lab = case(9, 6, V, K)
    idx[:] = np.arange(K) * 7
    lab[:] = 50
    z[0, 60:] = -np.inf                    # most of the row masked
    z[1] = -np.inf                         # nothing left
    z[2, 60:] = np.finfo(np.float32).min   # masked by the lowest value
    z[3, 100] = np.nan
    tl[4] = -np.inf                        # a teacher without weight
    idx[5] = 7                             # one column four times
    hp = dict(tau=1.0, w_kd=1.0, w_ce=1.0, w_z=0.1)
    loss, stats = orc.distill_fwd(z, idx, tl, lab, **hp)
    dz = orc.distill_bwd(z, idx, stats, np.ones(1, dtype=np.float32), lab, **hp)
    rows = [0, 2, 4, 5]
    el, bl, ez, bz = F.distill_rows(z[rows], idx[rows], tl[rows], lab[rows], **hp, logprobs=False)
    assert np.all(np.abs(loss[rows] - el) <= bl)
    assert np.all(np.abs(dz[rows] - ez) <= bz)
    assert np.all(dz[0, 60:] == 0) and np.all(dz[2, 60:] == 0)
    assert loss[1] == 0 and np.all(dz[1] == 0)
    assert np.isnan(loss[3]) and np.all(np.isnan(dz[3]))
