"""64-bit plain forms of the block norm, the codes by row or column, their product and the
gated activation, with the error that the binary32 calls may have against them.

V carries a value and a bound on the error of its binary32 counterpart; every operation adds
half a step of its result, U = 2^-24 relative (and what a flushed subnormal loses), to what its
operands bring.  The bounds of whole calls follow operation by operation, before any run."""
import math

import numpy as np

U = 2.0 ** -24
TINY = 2.0 ** -126


class V:
    def __init__(self, v, e=0.0):
        self.v = np.asarray(v, dtype=np.float64)
        self.e = np.broadcast_to(np.asarray(e, dtype=np.float64), self.v.shape)

    def _round(self, v, e):
        return V(v, e + U * (np.abs(v) + e) + TINY)

    def __mul__(self, o):
        o = o if isinstance(o, V) else V(o)
        return self._round(self.v * o.v, np.abs(self.v) * o.e + np.abs(o.v) * self.e + self.e * o.e)

    def __add__(self, o):
        o = o if isinstance(o, V) else V(o)
        return self._round(self.v + o.v, self.e + o.e)

    def __sub__(self, o):
        return self + V(-o.v, o.e)

    def __truediv__(self, o):
        o = o if isinstance(o, V) else V(o)
        low = np.abs(o.v) - o.e
        return self._round(self.v / o.v, (self.e + np.abs(self.v / o.v) * o.e) / low)

    def sqrt(self):
        low = np.maximum(self.v - self.e, 1e-300)
        return self._round(np.sqrt(self.v), self.e / (np.sqrt(low) + np.sqrt(self.v)))

    def __getitem__(self, i):
        return V(self.v[i], self.e[i])

    def row_sum(self):
        """Sum over the last axis, as S: at most 3 additions in a group, 3 in a chain, the tree."""
        D = self.v.shape[-1]
        C = 32
        while 16 * C < D:
            C *= 2
        return self._sum(-1, 6 + int(math.log2(C)))

    def token_sum(self):
        """Sum over the first axis: chunks of 8, the tree."""
        n = self.v.shape[0]
        return self._sum(0, 7 + math.ceil(math.log2(max(1, -(-n // 8)))))

    def _sum(self, axis, roundings):
        a = (np.abs(self.v) + self.e).sum(axis)
        return V(self.v.sum(axis), self.e.sum(axis) + 1.01 * roundings * U * a + self.v.shape[axis] * TINY)


def holds(got, ref, what=""):
    d = np.abs(np.asarray(got, dtype=np.float64) - ref.v)
    assert np.all(d <= 1.01 * ref.e + 1e-300), (what, float((d - ref.e).max()))


def rms(v, eps):
    D = v.v.shape[-1]
    m = (v * v).row_sum() / float(D) + np.float64(np.float32(eps))
    return (V(1.0) / m.sqrt())[..., None]


def norm_fwd(x, y, gate, gp, gn, alpha, beta, eps, post):
    """(h, p) and then u of a stored h by norm_u."""
    if y is None:
        return V(x)
    p = V(y)
    if post:
        p = p * rms(p, eps)
        if gp is not None:
            p = p * V(gp)
    if gate is not None:
        p = p * V(gate)
    return V(x) * np.float64(np.float32(alpha)) + p * np.float64(np.float32(beta))


def norm_u(h, gn, eps):
    h = V(h)
    u = h * rms(h, eps)
    return u if gn is None else u * V(gn)


def _back(v, unit, r):
    D = v.v.shape[-1]
    c = ((v * unit).row_sum() / float(D))[..., None]
    return r * (v - unit * c)


def norm_bwd(dh, du, h, y, gate, gp, gn, stats, alpha, beta, post):
    """(dx, dy, dgate, dgp, dgn)"""
    r1, r2 = V(stats[:, :1]), V(stats[:, 1:])
    dgn = dy = dgate = dgp = None
    g = None if dh is None else V(dh)
    if du is not None:
        hn = V(h) * r2
        v = V(du) if gn is None else V(du) * V(gn)
        if gn is not None:
            dgn = (V(du) * hn).token_sum()
        e = _back(v, hn, r2)
        g = e if g is None else g + e
    if y is None:
        return g, dy, dgate, dgp, dgn
    dx, b = g * np.float64(np.float32(alpha)), g * np.float64(np.float32(beta))
    yn = V(y) * r1 if post else V(y)
    p = yn * V(gp) if gp is not None else yn
    q = b
    if gate is not None:
        dgate = b * p
        dgate = dgate if np.ndim(gate) == 2 else dgate.token_sum()
        q = b * V(gate)
    dy = q
    if post:
        if gp is not None:
            dgp = (q * yn).token_sum()
            q = q * V(gp)
        dy = _back(q, yn, r1)
    return dx, dy, dgate, dgp, dgn


def codes(v, s):
    """Codes of float32 values by float32 scales: the quotient in 64 bits rounds to binary32 as
    the exact one does (53 >= 2 24 + 2 bits)."""
    with np.errstate(all="ignore"):
        q = (v.astype(np.float64) / s.astype(np.float64)).astype(np.float32)
    q = np.rint(np.where(np.isnan(q) | (s == 0), np.float32(0), q))
    return np.clip(q, -127, 127).astype(np.int8)


def quant_rows(x, mul, columns):
    v = x.astype(np.float32)
    if mul is not None:
        v = v * (mul[:, None] if columns else mul)
    s = (np.abs(v).max(0 if columns else 1).astype(np.float64) / 127.0).astype(np.float32)
    return codes(v, s if columns else s[:, None]), s


def sigmoids(g):
    """sig(g), sig(-g); exp_r is within 4 U (reduction, 8 rounded steps of which the last weighs
    most, scaling)."""
    e = V(np.exp(-np.abs(g.v)), 4 * U * np.exp(-np.abs(g.v)) + np.exp(-np.abs(g.v)) * 1.01 * g.e + TINY)
    w = V(1.0) / (V(np.ones_like(e.v)) + e)
    ew = e * w
    pos = g.v >= 0
    return (V(np.where(pos, w.v, ew.v), np.where(pos, w.e, ew.e)), V(np.where(pos, ew.v, w.v), np.where(pos, ew.e, w.e)))


def swiglu_fwd(gu):
    F = gu.shape[1] // 2
    g, u = V(gu[:, :F]), V(gu[:, F:])
    return g * sigmoids(g)[0] * u


def swiglu_bwd(da, g, u):
    """(dgate, dup) of gate and up as V."""
    s, t = sigmoids(g)
    return V(da) * u * s * (V(np.ones_like(g.v)) + g * t), V(da) * (g * s)


def decode(codes_, scales, F):
    """V of gate and up out of the 8-bit copy."""
    n = codes_.shape[0]
    x = V(codes_.astype(np.float64)) * V(scales[..., None])
    v, e = (t.reshape(n, 2, -1)[:, :, :F] for t in (x.v, x.e))
    return V(v[:, 0], e[:, 0]), V(v[:, 1], e[:, 1])
