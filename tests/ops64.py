"""64-bit plain forms of the embedding, the per-head norm with rotation and the
distillation loss, with the rounding bounds that the binary32 calls have to keep
against them.  U is half a binary32 step relative to the value; every bound
counts roundings along the longest chain of the call's definition."""
import math

import numpy as np

U = 2.0 ** -24


def sum_roundings(L):
    """Roundings on the longest path of a canonical sum of L terms."""
    C = max(1, -(-L // 64))
    return min(L, 64) - 1 + math.ceil(math.log2(C)) if L else 0


# ---------------------------------------------------------------- embedding

def embed_fwd(W, tokens, scale, s_w, pad):
    tok = np.asarray(tokens).ravel()
    ok = (tok >= 0) & (tok < W.shape[0]) & (tok != pad)
    y = W[np.where(ok, tok, 0)].astype(np.float64) * (1.0 if s_w is None else float(s_w)) * float(np.float32(scale))
    return np.where(ok[:, None], y, 0.0)


def embed_bwd(dout, tokens, V, scale, pad, acc=None):
    """(gradient, bound)."""
    tok = np.asarray(tokens).ravel()
    D = dout.shape[-1]
    g, a = np.zeros((V, D)), np.zeros((V, D))
    cnt = np.zeros(V, dtype=np.int64)
    for i, t in enumerate(tok):
        if 0 <= t < V and t != pad:
            g[t] += dout[i].astype(np.float64)
            a[t] += np.abs(dout[i].astype(np.float64))
            cnt[t] += 1
    sc = float(np.float32(scale))
    k = np.array([sum_roundings(int(c)) + 2 for c in cnt])[:, None]
    g, bound = g * sc, a * abs(sc) * k * U * 1.01
    if acc is not None:
        g = g + acc
        bound = bound + U * np.abs(g) * 1.01
    return g, bound


# ---------------------------------------------------------------- norm and rotation

def pairs(R, interleaved):
    j = np.arange(R // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + R // 2)


def rotate(y, cs, R, interleaved, back=False):
    a, b = pairs(R, interleaved)
    c, s = cs[:, None, :R // 2], cs[:, None, R // 2:]
    if back:
        s = -s
    o = y.copy()
    o[..., a] = y[..., a] * c - y[..., b] * s
    o[..., b] = y[..., b] * c + y[..., a] * s
    return o


def mix(y, R, interleaved):
    """What a rotated element's error is measured by: both members of its pair."""
    a, b = pairs(R, interleaved)
    m = np.abs(y)
    o = m.copy()
    o[..., a] = o[..., b] = m[..., a] + m[..., b]
    return o


def norm_roundings(D):
    """Relative roundings of r: the squares and their sum (halved by the root),
    the division, the sum with eps, the root and the reciprocal."""
    return (1 + 3 + math.ceil(math.log2(max(1, -(-D // 4)))) + 2) / 2 + 2


def qk_fwd(x, rope, pos, gain, eps, interleaved):
    x = x.astype(np.float64)
    D, R = x.shape[-1], rope.shape[1]
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps)))
    if gain is not None:
        y = y * gain
    o = rotate(y, rope[pos].astype(np.float64), R, interleaved)
    return o, (norm_roundings(D) + 5) * U * mix(y, R, interleaved) * 1.01


def qk_bwd(do, x, rope, pos, gain, eps, interleaved):
    """(dx, bound, dgain, bound)."""
    x, do = x.astype(np.float64), do.astype(np.float64)
    n, H, D = x.shape
    R = rope.shape[1]
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps)))
    h = x * r
    dy = rotate(do, rope[pos].astype(np.float64), R, interleaved, back=True)
    ady = mix(do, R, interleaved)           # |cos|, |sin| <= 1
    nr = norm_roundings(D) + 1              # of h
    u, au = (dy, ady) if gain is None else (dy * gain, ady * np.abs(gain))
    eu = 3 * U                              # two products, a sum, (the gain)
    c1 = (u * h).mean(-1, keepdims=True)
    ac1 = (au * np.abs(h)).mean(-1, keepdims=True)
    ec1 = (nr + 4 + 1 + 3 + math.ceil(math.log2(max(1, -(-D // 4)))) + 1) * U
    dx = r * (u - h * c1)
    bound = r * (au * (eu + U) + np.abs(h) * ac1 * (ec1 + (nr + 2) * U) + (nr + 2) * U * (au + np.abs(h) * ac1))
    dg = bg = None
    if gain is not None:
        dg = (dy * h).sum((0, 1))
        bg = (ady * np.abs(h)).sum((0, 1)) * (nr + 4 + sum_roundings(n * H)) * U * 1.01
    return dx, bound * 1.01, dg, bg


# ---------------------------------------------------------------- distillation

def distill_rows(z, idx, tl, label, tau, w_kd, w_ce, w_z, logprobs):
    """Per row (loss, bound, dz for an upstream gradient of 1, bound)."""
    z = z.astype(np.float64)
    n, V = z.shape
    loss, lb = np.zeros(n), np.zeros(n)
    dz, db = np.zeros((n, V)), np.zeros((n, V))
    tau32 = float(np.float32(tau))
    for r in range(n):
        fin = np.isfinite(z[r])
        if not fin.any():
            continue
        u = z[r] / tau32
        lse_t = np.log(np.sum(np.exp(u - u[fin].max()))) + u[fin].max()
        lse = np.log(np.sum(np.exp(z[r] - z[r][fin].max()))) + z[r][fin].max()
        q, q1 = np.exp(u - lse_t), np.exp(z[r] - lse)
        ok = (idx[r] >= 0) & (idx[r] < V)
        t = tl[r][ok].astype(np.float64)
        cols = idx[r][ok]
        t = t if logprobs else t / tau32
        live = np.isfinite(t)
        t, cols = t[live], cols[live]
        if t.size:
            logp = t if logprobs else t - (np.log(np.sum(np.exp(t - t.max()))) + t.max())
            p = np.exp(logp)
        else:
            logp = p = np.zeros(0)
        P = p.sum()
        # e(x): the argument's difference and its two products (x log2 e), the polynomial and
        # the scaling; relative error |x| 2U + |u| 3U + 4U; sums: 8 + 7 + 32 + 5 roundings of
        # blocks and joins (V < 2^20) and the join's own e(.)
        mu, span = np.abs(u[fin]).max(), u[fin].max() - u[fin].min()
        mz, span1 = np.abs(z[r][fin]).max(), z[r][fin].max() - z[r][fin].min()
        ls_t, ls = U * (6 * mu + 2 * min(span, 100) + 70), U * (6 * mz + 2 * min(span1, 100) + 70)
        mt = np.abs(t).max() if t.size else 0.0
        rp = U * (6 * mt + 2 * min(t.max() - t.min() if t.size else 0.0, 100) + 50 + t.size / 32)
        d = logp - (u[cols] - lse_t)
        with np.errstate(invalid="ignore"):
            kd = np.sum(np.where(p > 0, p * d, 0.0)) if w_kd else 0.0
        loss[r] = w_kd * tau32 ** 2 * kd
        lb[r] = w_kd * tau32 ** 2 * (P * (ls_t + rp + U * (4 * mu + 4 * mt)) + rp * np.sum(np.abs(p * d)))
        b = 0.0
        if w_ce and label[r] >= 0:
            loss[r] += w_ce * (lse - z[r][label[r]])
            lb[r] += w_ce * ls
            b += w_ce
        loss[r] += w_z * lse ** 2
        lb[r] += w_z * 2 * abs(lse) * ls + U * abs(loss[r])
        b += 2 * w_z * lse
        # e to l: twice an e's error; the coefficients: ten roundings
        rq, rq1 = 2 * ls_t + 12 * U, 2 * ls + 12 * U + (ls / max(abs(lse), 1e-3) if w_z else 0.0)
        dz[r] = w_kd * tau32 * P * q + b * q1
        db[r] = w_kd * tau32 * P * q * (rq + rp) + abs(b) * q1 * rq1
        if w_kd:
            np.add.at(dz[r], cols, -w_kd * tau32 * p)
            np.add.at(db[r], cols, w_kd * tau32 * p * (rp + (4 + p.size) * U) + 2 * U * np.abs(q[cols]))
        if w_ce and label[r] >= 0:
            dz[r][label[r]] -= w_ce
            db[r][label[r]] += 4 * U * w_ce
        db[r] += 1e-37
    return loss, lb, dz, db
