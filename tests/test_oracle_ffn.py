"""The oracle's block norm, codes by row and column, product of codes and gated activation against
64-bit plain forms (bounds that count roundings), hand-worked orders, and gradients against
differences."""
import numpy as np
import pytest

import ffn64 as F

rng = np.random.default_rng
f32 = np.float32

NORM = [(1, 1), (2, 3), (5, 4), (3, 37), (17, 128), (33, 512), (4, 513), (2, 1001), (3, 2048), (1, 5000), (2, 16384)]


def norm_case(n, D, gate, post, gains, seed=0):
    g = rng(1000 * n + D + seed)
    r = lambda *s: g.standard_normal(s).astype(f32)  # noqa: E731
    c = dict(x=1.5 * r(n, D), y=0.7 * r(n, D), gate=None, g_post=None, g_pre=None)
    if gate:
        c["gate"] = (0.5 + 0.2 * r(D)).astype(f32) if gate == "channel" else (0.5 + 0.2 * r(n, D)).astype(f32)
    if gains:
        c["g_post"] = (1 + 0.1 * r(D)).astype(f32) if post else None
        c["g_pre"] = (1 + 0.1 * r(D)).astype(f32)
    if n > 2:
        c["x"][1], c["y"][1] = 0, 0
    c.update(dh=1e-3 * r(n, D), du=1e-3 * r(n, D))
    return c


@pytest.mark.parametrize("n,D", NORM)
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gains", [False, True])
def test_block_norm(orc, n, D, gate, post, gains):
    c = norm_case(n, D, gate, post, gains)
    kw = dict(gate=c["gate"], g_post=c["g_post"], g_pre=c["g_pre"], alpha=0.75, beta=0.3)
    h, u, st = orc.block_norm_fwd(c["x"], c["y"], post=post, eps=1e-5, **kw)
    F.holds(h, F.norm_fwd(c["x"], c["y"], c["gate"], c["g_post"], None, 0.75, 0.3, 1e-5, post), "h")
    F.holds(u, F.norm_u(h, c["g_pre"], 1e-5), "u")
    F.holds(st[:, 1:], F.rms(F.V(h), 1e-5), "r2")
    assert post or not st[:, 0].any()
    got = orc.block_norm_bwd(c["dh"], c["du"], h, c["y"], st, post=post, **kw)
    exp = F.norm_bwd(c["dh"], c["du"], h, c["y"], c["gate"], c["g_post"], c["g_pre"], st, 0.75, 0.3, post)
    for name, a, b in zip(("dx", "dy", "dgate", "dg_post", "dg_pre"), got, exp):
        assert (a is None) == (b is None), name
        if a is not None:
            F.holds(a, b, name)


def test_block_norm_parts(orc):
    """The norm before a block alone; no stream gradient; no gradient of u."""
    c = norm_case(6, 70, None, False, True)
    h, u, st = orc.block_norm_fwd(c["x"], g_pre=c["g_pre"])
    assert h is None
    F.holds(u, F.norm_u(c["x"], c["g_pre"], 1e-6))
    dx, dy, dgate, dgp, dgn = orc.block_norm_bwd(None, c["du"], c["x"], None, st, g_pre=c["g_pre"])
    ex = F.norm_bwd(None, c["du"], c["x"], None, None, None, c["g_pre"], st, 1, 1, False)
    F.holds(dx, ex[0])
    F.holds(dgn, ex[4])
    dx, dy, *_ = orc.block_norm_bwd(c["dh"], None, None, c["y"], st, alpha=0.5, beta=2.0)
    assert np.array_equal(dx, c["dh"] * f32(0.5)) and np.array_equal(dy, c["dh"] * f32(2))


def test_row_sum_order(orc):
    """Groups of 4 left to right, groups g, g + 32, .. in a chain, the chains by the tree: 2^24
    absorbs single ones that are added to it, and only those."""
    D = 512
    v = np.ones((1, D), dtype=f32)
    v[0, 0] = 2.0 ** 12
    _, _, st = orc.block_norm_fwd(v, eps=0.0)
    # chain 0: 2^24 (its group's ones are lost), then three groups of 4 (2^24 + 4, + 8, + 12); the
    # tree adds 16, 32, 64, 128 and 256 of the other chains, all exact
    S = 2.0 ** 24 + 12 + 16 * 31
    r = f32(1) / np.sqrt(f32(S) / f32(D))
    assert st[0, 1] == r


def test_token_sum_order(orc):
    """Chunks of 8 tokens, left to right, then the tree."""
    n = 40
    h, du = np.ones((n, 1), dtype=f32), np.ones((n, 1), dtype=f32)
    du[0] = 2.0 ** 24
    st = np.tile(f32([0, 1]), (n, 1))
    dgn = orc.block_norm_bwd(None, du, h, None, st, g_pre=np.ones(1, dtype=f32))[4]
    assert dgn[0] == 2.0 ** 24 + 32                     # the first chunk's other tokens are lost
    dgn = orc.block_norm_bwd(None, du, h, None, st, g_pre=np.ones(1, dtype=f32), acc=[None, None, f32([4.0])])[4]
    assert dgn[0] == 2.0 ** 24 + 36
    none = np.zeros((0, 3), dtype=f32)
    assert not orc.block_norm_bwd(None, none, none, None, np.zeros((0, 2), f32), g_pre=np.ones(3, f32))[4].any()


def plain(x, y, gate, gp, gn, alpha, beta, eps, post):
    def unit(v):
        return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    p = unit(y) * gp if post else y
    h = alpha * x + beta * p * gate
    return h, unit(h) * gn


@pytest.mark.parametrize("gate", ["channel", "token"])
@pytest.mark.parametrize("post", [False, True])
def test_block_norm_gradient_against_differences(orc, gate, post):
    """dx, dy, dgate and the gains' gradients against central differences of the formula in 64 bits:
    step t leaves an error of t^2 times the third derivative (order 1) and 2^-52 / t of rounding."""
    c = norm_case(3, 10, gate, post, True, seed=7)
    gp = c["g_post"] if post else np.ones(10, f32)
    args = {k: np.asarray(v, dtype=np.float64) for k, v in
            dict(x=c["x"], y=c["y"], gate=c["gate"], gp=gp, gn=c["g_pre"]).items()}
    args["y"][1] = c["y"][1] = 0.3                              # no point at the norm's kink of eps
    args["x"][1] = c["x"][1] = -0.6
    g = rng(3)
    wh, wu = g.standard_normal((3, 10)).astype(f32), g.standard_normal((3, 10)).astype(f32)

    def total(a):
        h, u = plain(a["x"], a["y"], a["gate"], a["gp"], a["gn"], 0.75, float(f32(0.3)), 1e-6, post)
        return (h * wh).sum() + (u * wu).sum()

    h, u, st = orc.block_norm_fwd(c["x"], c["y"], gate=c["gate"], g_post=c["g_post"], g_pre=c["g_pre"], alpha=0.75,
                                  beta=0.3, post=post)
    got = dict(zip(("x", "y", "gate", "gp", "gn"),
                   orc.block_norm_bwd(wh, wu, h, c["y"], st, gate=c["gate"], g_post=c["g_post"], g_pre=c["g_pre"],
                                      alpha=0.75, beta=0.3, post=post)))
    t = 1e-5
    for name, a in args.items():
        if got[name] is None:
            continue
        for i in np.ndindex(a.shape):
            old = a[i]
            a[i] = old + t
            hi = total(args)
            a[i] = old - t
            lo = total(args)
            a[i] = old
            # binary32 intermediate values of order 1 to 10 over at most 30 terms: 1e-5
            assert abs((hi - lo) / (2 * t) - got[name][i]) < 2e-5 * (1 + abs(got[name][i])), (name, i)


# ---------------------------------------------------------------- codes

@pytest.mark.parametrize("n,D", [(1, 1), (3, 5), (7, 130), (2, 6000), (40, 33)])
@pytest.mark.parametrize("columns", [False, True])
@pytest.mark.parametrize("with_mul", [False, True])
def test_quant_rows(orc, n, D, columns, with_mul):
    g = rng(n + D)
    x = g.standard_normal((n, D)).astype(f32)
    x[0] *= 1e-4
    x[:, D // 2] = 0
    mul = (0.01 + g.random(n if columns else D)).astype(f32) if with_mul else None
    q, s = orc.quant_rows(x, mul, columns)
    eq, es = F.quant_rows(x, mul, columns)
    assert np.array_equal(s, es) and np.array_equal(q, eq)


def test_quant_ties_and_the_unordinary(orc):
    x = f32([[127, 0.5, 1.5, -2.5, 126.5], [0, -0.0, 0, 0, 0], [np.inf, 1, -3, 0, 2], [np.nan, 127, -64, 0.5, 3],
             [1e-41, 1e-42, 0, 0, 0]])
    q, s = orc.quant_rows(x)
    assert q.tolist() == [[127, 0, 2, -2, 126], [0] * 5, [0] * 5, [0, 127, -64, 0, 3], [0] * 5]
    assert s[0] == 1 and s[1] == 0 and np.isinf(s[2]) and s[3] == 1 and s[4] == 0
    q, s = orc.quant_rows(np.zeros((0, 3), f32), columns=True)
    assert s.tolist() == [0, 0, 0]


@pytest.mark.parametrize("M,N,K", [(1, 1, 0), (1, 1, 1), (3, 5, 7), (17, 4, 300), (2, 3, 40000)])
@pytest.mark.parametrize("a_t", [False, True])
@pytest.mark.parametrize("b_t", [False, True])
def test_matmul(orc, M, N, K, a_t, b_t):
    g = rng(M + N + K)
    a, b = g.integers(-127, 128, (M, K)).astype(np.int8), g.integers(-127, 128, (N, K)).astype(np.int8)
    if M > 1:
        a[1], b[0] = 127, 127
    sa, sb = (g.random(M) * 0.1).astype(f32), (g.random(N) * 0.01).astype(f32)
    acc = a.astype(np.int64) @ b.astype(np.int64).T
    v = acc.astype(f32) * sa[:, None] * sb
    at, bt = a.T if a_t else a, b.T if b_t else b
    assert np.array_equal(orc.matmul_i8(at, bt, sa, sb, a_t, b_t), v)
    old = g.standard_normal((M, N)).astype(f32)
    assert np.array_equal(orc.matmul_i8(at, bt, sa, sb, a_t, b_t, old), old + v)
    assert np.array_equal(orc.matmul_i8(at, bt, a_t=a_t, b_t=b_t), acc.astype(f32))


# ---------------------------------------------------------------- gated activation

@pytest.mark.parametrize("n,Fw", [(1, 1), (3, 127), (2, 128), (2, 129), (5, 300)])
def test_swiglu(orc, n, Fw):
    g = rng(n + Fw)
    gu = (3 * g.standard_normal((n, 2 * Fw))).astype(f32)
    gu[0, 0] = 0
    a, codes, scales = orc.swiglu_fwd(gu)
    F.holds(a, F.swiglu_fwd(gu))
    G = -(-Fw // 128)
    pad = np.zeros((n, 2, G * 128), dtype=f32)
    pad[:, :, :Fw] = gu.reshape(n, 2, Fw)
    eq, es = F.quant_rows(pad.reshape(-1, 128), None, False)
    assert np.array_equal(codes.reshape(-1, 128), eq) and np.array_equal(scales.ravel(), es)
    da = g.standard_normal((n, Fw)).astype(f32)
    for src, (gv, uv) in ((dict(gu=gu), (F.V(gu[:, :Fw]), F.V(gu[:, Fw:]))),
                          (dict(codes=codes, scales=scales), F.decode(codes, scales, Fw))):
        dgu = orc.swiglu_bwd(da, **src)
        dg, du = F.swiglu_bwd(da, gv, uv)
        F.holds(dgu[:, :Fw], dg)
        F.holds(dgu[:, Fw:], du)


def test_swiglu_far_from_zero(orc):
    """sig neither overflows nor loses bits far out: silu(90) = 90, silu(-90) = -90 e^-90 = 0 by
    the flush; the slopes 1 and 0."""
    gu = f32([[90, -90, 20, -20, -0.0, 1, 1, 1, 1, 1]])
    a, *_ = orc.swiglu_fwd(gu)
    assert a[0, 0] == 90 and a[0, 1] == 0 and np.signbit(a[0, 4])
    F.holds(a[:, 2:4], F.swiglu_fwd(gu[:, [2, 3, 7, 8]]))
    d = orc.swiglu_bwd(np.ones((1, 5), f32), gu=gu)
    assert d[0, 0] == 1 and d[0, 1] == 0 and d[0, 4] == 0.5


def test_swiglu_gradient_against_differences(orc):
    g = rng(5)
    gu, da = g.standard_normal((2, 12)).astype(f32), g.standard_normal((2, 6)).astype(f32)
    got = orc.swiglu_bwd(da, gu=gu)
    x, t = gu.astype(np.float64), 1e-5

    def total(x):
        return (da * x[:, :6] / (1 + np.exp(-x[:, :6])) * x[:, 6:]).sum()

    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + t
        hi = total(x)
        x[i] = old - t
        lo = total(x)
        x[i] = old
        assert abs((hi - lo) / (2 * t) - got[i]) < 2e-6 * (1 + abs(got[i]))


@pytest.mark.parametrize("T,N,K", [(40, 12, 9), (7, 33, 20)])
def test_gradient_products(orc, T, N, K):
    """The gradients of Y = X W^T as products of codes, against those of the dequantised product: a code
    is at most half a step from its value (and two roundings of the value, its scale and its product),
    so dX is off by half a step times the sum of the codes that it meets, and dW alike."""
    g = rng(T)
    X, W, dY = (g.standard_normal(s).astype(f32) for s in ((T, K), (N, K), (T, N)))
    xq, sx = orc.quant_rows(X)
    wq, sw = orc.quant_rows(W)
    Xd, Wd = xq * sx[:, None].astype(np.float64), wq * sw[:, None].astype(np.float64)
    q, qs = orc.quant_rows(dY, sw)
    dX = orc.matmul_i8(q, wq, qs, None, False, True)
    bound = 0.5 * qs[:, None] * np.abs(wq).sum(0)[None].astype(np.float64)
    assert np.all(np.abs(dX - dY @ Wd) <= bound * (1 + 1e-4) + 1e-5 * np.abs(dY) @ np.abs(Wd))
    q, qs = orc.quant_rows(dY, sx, True)
    dW = orc.matmul_i8(q, xq, qs, None, True, True)
    bound = 0.5 * qs[:, None] * np.abs(xq).sum(0)[None].astype(np.float64)
    assert np.all(np.abs(dW - dY.T @ Xd) <= bound * (1 + 1e-4) + 1e-5 * np.abs(dY.T) @ np.abs(Xd))
    # and against differences of the dequantised product, weighted by dY (linear: exact but for 2^-52 / t)
    t = 1e-3
    for i in ((0, 0), (T - 1, K - 1)):
        hi, lo = Xd.copy(), Xd.copy()
        hi[i] += t
        lo[i] -= t
        d = ((hi @ Wd.T * dY).sum() - (lo @ Wd.T * dY).sum()) / (2 * t)
        assert abs(d - dX[i]) <= 0.5 * qs_of(orc, dY, sw)[i[0]] * np.abs(wq[:, i[1]]).sum() * (1 + 1e-4) + 1e-6


def qs_of(orc, dY, mul):
    return orc.quant_rows(dY, mul)[1]
