"""GPU: the block norm, the codes by row and column, the product of codes and the gated activation,
bit for bit against the oracle over their types, widths, strides, forms and lengths."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import bitwise_reproducible_int8_gb300 as R  # noqa: E402
import ffn64 as F  # noqa: E402
from gpu_helpers import dev, host  # noqa: E402
from test_gpu_blocks import bf, same, strided  # noqa: E402
from test_oracle_ffn import norm_case  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
rng = np.random.default_rng
f32 = np.float32

LAYOUTS = {"dense": (0, 0), "strided": (8, 0), "odd": (3, 1)}


# ---------------------------------------------------------------- codes

QUANT = [(1, 1), (1, 5000), (3, 5), (5, 127), (4, 512), (9, 513), (130, 96), (33, 2048), (7, 8192), (5, 8193), (3, 20000),
         (1000, 33), (257, 1001)]


@pytest.mark.parametrize("n,D", QUANT)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("columns", [False, True])
@pytest.mark.parametrize("with_mul", [False, True])
@pytest.mark.parametrize("kind", [F32, BF])
def test_quant_rows(orc, n, D, layout, columns, with_mul, kind):
    g = rng(n + D)
    x = (g.standard_normal((n, D)) * 10.0 ** g.integers(-6, 6, (n, 1))).astype(f32)
    x[n // 2] = 0
    x[:, D // 3] = 0
    x = bf(x) if kind == BF else x
    mul = (0.01 + g.random(n if columns else D)).astype(f32) if with_mul else None
    extra, off = LAYOUTS[layout]
    q = strided(np.full((n, D), 55, dtype=np.int8), extra, off, torch.int8)
    s = torch.full((D if columns else n,), 9.0, device="cuda")
    R.repro_quant_rows_i8(strided(x, extra, off, kind), q, s, mul=None if mul is None else dev(mul), columns=columns)
    eq, es = orc.quant_rows(x, mul, columns)
    same(host(s), es)
    assert np.array_equal(host(q), eq)


@pytest.mark.parametrize("columns", [False, True])
def test_quant_ties(orc, columns):
    """Quotients that are halves, or a unit or two from them, for scales of every size: the shortcut
    past the division has to round all of them as it does."""
    g = rng(11)
    S, L = 600, 1024
    top = (g.random(S) + 1).astype(f32) * f32(2.0) ** g.integers(-60, 60, S).astype(f32)
    s = (top.astype(np.float64) / 127).astype(f32)
    halves = (g.integers(-127, 127, (S, L)) + 0.5) * s[:, None].astype(np.float64)
    x = halves.astype(f32)
    bump = g.integers(-2, 3, (S, L))
    x = (x.view(np.int32) + bump.astype(np.int32)).view(f32)
    x[:, 0] = top
    x = np.where(np.abs(x) > top[:, None], top[:, None], x)
    xs = np.ascontiguousarray(x.T) if columns else x
    q, sc = torch.empty(xs.shape, dtype=torch.int8, device="cuda"), torch.empty(S, device="cuda")
    R.repro_quant_rows_i8(dev(xs), q, sc, columns=columns)
    eq, es = orc.quant_rows(xs, None, columns)
    same(host(sc), es)
    assert np.array_equal(host(q), eq)


def test_quant_unordinary(orc):
    tiny = f32(2.0) ** -126
    x = np.zeros((9, 40), f32)
    x[0, :5] = [np.inf, 1, -3, 0, 2]
    x[1, :5] = [np.nan, 127, -64, 0.5, 3]
    x[2, :3] = [tiny, tiny / 2, -tiny]
    x[3, :3] = [127 * tiny, 0.5 * tiny, -64 * tiny]
    x[4, :3] = [3e38, -1e38, 1e37]
    x[5] = np.nan
    x[6, :2] = [-np.inf, np.nan]
    x[7, :3] = [f32(2.0) ** -100, f32(2.0) ** -101, 0]
    for columns in (False, True):
        xs = np.ascontiguousarray(x.T) if columns else x
        q, s = torch.empty(xs.shape, dtype=torch.int8, device="cuda"), torch.empty(9, device="cuda")
        R.repro_quant_rows_i8(dev(xs), q, s, columns=columns)
        eq, es = orc.quant_rows(xs, None, columns)
        same(host(s), es)
        assert np.array_equal(host(q), eq)
    s = torch.full((40,), 3.0, device="cuda")
    R.repro_quant_rows_i8(torch.empty((0, 40), device="cuda"), torch.empty((0, 40), dtype=torch.int8, device="cuda"), s,
                          columns=True)
    assert not host(s).any()


# ---------------------------------------------------------------- gated activation

@pytest.mark.parametrize("n,Fw", [(1, 1), (3, 127), (2, 128), (5, 129), (33, 256), (4, 1001), (130, 384), (2, 5632)])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("kind", [F32, BF])
@pytest.mark.parametrize("a_kind", [F32, BF])
def test_swiglu(orc, n, Fw, layout, kind, a_kind):
    g = rng(n + Fw)
    gu = (3 * g.standard_normal((n, 2 * Fw))).astype(f32)
    if Fw > 5:
        gu[0, :6] = [0, -0.0, 90, -90, 1e-41, 300]
    gu = bf(gu) if kind == BF else gu
    ea, codes, scales = orc.swiglu_fwd(gu)
    extra, off = LAYOUTS[layout]
    G = -(-Fw // 128)
    gt = strided(gu, extra, off, kind)
    for keep in (False, True):
        a = strided(np.zeros((n, Fw), f32), extra, off, a_kind)
        ct = torch.full((n, 2, G, 128), 99, dtype=torch.int8, device="cuda") if keep else None
        st = torch.full((n, 2, G), 9.0, device="cuda") if keep else None
        R.repro_swiglu_fwd(gt, a, ct, st)
        same(host(a.float()), bf(ea) if a_kind == BF else ea)
    assert np.array_equal(host(ct), codes)
    same(host(st), scales)
    da = g.standard_normal((n, Fw)).astype(f32)
    da = bf(da) if a_kind == BF else da
    dt = strided(da, extra, off, a_kind)
    for src, t in ((dict(gu=gu), dict(gu=gt)), (dict(codes=codes, scales=scales), dict(codes=ct, scales=st))):
        dgu = strided(np.zeros((n, 2 * Fw), f32), extra, off, kind)
        R.repro_swiglu_bwd(dt, dgu, **t)
        e = orc.swiglu_bwd(da, **src)
        same(host(dgu.float()), bf(e) if kind == BF else e)


def test_swiglu_unordinary(orc):
    """Infinities and NaN as the operations give them; a group that holds an infinity has no finite
    copy, one that holds a NaN passes over it."""
    gu = np.ones((4, 512), f32)
    gu[0, 3], gu[1, 300], gu[2, 7], gu[3, 5] = np.inf, np.nan, -np.inf, np.nan
    ea, codes, scales = orc.swiglu_fwd(gu)
    a, ct, st = (torch.empty(s, device="cuda", dtype=t) for s, t in
                 (((4, 256), F32), ((4, 2, 2, 128), torch.int8), ((4, 2, 2), F32)))
    R.repro_swiglu_fwd(dev(gu), a, ct, st)
    same(host(a), ea)
    same(host(st), scales)
    assert np.array_equal(host(ct), codes)
    for src, t in ((dict(gu=gu), dict(gu=dev(gu))), (dict(codes=codes, scales=scales), dict(codes=ct, scales=st))):
        dgu = torch.empty((4, 512), device="cuda")
        R.repro_swiglu_bwd(torch.ones((4, 256), device="cuda"), dgu, **t)
        same(host(dgu), orc.swiglu_bwd(np.ones((4, 256), f32), **src))


# ---------------------------------------------------------------- block norm

NORM = [(1, 1), (2, 3), (5, 4), (3, 37), (17, 128), (33, 512), (4, 513), (2, 1001), (35, 1024), (16, 2048), (50, 2048), (3, 4096),
        (2, 5000), (3, 8192), (2, 8200), (17, 16384)]


@pytest.mark.parametrize("n,D", NORM)
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gains", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("kind,u_kind", [(F32, F32), (BF, F32), (F32, BF), (BF, BF)])
def test_block_norm(orc, n, D, gate, post, gains, layout, kind, u_kind):
    norm_check(orc, n, D, gate, post, gains, layout, kind, u_kind)


# more than 2^21 elements: the backward takes chunks of tokens, not single ones
LONG = [(1030, 2048), (2100, 1001), (70000, 32), (4200, 512), (2000, 1060), (517, 4096), (300, 8192), (129, 16384)]


@pytest.mark.parametrize("n,D", LONG)
@pytest.mark.parametrize("gate,post", [(None, True), ("channel", False), ("channel", True), ("token", True)])
@pytest.mark.parametrize("kind,u_kind", [(F32, F32), (BF, F32), (F32, BF)])
def test_block_norm_chunks(orc, n, D, gate, post, kind, u_kind):
    norm_check(orc, n, D, gate, post, True, "strided", kind, u_kind)


def norm_check(orc, n, D, gate, post, gains, layout, kind, u_kind):
    c = norm_case(n, D, gate, post, gains)
    narrow = ("x", "y", "dh") + (("gate",) if gate == "token" else ())
    if kind == BF:
        c.update({k: bf(c[k]) for k in narrow})
    if u_kind == BF:
        c["du"] = bf(c["du"])
    extra, off = LAYOUTS[layout]
    rows = lambda a, t: strided(a, extra, off, t)  # noqa: E731
    blank = lambda t: strided(np.full((n, D), 5.0, f32), extra, off, t)  # noqa: E731
    opt = lambda a: None if a is None else dev(a)  # noqa: E731
    gt = None if gate is None else dev(c["gate"]) if gate == "channel" else rows(c["gate"], kind)
    kw = dict(gate=gt, g_post=opt(c["g_post"]), g_pre=opt(c["g_pre"]), post=post, alpha=0.75, beta=0.3)
    okw = dict(gate=c["gate"], g_post=c["g_post"], g_pre=c["g_pre"], post=post, alpha=0.75, beta=0.3)
    y, h, u, st = rows(c["y"], kind), blank(kind), blank(u_kind), torch.full((n, 2), 7.0, device="cuda")
    R.repro_block_norm_fwd(rows(c["x"], kind), y, h, u, stats=st, eps=1e-5, **kw)
    eh, eu, es = orc.block_norm_fwd(c["x"], c["y"], eps=1e-5, h_bf16=kind == BF, **okw)
    same(host(h.float()), eh, "h")
    same(host(u.float()), bf(eu) if u_kind == BF else eu, "u")
    same(host(st), es, "stats")
    g = rng(D)
    for accumulate in (False, True):
        old = [g.standard_normal(D).astype(f32) for _ in range(3)] if accumulate else None
        sums = [dev(o.copy()) for o in old] if accumulate else [torch.full((D,), 3.0, device="cuda") for _ in range(3)]
        dgate = None if gate is None else sums[0] if gate == "channel" else blank(kind)
        dgp, dgn = sums[1] if c["g_post"] is not None else None, sums[2] if c["g_pre"] is not None else None
        dx, dy = blank(kind), blank(kind)
        R.repro_block_norm_bwd(rows(c["dh"], kind), rows(c["du"], u_kind), h, y, st, dx, dy, dgate=dgate, dg_post=dgp,
                               dg_pre=dgn, accumulate=accumulate, **kw)
        exp = orc.block_norm_bwd(c["dh"], c["du"], eh, c["y"], es, acc=old, **okw)
        for name, t, e in zip(("dx", "dy", "dgate", "dg_post", "dg_pre"), (dx, dy, dgate, dgp, dgn), exp):
            assert (t is None) == (e is None), name
            if t is not None:
                same(host(t.float()), bf(e) if t.dtype == BF else e, name)


@pytest.mark.parametrize("n,D", [(1, 7), (40, 300), (19, 2048)])
def test_block_norm_parts(orc, n, D):
    """The norm before a block alone, h in place of x, dx in place of dh, one gradient without the
    other, no norm of h, no stats."""
    c = norm_case(n, D, None, False, True)
    gn = dev(c["g_pre"])
    x, u, st = dev(c["x"]), torch.empty((n, D), device="cuda"), torch.empty((n, 2), device="cuda")
    R.repro_block_norm_fwd(x, None, None, u, stats=st, g_pre=gn)
    _, eu, es = orc.block_norm_fwd(c["x"], g_pre=c["g_pre"])
    same(host(u), eu)
    same(host(st), es)
    dx, dgn = torch.empty((n, D), device="cuda"), torch.empty(D, device="cuda")
    R.repro_block_norm_bwd(None, dev(c["du"]), x, None, st, dx, None, g_pre=gn, dg_pre=dgn)
    e = orc.block_norm_bwd(None, c["du"], c["x"], None, es, g_pre=c["g_pre"])
    same(host(dx), e[0])
    same(host(dgn), e[4])
    y = dev(c["y"])
    R.repro_block_norm_fwd(x, y, x, None, alpha=0.5, beta=2.0, post=True)
    eh = orc.block_norm_fwd(c["x"], c["y"], alpha=0.5, beta=2.0, post=True, want_u=False)[0]
    same(host(x), eh)
    dh, dy = dev(c["dh"]), torch.empty((n, D), device="cuda")
    es = orc.block_norm_fwd(c["x"], c["y"], alpha=0.5, beta=2.0, post=True)[2]
    R.repro_block_norm_bwd(dh, None, None, y, dev(es), dh, dy, alpha=0.5, beta=2.0, post=True)
    e = orc.block_norm_bwd(c["dh"], None, None, c["y"], es, alpha=0.5, beta=2.0, post=True)
    same(host(dh), e[0])
    same(host(dy), e[1])


def test_block_norm_unordinary(orc):
    """Subnormals, infinities and NaN as the operations give them, row by row."""
    n, D = 6, 200
    c = norm_case(n, D, "token", True, True)
    c["x"][0, 3], c["y"][2, 5], c["y"][3, 0] = np.inf, np.nan, -np.inf
    c["x"][4], c["y"][4] = 1e-41, 1e-40
    c["du"][5, 7], c["dh"][5, 8] = 1e-42, np.inf
    okw = dict(gate=c["gate"], g_post=c["g_post"], g_pre=c["g_pre"], post=True)
    kw = {k: dev(v) if isinstance(v, np.ndarray) else v for k, v in okw.items()}
    h, u, st = (torch.empty((n, k), device="cuda") for k in (D, D, 2))
    y = dev(c["y"])
    R.repro_block_norm_fwd(dev(c["x"]), y, h, u, stats=st, **kw)
    eh, eu, es = orc.block_norm_fwd(c["x"], c["y"], **okw)
    for t, e in ((h, eh), (u, eu), (st, es)):
        same(host(t), e)
    out = [torch.empty((n, D), device="cuda") for _ in range(3)] + [torch.empty(D, device="cuda") for _ in range(2)]
    R.repro_block_norm_bwd(dev(c["dh"]), dev(c["du"]), h, y, st, out[0], out[1], dgate=out[2], dg_post=out[3], dg_pre=out[4], **kw)
    for t, e in zip(out, orc.block_norm_bwd(c["dh"], c["du"], eh, c["y"], es, **okw)):
        same(host(t), e)


def test_block_norm_no_rows():
    none = torch.empty((0, 64), device="cuda")
    R.repro_block_norm_fwd(none, None, None, none)
    st, g = torch.empty((0, 2), device="cuda"), torch.ones(64, device="cuda")
    for accumulate, want in ((True, 5.0), (False, 0.0)):
        dg = torch.full((64,), 5.0, device="cuda")
        R.repro_block_norm_bwd(None, none, none, None, st, none, None, g_pre=g, dg_pre=dg, accumulate=accumulate)
        assert (host(dg) == want).all()


# ---------------------------------------------------------------- product of codes

MM = [(1, 1, 1), (1, 5, 16), (1, 130, 5632), (3, 7, 100), (8, 64, 512), (9, 33, 513), (16, 100, 1000), (17, 5, 8), (64, 64, 64),
      (65, 300, 77), (128, 256, 512), (129, 257, 520), (200, 70, 2049), (256, 256, 1024), (300, 520, 640), (700, 260, 96), (5, 130, 528), (33, 300, 1040),
      (100, 129, 2064), (64, 128, 16), (128, 1000, 5632)]


def codes(g, *shape):
    return g.integers(-127, 128, shape).astype(np.int8)


def mm_case(M, N, K, seed=0):
    g = rng(M + N + K + seed)
    a, b = codes(g, M, K), codes(g, N, K)
    a[M // 2], b[N // 3] = 127, 127                       # sums as large as they get
    if N > 1:
        b[0] = -127
    return a, b, (0.01 + g.random(M)).astype(f32), (0.001 + g.random(N)).astype(f32)


def mm_check(orc, M, N, K, a_t, b_t, layout="dense", kind=F32, accumulate=False, scales=True):
    a, b, sa, sb = mm_case(M, N, K)
    extra, off = LAYOUTS[layout]
    at, bt = (np.ascontiguousarray(v.T) if t else v for v, t in ((a, a_t), (b, b_t)))
    old = rng(M).standard_normal((M, N)).astype(f32)
    y = strided(old, extra, off, kind)
    sa, sb = (sa, sb) if scales else (None, None)
    R.repro_matmul_i8(strided(at, extra, off, torch.int8), strided(bt, extra, off, torch.int8), y,
                      None if sa is None else dev(sa), None if sb is None else dev(sb), a_t, b_t, accumulate)
    e = orc.matmul_i8(at, bt, sa, sb, a_t, b_t, old if accumulate else None)
    same(host(y.float()), bf(e) if kind == BF else e)


@pytest.mark.parametrize("M,N,K", MM)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("a_t,b_t", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("path", [0, -1])
def test_matmul(orc, M, N, K, layout, a_t, b_t, path):
    R.repro_set_launch_cfg(fwd_path=path)
    try:
        mm_check(orc, M, N, K, a_t, b_t, layout, F32, False)
        mm_check(orc, M, N, K, a_t, b_t, layout, F32, True)
        mm_check(orc, M, N, K, a_t, b_t, layout, BF, False, scales=False)
    finally:
        R.repro_set_launch_cfg(reset=True)
    assert R.repro_device_check() == R.REPRO_OK


def test_matmul_no_terms():
    for M in (3, 40):
        a, b = (torch.empty((n, 0), dtype=torch.int8, device="cuda") for n in (M, 5))
        y = torch.full((M, 5), 4.0, device="cuda")
        R.repro_matmul_i8(a, b, y, accumulate=True)
        assert (host(y) == 4).all()
        R.repro_matmul_i8(a, b, y)
        assert not host(y).any()


def test_matmul_accumulates_subnormals(orc):
    """Old values and sums below the smallest normal are flushed, however the addition is done."""
    tiny = f32(2.0) ** -126
    for M in (4, 64, 200):
        a, b = np.ones((M, 8), np.int8), np.ones((64, 8), np.int8)
        sa = np.full(M, tiny / 8 * f32(1.5), f32)
        sa[1], sa[2] = -tiny, tiny
        sa = np.where(np.abs(sa) < tiny, tiny * f32(1.25), sa).astype(f32)
        sb = np.where(np.arange(64) % 2, f32(0.125), f32(0.0625))
        old = np.tile(f32([-tiny, 0.75 * tiny, 1.0, -1.5 * tiny]), (M, 16))
        y = dev(old.copy())
        R.repro_matmul_i8(dev(a), dev(b), y, dev(sa), dev(sb), accumulate=True)
        same(host(y), orc.matmul_i8(a, b, sa, sb, acc=old))


@pytest.mark.parametrize("K", [512, 1024, 4096, 133144])
def test_matmul_at_the_clamp(K):
    """Sums at the ends of the range, in every column of two tiles, against exact integers."""
    for M, N in ((257, 520), (100, 260)):
        clamp_check(M, N, K)


def clamp_check(M, N, K):
    g = rng(K)
    a, b = codes(g, M, K), codes(g, N, K)
    a[::5], a[1::5] = 127, -127
    b[::3], b[1::3] = 127, -127
    a[2, ::2], a[2, 1::2] = 127, -127
    a[3, 511::512] = 1
    at, bt = dev(a), dev(b)
    y = torch.empty((M, N), device="cuda")
    R.repro_matmul_i8(at, bt, y)
    exact = (at.double() @ bt.double().T).cpu().numpy()   # below 2^53: exact in any order
    assert np.array_equal(host(y), exact.astype(f32))


def test_matmul_many_tiles(orc):
    """More tiles than pairs of SMs, over ragged edges, both signs of every code; a sample of rows."""
    M, N, K = 5000, 5003, 1160
    a, b, sa, sb = mm_case(M, N, K)
    y = torch.empty((M, N), device="cuda")
    R.repro_matmul_i8(dev(a), dev(b), y, dev(sa), dev(sb))
    acc = (dev(a).double() @ dev(b).double().T).cpu().numpy()
    e = acc.astype(f32) * sa[:, None] * sb
    same(host(y), e)
    assert R.repro_device_check() == R.REPRO_OK


@pytest.mark.parametrize("hook", [dict(fwd_path=0), dict(fwd_selftest=1), dict(fwd_path=1)])
def test_matmul_paths_agree(hook):
    a, b, sa, sb = mm_case(300, 260, 700)
    out = []
    for cfg in ({}, hook):
        R.repro_set_launch_cfg(**cfg)
        y = torch.empty((300, 260), device="cuda")
        R.repro_matmul_i8(dev(a), dev(b), y, dev(sa), dev(sb))
        out.append(host(y))
        R.repro_set_launch_cfg(reset=True)
    same(out[0], out[1])
    R.repro_device_check()                                  # takes the forced failure's report


def test_swiglu_reciprocals(orc):
    """sig(g) over 4 million gates of every size: e^-|g| takes values all over (0, 1], and with it the
    reciprocal of 1 + e."""
    g = rng(21)
    gate = np.concatenate([g.uniform(-20, 20, 1 << 21), g.uniform(-1, 1, 1 << 20),
                           10.0 ** g.uniform(-12, 2, 1 << 20) * g.choice([-1, 1], 1 << 20)]).astype(f32)
    gu = np.stack([gate.reshape(-1, 1024), np.ones((gate.size // 1024, 1024), f32)], 1).reshape(-1, 2048)
    a, dgu = torch.empty((gu.shape[0], 1024), device="cuda"), torch.empty(gu.shape, device="cuda")
    R.repro_swiglu_fwd(dev(gu), a)
    same(host(a), orc.swiglu_fwd(gu)[0])
    R.repro_swiglu_bwd(torch.ones_like(a), dgu, gu=dev(gu))
    same(host(dgu), orc.swiglu_bwd(np.ones(a.shape, f32), gu=gu))


# ---------------------------------------------------------------- alignment and far offsets

def test_floats_on_four_bytes(orc):
    """Statistics, gains, gates and scales need their own type's alignment only."""
    n, D = 9, 64
    c = norm_case(n, D, "channel", True, True)
    off = lambda a: strided(np.asarray(a, f32).reshape(1, -1), 0, 1)[0] if a.ndim == 1 else strided(a, 0, 1)  # noqa: E731
    kw = dict(gate=off(c["gate"]), g_post=off(c["g_post"]), g_pre=off(c["g_pre"]), post=True)
    okw = dict(gate=c["gate"], g_post=c["g_post"], g_pre=c["g_pre"], post=True)
    h, u, st = (off(np.zeros((n, k), f32)) for k in (D, D, 2))
    R.repro_block_norm_fwd(dev(c["x"]), dev(c["y"]), h, u, stats=st, **kw)
    eh, eu, es = orc.block_norm_fwd(c["x"], c["y"], **okw)
    for t, e in ((h, eh), (u, eu), (st, es)):
        same(host(t), e)
    out = [off(np.zeros((n, D), f32)) for _ in range(2)] + [off(np.zeros(D, f32)) for _ in range(3)]
    R.repro_block_norm_bwd(dev(c["dh"]), dev(c["du"]), dev(eh), dev(c["y"]), st, out[0], out[1], dgate=out[2], dg_post=out[3],
                           dg_pre=out[4], **kw)
    for t, e in zip(out, orc.block_norm_bwd(c["dh"], c["du"], eh, c["y"], es, **okw)):
        same(host(t), e)
    a, b, sa, sb = mm_case(40, 96, 128)
    for M in (3, 40):
        y = off(np.zeros((M, 96), f32))
        R.repro_matmul_i8(dev(a[:M]), dev(b), y, off(sa[:M]), off(sb))
        same(host(y), orc.matmul_i8(a[:M], b, sa[:M], sb))
    gu = rng(1).standard_normal((5, 256)).astype(f32)
    ea, codes_, scales = orc.swiglu_fwd(gu)
    av, ct, sv = off(np.zeros((5, 128), f32)), torch.empty((5, 2, 1, 128), dtype=torch.int8, device="cuda"), off(np.zeros(10, f32))
    R.repro_swiglu_fwd(off(gu), av, ct, sv)
    same(host(av), ea)
    same(host(sv), scales.ravel())
    dgu = off(np.zeros((5, 256), f32))
    R.repro_swiglu_bwd(av, dgu, codes=ct, scales=sv)
    same(host(dgu), orc.swiglu_bwd(ea, codes=codes_, scales=scales))


def test_lowest_codes(orc):
    """-128, which no quantiser gives: its sums are exact too."""
    for M, N, K in ((3, 70, 1024), (40, 200, 1536), (300, 260, 2048)):
        a, b = np.full((M, K), -128, np.int8), np.full((N, K), -128, np.int8)
        a[1], b[1] = 127, 127
        b[2, ::3] = 1
        y = torch.empty((M, N), device="cuda")
        R.repro_matmul_i8(dev(a), dev(b), y)
        same(host(y), (a.astype(np.int64) @ b.astype(np.int64).T).astype(f32))


def far(rows, width, dtype, seed):
    """[rows, width] of more than 2^31 elements: one block of rows over and over, the last ones new."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty((rows, width), dtype=dtype, device="cuda")
    head = torch.randn((1000, width), generator=g, device="cuda").to(dtype)
    for lo in range(0, rows, 1000):
        t[lo:lo + 1000] = head[:min(1000, rows - lo)]
    t[-7:] = torch.randn((7, width), generator=g, device="cuda").to(dtype)
    return t


def test_offsets_past_32_bits():
    """The last rows of tensors of more than 2^31 elements, against the same rows by themselves."""
    n, D = 270000, 8192
    x, y = far(n, D, BF, 1), far(n, D, BF, 2)
    h, u, st = torch.empty_like(x), torch.empty_like(x), torch.empty((n, 2), device="cuda")
    gain = torch.linspace(0.5, 1.5, D, device="cuda")
    R.repro_block_norm_fwd(x, y, h, u, stats=st, g_post=gain, g_pre=gain, post=True)
    t = slice(n - 9, n)
    h2, u2, st2 = torch.empty((9, D), dtype=BF, device="cuda"), torch.empty((9, D), dtype=BF, device="cuda"), torch.empty((9, 2), device="cuda")
    R.repro_block_norm_fwd(x[t], y[t], h2, u2, stats=st2, g_post=gain, g_pre=gain, post=True)
    assert torch.equal(h[t], h2) and torch.equal(u[t], u2) and torch.equal(st[t], st2)
    dx, dy, dg = x, torch.empty_like(x), torch.empty(D, device="cuda")   # x is done with
    R.repro_block_norm_bwd(None, u, h, y, st, dx, dy, g_post=gain, g_pre=gain, dg_post=dg, dg_pre=torch.empty_like(dg), post=True)
    dx2, dy2 = torch.empty_like(h2), torch.empty_like(h2)
    R.repro_block_norm_bwd(None, u[t], h2, y[t], st2, dx2, dy2, g_post=gain, g_pre=gain, dg_post=dg, dg_pre=torch.empty_like(dg),
                           post=True)
    assert torch.equal(dx[t], dx2) and torch.equal(dy[t], dy2)
    del x, y, u, dx, dy
    q, s = torch.empty((n, D), dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    R.repro_quant_rows_i8(h, q, s)
    q2, s2 = torch.empty((9, D), dtype=torch.int8, device="cuda"), torch.empty(9, device="cuda")
    R.repro_quant_rows_i8(h[t], q2, s2)
    assert torch.equal(q[t], q2) and torch.equal(s[t], s2)
    c = torch.empty(D, device="cuda")
    R.repro_quant_rows_i8(h, q, c, columns=True)
    assert torch.equal(c, h.abs().amax(0).float() / torch.full((1,), 127.0, device="cuda"))
    assert int((q[-7:].float() - (h[-7:].float() / c).round()).abs().max()) == 0
    a, codes_, sc = torch.empty((n, D // 2), dtype=BF, device="cuda"), q.view(n, 2, D // 256, 128), torch.empty((n, 2, D // 256), device="cuda")
    R.repro_swiglu_fwd(h, a, codes_, sc)
    a2, codes2, sc2 = torch.empty((9, D // 2), dtype=BF, device="cuda"), torch.empty((9, 2, D // 256, 128), dtype=torch.int8, device="cuda"), torch.empty((9, 2, D // 256), device="cuda")
    R.repro_swiglu_fwd(h[t], a2, codes2, sc2)
    assert torch.equal(a[t], a2) and torch.equal(codes_[t], codes2) and torch.equal(sc[t], sc2)
    dgu, dgu2 = torch.empty_like(h), torch.empty_like(h2)
    R.repro_swiglu_bwd(a, dgu, codes=codes_, scales=sc)
    R.repro_swiglu_bwd(a2, dgu2, codes=codes2, scales=sc2)
    assert torch.equal(dgu[t], dgu2)
    del a, codes_, sc, dgu, q, h
    M, N, K = 60000, 40000, 96
    g = torch.Generator(device="cuda").manual_seed(5)
    am, bm = (torch.randint(-127, 128, (r, K), generator=g, device="cuda", dtype=torch.int8) for r in (M, N))
    ym = torch.empty((M, N), device="cuda")
    R.repro_matmul_i8(am, bm, ym)
    assert torch.equal(ym[-300:], (am[-300:].double() @ bm.double().T).float())
    assert R.repro_device_check() == R.REPRO_OK


def test_wide_rows_and_many_columns(orc):
    """Codes of rows past what a thread keeps, and of a wide matrix by columns, in odd widths."""
    g = rng(9)
    for n, D in ((2, 40001), (3, 65536), (900, 5001)):
        x = g.standard_normal((n, D)).astype(f32)
        for columns in (False, True):
            q, s = torch.empty((n, D), dtype=torch.int8, device="cuda"), torch.empty(D if columns else n, device="cuda")
            R.repro_quant_rows_i8(dev(x), q, s, columns=columns)
            eq, es = orc.quant_rows(x, None, columns)
            same(host(s), es)
            assert np.array_equal(host(q), eq)
