"""GPU: the embedding, the per-head norm with rotation and the distillation loss,
bit for bit against the oracle over their types, widths, strides, masks and
lengths, and within counted roundings of 64-bit plain forms."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import bitwise_reproducible_int8_gb300 as R  # noqa: E402
import ops64 as F  # noqa: E402
from gpu_helpers import assert_bits_equal, dev, host  # noqa: E402
from test_oracle_blocks import HP, case as distill_case, rope_table  # noqa: E402

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
rng = np.random.default_rng


def bf(a):
    """float32 array rounded to bf16, as float32."""
    return torch.from_numpy(np.ascontiguousarray(a)).to(BF).float().numpy()


def strided(a, extra=0, offset=0, dtype=torch.float32):
    """A device copy of matrix a with rows a.shape[1] + extra apart, `offset`
    elements past an aligned start; what surrounds it is NaN."""
    n, D = a.shape
    buf = torch.full((offset + n * (D + extra) + 8,), float("nan"), device="cuda").to(dtype) \
        if dtype.is_floating_point else torch.full((offset + n * (D + extra) + 8,), 77, device="cuda", dtype=dtype)
    v = buf[offset:offset + n * (D + extra)].view(n, D + extra)[:, :D]
    v.copy_(torch.from_numpy(np.ascontiguousarray(a)).to(dtype))
    return v


def same(got, exp, what=""):
    """Equal bits; NaNs need only be NaNs."""
    got, exp = np.asarray(got), np.asarray(exp)
    nan = np.isnan(exp)
    assert np.array_equal(np.isnan(got), nan), what
    assert_bits_equal(np.where(nan, np.float32(0), got), np.where(nan, np.float32(0), exp), what)


# ---------------------------------------------------------------- embedding

@pytest.mark.parametrize("n,V,D", [(1, 1, 1), (1, 7, 2048), (5, 3, 3), (65, 50, 512), (300, 1000, 130), (33, 9, 1001),
                                   (2000, 4000, 516)])
@pytest.mark.parametrize("table", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("layout", ["dense", "strided", "odd"])
def test_embed_fwd(orc, n, V, D, table, layout):
    g = rng(n * D + V)
    tok = g.integers(0, V, n)
    pad = int(tok[-1])
    extra, off = {"dense": (0, 0), "strided": (8, 0), "odd": (3, 1)}[layout]
    s_w = None
    if table == "i8":
        W = g.integers(-127, 128, (V, D)).astype(np.int8)
        s_w = np.float32(0.0127)
        Wt = strided(W, extra, off, torch.int8)
    else:
        W = (g.standard_normal((V, D)) * 0.02).astype(np.float32)
        W[0, 0] = np.float32(1e-41)                        # read as zero
        W = bf(W) if table == "bf16" else W
        Wt = strided(W, extra, off, BF if table == "bf16" else torch.float32)
    exp = orc.embed_fwd(W, tok, 31.6, s_w, pad)
    for out_t in (torch.float32, BF):
        out = strided(np.zeros((n, D), dtype=np.float32), extra, off, out_t)
        tk = dev(tok.astype(np.int32 if n % 2 else np.int64))
        R.repro_embed_fwd(Wt, tk, out, scale=31.6, s_w=None if s_w is None else dev(np.float32([s_w])), pad=pad)
        same(host(out.float()), exp if out_t == torch.float32 else bf(exp))
    exp64 = F.embed_fwd(W, tok, 31.6, s_w, pad)
    assert np.all(np.abs(exp - exp64) <= 2.01 * F.U * np.abs(exp64) + 1e-37)


@pytest.mark.parametrize("n,V,D", [(0, 5, 4), (1, 1, 1), (3, 70000, 5), (63, 1, 4), (64, 1, 130), (65, 1, 7), (129, 2, 260),
                                   (300, 1000, 130), (5000, 1, 33), (20000, 3000, 20), (4097, 300, 1001), (1000, 256, 64),
                                   (1000, 65536, 12), (9000, 66000, 8)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "odd"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_bwd(orc, n, V, D, kind, accumulate):
    g = rng(n + D + V)
    p = 1.0 / (np.arange(V) + 2.0)
    tok = g.permutation(V)[g.choice(V, n, p=p / p.sum())] if n else np.zeros(0, dtype=np.int64)
    pad = int(tok[n // 2]) if n > 200 and V > 1 else -1
    d = (g.standard_normal((n, D)) * 1e-3).astype(np.float32)
    d = bf(d) if kind == "bf16" else d
    extra, off = (3, 1) if kind == "odd" else (0, 0)
    acc = g.standard_normal((V, D)).astype(np.float32) if accumulate else None
    dW = strided(np.full((V, D), 5.0, dtype=np.float32) if acc is None else acc, extra, off)
    dt = strided(d, extra, off, BF if kind == "bf16" else torch.float32)
    tk = dev(tok.astype(np.int64 if n % 2 else np.int32))
    R.repro_embed_bwd(dt, tk, dW, scale=0.37, pad=pad, accumulate=accumulate)
    exp = orc.embed_bwd(d, tok, V, 0.37, pad, acc)
    same(host(dW), exp)
    assert R.repro_device_check() == 0
    if n * D < 200000 and n:
        e64, bound = F.embed_bwd(d, tok, V, 0.37, pad, acc)
        assert np.all(np.abs(host(dW) - e64) <= bound)


@pytest.mark.parametrize("D", [8, 5])
def test_embed_bwd_subnormals(orc, D):
    """Old values, sums and results below the smallest normal are flushed, however
    the addition into the table is done."""
    tiny = np.float32(2.0 ** -126)
    d = np.tile(np.float32([1.5 * tiny, -1.25 * tiny, 0.5 * tiny, 3.0]), (6, 2))[:, :D]
    tok = np.array([0, 1, 1, 2, 3, 4])
    acc = np.zeros((6, D), dtype=np.float32)
    acc[0] = -1.25 * tiny
    acc[1] = 0.75 * tiny
    acc[2] = 1.0
    acc[3] = -1.5 * tiny
    for scale in (1.0, 0.25):
        dW = dev(acc.copy())
        R.repro_embed_bwd(dev(d), dev(tok), dW, scale=scale, accumulate=True)
        same(host(dW), orc.embed_bwd(d, tok, 6, scale, -1, acc))


def test_embed_out_of_range_tokens(orc):
    g = rng(1)
    W, d = g.standard_normal((10, 36)).astype(np.float32), g.standard_normal((5, 36)).astype(np.float32)
    for bad in (10, 1 << 40, -2):
        tok = np.array([3, bad, 9, -1, 3])
        out = torch.full((5, 36), 9.0, device="cuda")
        R.repro_embed_fwd(dev(W), dev(tok), out)
        assert R.repro_device_check() == R.REPRO_ERR_INDEX and R.repro_device_check() == 0
        same(host(out), orc.embed_fwd(W, tok))
        dW = torch.full((10, 36), 9.0, device="cuda")
        R.repro_embed_bwd(dev(d), dev(tok), dW)
        assert R.repro_device_check() == R.REPRO_ERR_INDEX
        same(host(dW), orc.embed_bwd(d, tok, 10))


# ---------------------------------------------------------------- norm and rotation

QK = [(1, 1, 1, 1, 0), (3, 2, 1, 2, 2), (5, 3, 3, 6, 4), (4, 4, 2, 32, 32), (7, 2, 1, 33, 10), (9, 8, 2, 64, 64),
      (3, 5, 1, 80, 40), (130, 3, 1, 96, 96), (50, 16, 4, 128, 128), (11, 4, 4, 128, 40), (6, 2, 2, 130, 130),
      (10, 3, 1, 192, 64), (4, 2, 1, 256, 256), (3, 2, 2, 300, 300), (2, 1, 1, 512, 512), (70, 1, 0, 128, 128)]


@pytest.mark.parametrize("n,Hq,Hkv,D,R_", QK)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("kind", ["f32", "bf16", "odd"])
@pytest.mark.parametrize("with_gain", [False, True])
def test_qk_norm_rope(orc, n, Hq, Hkv, D, R_, inter, kind, with_gain):
    g = rng(n + D)
    H = Hq + 2 * Hkv
    x = (1.3 * g.standard_normal((n, H * D))).astype(np.float32)
    x[0, :D] = 0.0
    x = bf(x) if kind == "bf16" else x
    dt = BF if kind == "bf16" else torch.float32
    extra, off = (3, 1) if kind == "odd" else (0, 0)
    xt = strided(x, extra, off, dt)
    ld = xt.stride(0)

    def heads(t, lo, h):
        return t.as_strided((n, h, D), (ld, D, 1), t.storage_offset() + lo * D)

    xs = x.reshape(n, H, D)
    P = 300
    rope, pos = rope_table(P, R_), g.integers(0, P, n).astype(np.int32)
    gains = [(1 + 0.1 * g.standard_normal(D)).astype(np.float32) if with_gain else None for _ in range(2)]
    tg = [None if v is None else dev(v) for v in gains]
    q, k = heads(xt, 0, Hq), heads(xt, Hq, Hkv) if Hkv else None
    qo = torch.full((n, Hq, D), 7.0, device="cuda")
    ko = torch.full((n, Hkv, D), 7.0, device="cuda") if Hkv else None
    rt = dev(rope) if R_ else None
    kw = dict(g_q=tg[0], g_k=tg[1] if Hkv else None, positions=dev(pos), eps=1e-5, interleaved=inter)
    R.repro_qk_norm_rope_fwd(q, k, rt, qo, ko, **kw)
    part = {"q": (0, Hq, gains[0]), "k": (Hq, Hkv, gains[1])}
    for nm, o in (("q", qo), ("k", ko)):
        if o is None:
            continue
        lo, h, gain = part[nm]
        same(host(o), orc.qk_fwd(xs[:, lo:lo + h], rope, pos, gain, 1e-5, inter), nm)
        exp, bound = F.qk_fwd(xs[:, lo:lo + h], rope, pos, gain, 1e-5, inter)
        assert np.all(np.abs(host(o) - exp) <= bound)
    # backward, into the gradient of the fused row
    dxt = strided(np.full((n, H * D), 3.0, dtype=np.float32), extra, off, dt)
    dq, dk = heads(dxt, 0, Hq), heads(dxt, Hq, Hkv) if Hkv else None
    do = {nm: (1e-3 * g.standard_normal((n, h, D))).astype(np.float32) for nm, (_, h, _) in part.items()}
    acc = [g.standard_normal(D).astype(np.float32) for _ in range(2)]
    for accumulate in (False, True):
        dg = [dev(a.copy()) if with_gain else None for a in acc]
        if not Hkv:
            dg[1] = None
        R.repro_qk_norm_rope_bwd(dev(do["q"]), dev(do["k"]) if Hkv else None, q, k, rt, dq, dk, dg_q=dg[0], dg_k=dg[1],
                                 accumulate=accumulate, **kw)
        for i, (nm, t) in enumerate((("q", dq), ("k", dk))):
            if t is None:
                continue
            lo, h, gain = part[nm]
            dx, eg = orc.qk_bwd(do[nm], xs[:, lo:lo + h], rope, pos, gain, 1e-5, inter, acc[i] if accumulate else None)
            same(host(t.float()), bf(dx) if kind == "bf16" else dx, "d" + nm)
            if with_gain:
                same(host(dg[i]), eg, "dg_" + nm)
            if not accumulate:
                ex, bx, e2, bg = F.qk_bwd(do[nm], xs[:, lo:lo + h], rope, pos, gain, 1e-5, inter)
                assert np.all(np.abs(dx - ex) <= bx + 1e-37)
                if with_gain:
                    assert np.all(np.abs(host(dg[i]) - e2) <= bg + 1e-37)
    v = host(dxt.float()).reshape(n, H, D)[:, Hq + Hkv:]
    assert np.all(v == 3.0)                                # the values' gradient is not touched
    assert R.repro_device_check() == 0


@pytest.mark.parametrize("with_gain", [False, True])
def test_qk_positions(orc, with_gain):
    """Positions left out count within the sequence; out-of-range ones are
    reported and give zero rows and terms; head strides beyond the width."""
    g = rng(5)
    B, T, H, D = 2, 37, 3, 64
    rope = rope_table(T, D)
    wide = torch.randn(B, T, H, D + 4, device="cuda")
    q = wide[..., :D]
    x = host(q).reshape(B * T, H, D)
    gain = (1 + 0.1 * g.standard_normal(D)).astype(np.float32) if with_gain else None
    gt = None if gain is None else dev(gain)
    out = torch.empty(B, T, H, D, device="cuda")
    R.repro_qk_norm_rope_fwd(q, None, dev(rope), out, None, g_q=gt)
    pos = np.tile(np.arange(T, dtype=np.int32), B)
    same(host(out).reshape(-1, H, D), orc.qk_fwd(x, rope, pos, gain))
    do = g.standard_normal((B * T, H, D)).astype(np.float32)
    for bad in (T, -1):
        pos[5] = pos[70] = bad
        R.repro_qk_norm_rope_fwd(q, None, dev(rope), out, None, g_q=gt, positions=dev(pos))
        assert R.repro_device_check() == R.REPRO_ERR_INDEX
        same(host(out).reshape(-1, H, D), orc.qk_fwd(x, rope, pos, gain))
        dq, dg = torch.empty(B, T, H, D, device="cuda"), torch.empty(D, device="cuda") if with_gain else None
        R.repro_qk_norm_rope_bwd(dev(do), None, q, None, dev(rope), dq, None, g_q=gt, dg_q=dg, positions=dev(pos))
        assert R.repro_device_check() == R.REPRO_ERR_INDEX
        dx, eg = orc.qk_bwd(do, x, rope, pos, gain)
        same(host(dq).reshape(-1, H, D), dx)
        if with_gain:
            same(host(dg), eg)


def test_qk_no_tokens():
    dg = torch.full((64,), 3.0, device="cuda")
    e = torch.empty(0, 2, 64, device="cuda")
    R.repro_qk_norm_rope_bwd(e, None, e, None, None, e, None, g_q=dg.clone(), dg_q=dg)
    assert torch.all(dg == 0)


# ---------------------------------------------------------------- distillation

def run_distill(z, idx, tl, lab, g, hp, zt, t_dtype=torch.float32, int_t=np.int32, in_place=False):
    """(loss, stats, gradient) from the device."""
    n, V = z.shape
    K = idx.shape[1]
    loss, stats = torch.empty(n, device="cuda"), torch.empty((n, R.REPRO_DISTILL_STATS + K), device="cuda")
    it, lt = dev(idx.astype(int_t)), dev(lab.astype(int_t))
    R.repro_distill_fwd(zt, it, dev(tl).to(t_dtype), loss, stats, labels=lt, **hp)
    dz = zt if in_place else torch.empty(zt.shape, dtype=zt.dtype, device="cuda")
    R.repro_distill_bwd(zt, it, stats, dev(g), dz, labels=lt, **hp)
    return host(loss), host(stats), host(dz.float())


@pytest.mark.parametrize("n,V,K", [(1, 1, 1), (3, 31, 0), (5, 130, 7), (2, 1023, 33), (4, 1024, 40), (3, 1025, 64),
                                   (7, 5001, 100), (2, 70000, 64), (3, 300, 200), (2, 9000, 300)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "odd", "odd16"])
@pytest.mark.parametrize("hp", HP)
def test_distill(orc, n, V, K, kind, hp):
    z, idx, tl, lab = distill_case(V, n, V, K)
    if hp.get("logprobs"):
        tl = (tl - 6).astype(np.float32)
    wide = kind in ("f32", "odd")
    if not wide:
        z, tl = bf(z), bf(tl)
    zt = strided(z, *((3, 1) if kind.startswith("odd") else (0, 0)), torch.float32 if wide else BF)
    g = (rng(K).standard_normal(1 if K % 2 else n)).astype(np.float32)
    full = dict(tau=1.0, w_kd=1.0, w_ce=0.0, w_z=0.0)
    full.update(hp)
    el, es = orc.distill_fwd(z, idx, tl, lab, **full)
    back = {k: v for k, v in full.items() if k != "logprobs"}
    ez = orc.distill_bwd(z, idx, es, g, lab, **back)
    loss, stats, dz = run_distill(z, idx, tl, lab, g, hp, zt, torch.float32 if wide else BF,
                                  np.int64 if kind == "odd" else np.int32)
    same(stats, es, "stats")
    same(loss, el, "loss")
    same(dz, ez if wide else bf(ez), "dz")
    l64, lb, z64, zb = F.distill_rows(z, idx, tl, lab, **{"logprobs": False, **full})
    assert np.all(np.abs(loss - l64) <= lb)
    gg = np.broadcast_to(g, n)[:, None].astype(np.float64)
    assert np.all(np.abs(ez - z64 * gg) <= (zb + 4 * F.U * np.abs(z64)) * np.abs(gg))
    # in place, the same bits
    _, _, again = run_distill(z, idx, tl, lab, g, hp, zt, torch.float32 if wide else BF,
                              np.int64 if kind == "odd" else np.int32, in_place=True)
    same(again, ez if wide else bf(ez), "dz in place")
    assert R.repro_device_check() == 0


@pytest.mark.parametrize("n,V,K", [(5000, 130, 7), (2500, 3100, 20), (2300, 9001, 20)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("hp", [dict(), dict(tau=2.0, w_kd=0.7, w_ce=0.3), dict(tau=1.5, w_kd=0.7, w_z=1e-3)])
def test_distill_many_rows(orc, n, V, K, kind, hp):
    """Rows enough for a CTA to own its rows, and for several blocks a warp."""
    z, idx, tl, lab = distill_case(V, n, V, K)
    z = bf(z) if kind == "bf16" else z
    g = np.float32([0.01])
    full = dict(tau=1.0, w_kd=1.0, w_ce=0.0, w_z=0.0)
    full.update(hp)
    el, es = orc.distill_fwd(z, idx, tl, lab, **full)
    ez = orc.distill_bwd(z, idx, es, g, lab, **full)
    zt = strided(z, dtype=BF if kind == "bf16" else torch.float32)
    loss, stats, dz = run_distill(z, idx, tl, lab, g, hp, zt)
    same(stats, es, "stats")
    same(loss, el, "loss")
    same(dz, bf(ez) if kind == "bf16" else ez, "dz")


@pytest.mark.parametrize("tau", [1.0, 1.5, 2.0])
def test_distill_masked_rows(orc, tau):
    V, K = 3000, 4
    z, idx, tl, lab = distill_case(9, 7, V, K)
    idx[:] = np.arange(K) * 701
    lab[:] = 50
    z[0, 60:] = -np.inf                    # a block with nothing in it
    z[1] = -np.inf                         # a row with nothing in it
    z[2, 60:] = np.finfo(np.float32).min
    z[3, 2100] = np.nan
    tl[4] = -np.inf                        # a teacher without weight
    idx[5] = 701                           # one column four times
    idx[6] = -1                            # no teacher
    z[6, 7] = np.inf
    hp = dict(tau=tau, w_kd=1.0, w_ce=1.0, w_z=0.1)
    g = np.linspace(-1, 2, 7).astype(np.float32)
    el, es = orc.distill_fwd(z, idx, tl, lab, **hp)
    ez = orc.distill_bwd(z, idx, es, g, lab, **hp)
    loss, stats, dz = run_distill(z, idx, tl, lab, g, hp, dev(z))
    same(stats, es)
    same(loss, el)
    same(dz, ez)
    assert loss[1] == 0 and np.all(dz[1] == 0) and np.isnan(loss[3]) and np.all(dz[0, 60:701] == 0)
    assert R.repro_device_check() == 0


def test_distill_out_of_range(orc):
    z, idx, tl, lab = distill_case(9, 3, 500, 4)
    hp = dict(w_kd=1.0, w_ce=0.5)
    g = np.ones(3, dtype=np.float32)
    for what in ("idx", "label"):
        i2, l2 = idx.copy(), lab.copy()
        if what == "idx":
            i2[1, 2] = 500
        else:
            l2[1] = 1 << 20
        loss, stats, dz = run_distill(z, i2, tl, l2, g, hp, dev(z))
        assert R.repro_device_check() == R.REPRO_ERR_INDEX and R.repro_device_check() == 0
        el, es = orc.distill_fwd(z, i2, tl, l2, **hp)
        same(loss, el)
        same(dz, orc.distill_bwd(z, i2, es, g, l2, **hp))


# ---------------------------------------------------------------- all of them

def test_side_stream_and_debug():
    """Calls on another stream than the current one, and the debug scan of
    strided and narrow inputs."""
    s = torch.cuda.Stream()
    table = torch.randn(50, 24, device="cuda")
    tok = torch.arange(40, device="cuda") % 50
    ref = torch.empty(40, 24, device="cuda")
    R.repro_embed_fwd(table, tok, ref, scale=2.0)
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    out, dW = torch.empty(40, 24, device="cuda"), torch.empty(50, 24, device="cuda")
    ws = torch.empty(R.repro_embed_bwd_ws_bytes(40, 50, 24), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    R.repro_embed_fwd(table, tok, out, scale=2.0, stream=s)
    R.repro_embed_bwd(out, tok, dW, ws=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(dW[:40], ref) and torch.all(dW[40:] == 0)
    R.repro_set_debug(R.REPRO_DEBUG_CHECK_FINITE)
    try:
        wide = torch.zeros(30, 3, 40, device="cuda", dtype=torch.bfloat16)
        wide[:, :, 33:] = float("nan")                    # between the rows: not looked at
        q = wide[:, :, :33]
        o = torch.empty(30, 3, 33, device="cuda")
        gain = torch.ones(40, device="cuda")[1:34]        # 4-byte aligned
        R.repro_qk_norm_rope_fwd(q, None, None, o, None, g_q=gain)
        assert R.repro_device_check() == 0
        q[29, 2, 32] = float("inf")
        R.repro_qk_norm_rope_fwd(q, None, None, o, None, g_q=gain)
        assert R.repro_device_check() == R.REPRO_ERR_NONFINITE
    finally:
        R.repro_set_debug(0)


def test_nan_in_masked_places(orc):
    """What padding, empty entries and strides leave out is never read into a result."""
    g = rng(2)
    d = g.standard_normal((300, 40)).astype(np.float32)
    tok = g.integers(0, 9, 300)
    d[tok == 4] = np.nan
    dW = torch.full((9, 40), 5.0, device="cuda")
    R.repro_embed_bwd(dev(d), dev(tok), dW, pad=4)
    same(host(dW), orc.embed_bwd(np.nan_to_num(d), tok, 9, 1.0, 4))
    assert not torch.isnan(dW).any()
    W = g.standard_normal((9, 40)).astype(np.float32)
    W[4] = np.nan
    out = torch.empty(300, 40, device="cuda")
    R.repro_embed_fwd(dev(W), dev(tok), out, pad=4)
    assert not torch.isnan(out).any()
    z, idx, tl, lab = distill_case(3, 4, 700, 9)
    idx[:, 5:] = -1
    bad = tl.copy()
    bad[:, 5:] = np.nan
    hp = dict(tau=2.0, w_kd=0.5, w_ce=0.5)
    gr = np.ones(1, dtype=np.float32)
    exp = run_distill(z, idx, tl, lab, gr, hp, dev(z))
    got = run_distill(z, idx, bad, lab, gr, hp, dev(z))
    for a, b in zip(got, exp):
        same(a, b)


def test_workspace_of_another_stream():
    """A call that makes its own workspace on a stream that is not current: memory freed
    on return is not handed to the current stream's work while the call runs."""
    s = torch.cuda.Stream()
    z = torch.randn(2000, 20000, device="cuda")
    idx = torch.randint(0, 20000, (2000, 8), device="cuda")
    tl = torch.randn(2000, 8, device="cuda")
    loss, stats = torch.empty(2000, device="cuda"), torch.empty(2000, R.REPRO_DISTILL_STATS + 8, device="cuda")
    R.repro_distill_fwd(z, idx, tl, loss, stats)
    want = loss.clone()
    torch.cuda.synchronize()
    nbytes = R.repro_distill_ws_bytes(2000, 20000)
    for _ in range(5):
        loss.zero_()
        torch.cuda.synchronize()
        R.repro_distill_fwd(z, idx, tl, loss, stats, stream=s)
        junk = torch.full((nbytes,), 0xff, dtype=torch.uint8, device="cuda")
        s.synchronize()
        del junk
        assert torch.equal(loss, want)


def test_runs_repeat():
    """The same bits from run to run at a size with many chunks per token."""
    g = torch.Generator(device="cuda").manual_seed(0)
    d = torch.randn(30000, 200, device="cuda", generator=g)
    tok = torch.randint(0, 7, (30000,), device="cuda", generator=g)
    z = torch.randn(64, 33000, device="cuda", generator=g)
    idx = torch.randint(0, 33000, (64, 20), device="cuda", generator=g)
    tl = torch.randn(64, 20, device="cuda", generator=g)
    first = None
    for _ in range(3):
        dW = torch.empty(9, 200, device="cuda")
        R.repro_embed_bwd(d, tok, dW)
        loss, stats = torch.empty(64, device="cuda"), torch.empty(64, R.REPRO_DISTILL_STATS + 20, device="cuda")
        R.repro_distill_fwd(z, idx, tl, loss, stats, tau=2.0)
        dz = torch.empty_like(z)
        R.repro_distill_bwd(z, idx, stats, torch.ones(1, device="cuda"), dz, tau=2.0)
        outs = [t.cpu() for t in (dW, loss, stats, dz)]
        if first is None:
            first = outs
        assert all(torch.equal(a, b) for a, b in zip(first, outs))


# ---------------------------------------------------------------- offsets past 32 bits

def test_embed_offsets_past_32_bits():
    """1.1 M rows of 2048: the output's and the gradient's offsets pass 2^31 elements."""
    n, V, D = 1100000, 3000, 2048
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randn(V, D, device="cuda", generator=g)
    tok = torch.randint(0, V, (n,), device="cuda", generator=g)
    out = torch.empty(n, D, device="cuda")
    R.repro_embed_fwd(table, tok, out, scale=2.0)
    part = torch.empty(1000, D, device="cuda")
    R.repro_embed_fwd(table, tok[-1000:].contiguous(), part, scale=2.0)
    assert torch.equal(out[-1000:], part)
    # a token that only the last rows have: its gradient is the sum of those rows alone
    tok[tok == 7] = 8
    tok[-130:] = 7
    dW, few = torch.empty(V, D, device="cuda"), torch.empty(V, D, device="cuda")
    R.repro_embed_bwd(out, tok, dW)
    R.repro_embed_bwd(out[-130:], tok[-130:].contiguous(), few)
    assert torch.equal(dW[7], few[7])
    assert R.repro_device_check() == 0


def test_qk_offsets_past_32_bits():
    n, Hq, Hkv, D = 900000, 16, 4, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    qkv = torch.empty(n, (Hq + 2 * Hkv) * D, device="cuda", dtype=BF).normal_(generator=g)
    heads = lambda t: (t.view(-1, Hq + 2 * Hkv, D)[:, :Hq], t.view(-1, Hq + 2 * Hkv, D)[:, Hq:Hq + Hkv])  # noqa: E731
    rope = dev(rope_table(64, D))
    pos = torch.arange(n, device="cuda", dtype=torch.int32) % 64
    q, k = heads(qkv)
    qo, ko = torch.empty(n, Hq, D, device="cuda"), torch.empty(n, Hkv, D, device="cuda")
    R.repro_qk_norm_rope_fwd(q, k, rope, qo, ko, positions=pos)
    m = 500
    qs, ks = heads(qkv[-m:])
    qp, kp = torch.empty(m, Hq, D, device="cuda"), torch.empty(m, Hkv, D, device="cuda")
    R.repro_qk_norm_rope_fwd(qs, ks, rope, qp, kp, positions=pos[-m:].contiguous())
    assert torch.equal(qo[-m:], qp) and torch.equal(ko[-m:], kp)
    dqkv = torch.empty_like(qkv)
    dq, dk = heads(dqkv)
    R.repro_qk_norm_rope_bwd(qo, ko, q, k, rope, dq, dk, positions=pos)
    part = torch.empty_like(qkv[-m:])
    dqs, dks = heads(part)
    R.repro_qk_norm_rope_bwd(qp, kp, qs, ks, rope, dqs, dks, positions=pos[-m:].contiguous())
    assert torch.equal(dq[-m:], dqs) and torch.equal(dk[-m:], dks)
    assert R.repro_device_check() == 0


def test_distill_offsets_past_32_bits():
    n, V, K = 70000, 33001, 5
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.empty(n, V, device="cuda", dtype=BF).normal_(generator=g)
    idx = torch.randint(0, V, (n, K), device="cuda", generator=g)
    tl = torch.randn(n, K, device="cuda", generator=g)
    one = torch.ones(1, device="cuda")

    def run(z, idx, tl):
        loss = torch.empty(z.shape[0], device="cuda")
        stats = torch.empty(z.shape[0], R.REPRO_DISTILL_STATS + K, device="cuda")
        R.repro_distill_fwd(z, idx, tl, loss, stats, tau=2.0)
        dz = torch.empty_like(z)
        R.repro_distill_bwd(z, idx, stats, one, dz, tau=2.0)
        return loss, stats, dz

    m = 300
    whole, part = run(z, idx, tl), run(z[-m:].clone(), idx[-m:].contiguous(), tl[-m:].contiguous())
    for a, b in zip(whole, part):
        assert torch.equal(a[-m:], b)
    assert R.repro_device_check() == 0
