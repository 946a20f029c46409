"""GPU: the feed-forward calls where their forms meet -- rows on 2-element boundaries, few and many
tokens of wide rows, calls at once on two streams, captured ones on new inputs, and the debug scan of
every float input."""
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import bitwise_reproducible_int8_gb300 as R  # noqa: E402
import test_gpu_ffn as T  # noqa: E402
from gpu_helpers import dev, host  # noqa: E402
from test_gpu_blocks import same  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
rng = np.random.default_rng
f32 = np.float32


# by tokens and, from 152 chunks of 8 on (of 128 threads three times as many), by chunks
@pytest.mark.parametrize("n,D", [(9, 50), (40, 1030), (2084, 2294), (1300, 4094), (620, 7298), (600, 7298), (40, 16382), (650, 16382)])
@pytest.mark.parametrize("layout", [(2, 2), (0, 0), (6, 4)])
@pytest.mark.parametrize("gate,post", [(None, True), ("channel", True), ("token", False)])
@pytest.mark.parametrize("kind,u_kind", [(F32, F32), (BF, BF), (BF, F32)])
def test_block_norm_on_pairs(orc, monkeypatch, n, D, layout, gate, post, kind, u_kind):
    monkeypatch.setitem(T.LAYOUTS, "pairs", layout)
    T.norm_check(orc, n, D, gate, post, True, "pairs", kind, u_kind)


# rows that leave a thread one or two groups of 4, by tokens and by chunks
@pytest.mark.parametrize("n,D", [(7, 124), (7, 129), (7, 252), (7, 257), (17000, 128), (17000, 126), (9000, 256), (9000, 255), (9000, 136)])
@pytest.mark.parametrize("layout", [(0, 0), (3, 1)])
@pytest.mark.parametrize("gate,post", [(None, True), ("channel", True), ("token", False)])
@pytest.mark.parametrize("kind,u_kind", [(F32, F32), (BF, BF)])
def test_block_norm_narrow(orc, monkeypatch, n, D, layout, gate, post, kind, u_kind):
    monkeypatch.setitem(T.LAYOUTS, "narrow", layout)
    T.norm_check(orc, n, D, gate, post, True, "narrow", kind, u_kind)


def calls():
    """name -> (call, its float inputs, its outputs)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s, t=F32: torch.randn(s, generator=g, device="cuda").to(t)  # noqa: E731
    c = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    e = lambda *s, t=F32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    n, D = 50, 260
    x, y, dh, du, h = (r(n, D) for _ in range(5))
    gate, gp, gn, st = r(D), r(D), r(D), r(n, 2).abs()
    rows = r(n, D)
    out = {}

    def add(name, fn, ins, outs):
        out[name] = (fn, ins, outs)

    for name, gt, dg in (("channel", gate, e(D)), ("rows", rows, e(n, D))):
        kw = dict(gate=gt, g_post=gp, g_pre=gn, post=True)
        o = [e(n, D), e(n, D), e(n, 2)]
        add("norm_fwd_" + name, lambda s=None, kw=kw, o=o: R.repro_block_norm_fwd(x, y, o[0], o[1], stats=o[2], stream=s, **kw),
            [x, y, gt, gp, gn], o)
        o = [e(n, D), e(n, D), dg, e(D), e(D)]
        add("norm_bwd_" + name,
            lambda s=None, kw=kw, o=o: R.repro_block_norm_bwd(dh, du, h, y, st, o[0], o[1], dgate=o[2], dg_post=o[3], dg_pre=o[4],
                                                              stream=s, **kw),
            [dh, du, h, y, st, gt, gp, gn], o)
    for columns in (False, True):
        o, mul = [torch.zeros((n, D), dtype=torch.int8, device="cuda"), e(D if columns else n)], r(n if columns else D).abs()
        add("quant_%d" % columns, lambda s=None, o=o, mul=mul, columns=columns: R.repro_quant_rows_i8(x, o[0], o[1], mul=mul,
                                                                                                        columns=columns, stream=s),
            [x, mul], o)
    for M, N, K, ta, tb in ((3, 70, 528, False, False), (40, 300, 2064, False, False), (700, 1300, 2000, False, False),
                            (300, 260, 4100, True, True), (30, 40, 77, False, True)):
        a, b = c(*((K, M) if ta else (M, K))), c(*((K, N) if tb else (N, K)))
        o, sa, sb = [e(M, N)], r(M), r(N)
        add("matmul_%d" % M, lambda s=None, a=a, b=b, o=o, sa=sa, sb=sb, ta=ta, tb=tb: R.repro_matmul_i8(a, b, o[0], sa, sb, ta, tb, stream=s),
            [sa, sb], o)
    Fw = 300
    gu, da = r(n, 2 * Fw), r(n, Fw)
    o = [e(n, Fw), torch.zeros((n, 2, 3, 128), dtype=torch.int8, device="cuda"), e(n, 2, 3)]
    add("swiglu_fwd", lambda s=None, o=o: R.repro_swiglu_fwd(gu, *o, stream=s), [gu], o)
    codes, scales = c(n, 2, 3, 128), r(n, 2, 3).abs()
    o1, o2 = [e(n, 2 * Fw)], [e(n, 2 * Fw)]
    add("swiglu_bwd", lambda s=None, o=o1: R.repro_swiglu_bwd(da, o[0], gu=gu, stream=s), [da, gu], o1)
    add("swiglu_bwd_kept", lambda s=None, o=o2: R.repro_swiglu_bwd(da, o[0], codes=codes, scales=scales, stream=s), [da, scales], o2)
    return out


def test_codes_near_a_half_s_last_place(orc):
    """Quotients next to where the rounded one stops being a tie: k + 1/2 +- half a last place.  v = V and
    s = S as whole numbers leave V 2^24 - S f = n, f = (2 k + 1) 2^(23 - E) +- 1 odd, so each small n has one S;
    of those, the scales that a maximum by 127 gives."""
    tops, vals = [], []
    for k in range(127):
        E = -1 if k == 0 else (2 * k + 1).bit_length() - 2
        for sign in (-1, 1):
            f = (2 * k + 1) * 2 ** (23 - E) + sign
            inv = pow(f, -1, 1 << 24)
            for n in range(-40, 41):
                S = -n * inv % (1 << 24)
                if S < 1 << 23:
                    continue
                s = f32(S * 2.0 ** -23)
                near = np.spacing(f32(127 * s)) * np.arange(-2, 3, dtype=f32) + f32(127 * s)
                m = near[near / f32(127) == s]
                if m.size:
                    v = f32((k + 0.5 + sign * 2.0 ** (E - 24)) * float(s))
                    tops.append(m[0])
                    vals.append(v + np.spacing(v) * np.arange(-3, 4, dtype=f32))
    x = np.concatenate([f32(tops)[:, None], f32(vals)], 1)
    x[::2, 1:] *= -1
    assert x.shape[0] > 5000
    x *= (2.0 ** rng(1).integers(-30, 31, (x.shape[0], 1))).astype(f32)
    eq, es = orc.quant_rows(x)
    for columns in (False, True):
        t = dev(np.ascontiguousarray(x.T if columns else x))
        q, s = torch.empty(t.shape, dtype=torch.int8, device="cuda"), torch.empty(x.shape[0], device="cuda")
        R.repro_quant_rows_i8(t, q, s, columns=columns)
        same(host(s), es)
        assert np.array_equal(host(q).T if columns else host(q), eq)


def test_codes_of_few_bits(orc):
    """bf16 values, whose quotients are ties often, by every significand of the maximum; NaN among them."""
    g = rng(4)
    top = (1 + np.arange(128) / 128).astype(f32)
    x = np.concatenate([top[:, None], T.bf((g.random((128, 700)) * top[:, None]).astype(f32))], 1)
    x[x > top[:, None]] = 0
    x[5, 9], x[6, 3::7] = np.nan, np.nan
    for kind in (F32, BF):
        for a in (x, np.ascontiguousarray(x.T)):
            for columns in (False, True):
                t = dev(a).to(kind)
                q, s = torch.empty(t.shape, dtype=torch.int8, device="cuda"), torch.empty(t.shape[columns], device="cuda")
                R.repro_quant_rows_i8(t, q, s, columns=columns)
                eq, es = orc.quant_rows(a, None, columns)
                same(host(s), es)
                assert np.array_equal(host(q), eq)
    gu = np.ascontiguousarray(np.tile(x[:, :512], (1, 2)))
    codes, scales = torch.empty((128, 2, 4, 128), dtype=torch.int8, device="cuda"), torch.empty((128, 2, 4), device="cuda")
    a = torch.empty((128, 512), device="cuda")
    R.repro_swiglu_fwd(dev(gu), a, codes, scales)
    ea, ec, es = orc.swiglu_fwd(gu)
    same(host(a), ea)
    same(host(scales), es)
    assert np.array_equal(host(codes), ec)


NAMES = ["norm_fwd_channel", "norm_fwd_rows", "norm_bwd_channel", "norm_bwd_rows", "quant_0", "quant_1", "matmul_3", "matmul_40",
         "matmul_700", "matmul_300", "matmul_30", "swiglu_fwd", "swiglu_bwd", "swiglu_bwd_kept"]


@pytest.mark.parametrize("name", NAMES)
def test_nonfinite_inputs_reported(name):
    fn, ins, _ = calls()[name]
    R.repro_set_debug(R.REPRO_DEBUG_CHECK_FINITE)
    try:
        fn()
        assert R.repro_device_check() == R.REPRO_OK
        for t in ins:
            for at, bad in ((0, float("nan")), (-1, float("inf")), (t.numel() // 2, -float("inf"))):
                flat = t.view(-1)
                old = flat[at].clone()
                flat[at] = bad
                fn()
                assert R.repro_device_check() == R.REPRO_ERR_NONFINITE
                flat[at] = old
        fn()
        assert R.repro_device_check() == R.REPRO_OK
    finally:
        R.repro_set_debug(0)
    ins[0].view(-1)[0] = float("nan")
    fn()
    assert R.repro_device_check() == R.REPRO_OK


@pytest.mark.parametrize("name", NAMES)
def test_captured_on_new_inputs(name):
    """A captured call reads its inputs at each replay, and its bits are an eager call's."""
    fn, ins, outs = calls()[name]
    fn()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        fn(st)
    for k in range(2):
        for t in ins:
            t.mul_(-0.5 if k else 3.0)
        fn()
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            graph.replay()
        st.synchronize()
        for o, w in zip(outs, want):
            same(host(o), host(w))
    assert R.repro_device_check() == R.REPRO_OK


def test_all_at_once():
    """Every call on two streams of its own, all in flight together, over and over: the same bits."""
    sets = [calls(), calls()]
    want = {}
    for name, (fn, _, outs) in sets[0].items():
        fn()
        want[name] = [host(o).copy() for o in outs]
    for s in sets:
        for _, _, outs in s.values():
            for o in outs:
                o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(8)]
    for k in range(20):
        for i, name in enumerate(NAMES):
            for j, s in enumerate(sets):
                s[name][0](streams[(2 * i + j) % 8])
    torch.cuda.synchronize()
    for s in sets:
        for name, (_, _, outs) in s.items():
            for o, w in zip(outs, want[name]):
                same(host(o), w, name)
    assert R.repro_device_check() == R.REPRO_OK


FIRST = """
import torch, bitwise_reproducible_int8_gb300 as R
a, b = (torch.randint(-127, 128, s, device="cuda", dtype=torch.int8) for s in ((%d, 700), (260, 700)))
y, ws = torch.zeros(%d, 260, device="cuda"), torch.empty(R.repro_matmul_i8_ws_bytes(%d, 260, 700), device="cuda", dtype=torch.uint8)
exact = (a.double() @ b.double().T).float()
st = torch.cuda.Stream()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=st):
    R.repro_matmul_i8(a, b, y, ws=ws, stream=st)
for _ in range(2):
    y.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        g.replay()
    st.synchronize()
    assert torch.equal(y, exact)
    y2 = torch.zeros_like(y)
    R.repro_matmul_i8(a, b, y2, ws=ws, stream=st)           # runs the check
    st.synchronize()
    assert torch.equal(y2, exact)
assert R.repro_device_check() == R.REPRO_OK
"""


@pytest.mark.parametrize("M", [40, 300])
def test_first_product_in_a_capture(M):
    """A process whose first product is captured: the CUDA cores there, the check with the next eager call."""
    r = subprocess.run([sys.executable, "-c", FIRST % (M, M, M)], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("M", [1, 2, 4, 5])
@pytest.mark.parametrize("N,K", [(16, 1), (16, 3), (512, 31), (528, 33), (1040, 700), (2048, 5632), (11264, 130), (48, 133144)])
@pytest.mark.parametrize("path", [0, -1])
def test_few_tokens_by_transposed_weights(orc, M, N, K, path):
    R.repro_set_launch_cfg(fwd_path=path)
    try:
        T.mm_check(orc, M, N, K, False, True)
        T.mm_check(orc, M, N, K, False, True, "strided", F32, True)
        T.mm_check(orc, M, N, K, False, True, "dense", BF, scales=False)
    finally:
        R.repro_set_launch_cfg(reset=True)
    assert R.repro_device_check() == R.REPRO_OK
