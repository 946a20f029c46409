"""GPU: the feed-forward calls where their forms meet -- rows on 2-element boundaries, few and many
tokens of wide rows, calls at once on two streams, captured ones on new inputs, and the debug scan of
every float input."""
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
