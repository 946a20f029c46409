"""GPU: layouts, streams and reports of the embedding, the per-head norm with rotation
and the distillation loss that are not the usual ones."""
import threading

import pytest

torch = pytest.importorskip("torch")

import bitwise_reproducible_int8_gb300 as R  # noqa: E402
from gpu_helpers import dev  # noqa: E402
from test_oracle_blocks import rope_table  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("D", [64, 33])
def test_heads_side_by_side(heads_first, D):
    """q, k and v of each head next to one another, in the inputs and in their gradient: the
    bits of tensors of their own."""
    n, H = 37, 4
    g = torch.Generator(device="cuda").manual_seed(4)
    shape = (H, n, 3, D) if heads_first else (n, H, 3, D)
    x = torch.randn(shape, device="cuda", generator=g)
    dx = torch.full(shape, 9.0, device="cuda")
    part = lambda t, i: (t.transpose(0, 1) if heads_first else t)[:, :, i]  # noqa: E731
    do = [torch.randn(n, H, D, device="cuda", generator=g) for _ in range(2)]
    gains = [torch.rand(D, device="cuda", generator=g) + 0.5 for _ in range(2)]
    rope = dev(rope_table(n, D - D % 2))

    def run(q, k, dq, dk):
        out = [torch.empty(n, H, D, device="cuda") for _ in range(2)]
        dg = [torch.empty(D, device="cuda") for _ in range(2)]
        R.repro_qk_norm_rope_fwd(q, k, rope, *out, g_q=gains[0], g_k=gains[1])
        R.repro_qk_norm_rope_bwd(*do, q, k, rope, dq, dk, g_q=gains[0], g_k=gains[1], dg_q=dg[0], dg_k=dg[1])
        return [*out, dq, dk, *dg]

    got = run(part(x, 0), part(x, 1), part(dx, 0), part(dx, 1))
    own = [part(x, i).contiguous() for i in range(2)]
    exp = run(*own, *(torch.empty_like(t) for t in own))
    for a, b in zip(got, exp):
        assert torch.equal(a, b)
    assert torch.all(part(dx, 2) == 9.0)


def test_widths_in_two_threads():
    """Two host threads in one variant of the backward with different widths: neither's
    shared-memory size gets in the other's way."""
    n, H = 8, 2

    def work(D, seed, failures):
        try:
            g = torch.Generator(device="cuda").manual_seed(seed)
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                x, do = (torch.randn(n, H, D, device="cuda", generator=g) for _ in range(2))
                gain, dx, dg = torch.ones(D, device="cuda"), torch.empty_like(x), torch.empty(D, device="cuda")
                ws = torch.empty(R.repro_qk_norm_rope_bwd_ws_bytes(n, H, 0, D), dtype=torch.uint8, device="cuda")
                for _ in range(3000):
                    R.repro_qk_norm_rope_bwd(do, None, x, None, None, dx, None, g_q=gain, dg_q=dg, ws=ws)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            failures.append((D, e))

    for widths in ((132, 256), (260, 512)):
        failures = []
        threads = [threading.Thread(target=work, args=(D, D, failures)) for D in widths]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not failures, failures


def test_index_and_nonfinite_reports_both_arrive():
    """A token out of range does not hide what the debug scan found."""
    assert R.repro_device_check() == R.REPRO_OK
    table, out = torch.randn(10, 8, device="cuda"), torch.empty(3, 8, device="cuda")
    table[4, 5] = float("nan")
    tok = torch.tensor([1, 10, 2], device="cuda")
    R.repro_set_debug(R.REPRO_DEBUG_CHECK_FINITE)
    try:
        R.repro_embed_fwd(table, tok, out)
        assert [R.repro_device_check() for _ in range(3)] == [R.REPRO_ERR_INDEX, R.REPRO_ERR_NONFINITE, R.REPRO_OK]
        R.repro_embed_fwd(table, tok[:1], out[:1])
        assert [R.repro_device_check() for _ in range(2)] == [R.REPRO_ERR_NONFINITE, R.REPRO_OK]
    finally:
        R.repro_set_debug(0)
        R.repro_device_check()
    R.repro_embed_fwd(table, tok, out)
    assert [R.repro_device_check() for _ in range(2)] == [R.REPRO_ERR_INDEX, R.REPRO_OK]


@pytest.mark.parametrize("handle", [False, True])
def test_workspace_beside_the_current_streams_work(handle):
    """A call on another stream makes its workspace while the current stream has yet to write
    memory it has already let go of."""
    n, V = 2000, 20000
    s = torch.cuda.Stream()
    z, tl = torch.randn(n, V, device="cuda"), torch.randn(n, 8, device="cuda")
    idx, tok = torch.randint(0, V, (n, 8), device="cuda"), torch.randint(0, 50, (n,), device="cuda")
    loss, stats = torch.empty(n, device="cuda"), torch.empty(n, R.REPRO_DISTILL_STATS + 8, device="cuda")
    dW = torch.empty(50, V, device="cuda")
    where = s.cuda_stream if handle else s

    def calls(**kw):
        R.repro_distill_fwd(z, idx, tl, loss, stats, **kw)
        R.repro_embed_bwd(z, tok, dW, **kw)

    calls()
    want = loss.clone(), dW.clone()
    sizes = R.repro_distill_ws_bytes(n, V), R.repro_embed_bwd_ws_bytes(n, 50, V)
    for _ in range(3):
        loss.zero_()
        dW.zero_()
        torch.cuda.synchronize()
        torch.cuda._sleep(1000000)
        for b in sizes:
            torch.empty(b, dtype=torch.uint8, device="cuda").fill_(0xff)
        calls(stream=where)
        torch.cuda.synchronize()
        assert torch.equal(loss, want[0]) and torch.equal(dW, want[1])


def test_single_token_of_a_long_sequence():
    """The last token of [1, T, H, D] whose sequence is longer than any token stride may be."""
    T, H, D = 140000, 16, 128
    whole = torch.zeros(1, T, H, D, device="cuda", dtype=torch.bfloat16)
    q = whole[:, -1:]
    q.normal_()
    assert q.stride(0) > 1 << 28
    rope = dev(rope_table(4, D))
    got, exp = torch.empty(1, 1, H, D, device="cuda"), torch.empty(1, 1, H, D, device="cuda")
    R.repro_qk_norm_rope_fwd(q, None, rope, got, None)
    R.repro_qk_norm_rope_fwd(q.clone(), None, rope, exp, None)
    assert torch.equal(got, exp)
    dq = torch.empty_like(whole)[:, -1:]
    own = torch.empty(1, 1, H, D, device="cuda", dtype=torch.bfloat16)
    R.repro_qk_norm_rope_bwd(got, None, q, None, rope, dq, None)
    R.repro_qk_norm_rope_bwd(got, None, q.clone(), None, rope, own, None)
    assert torch.equal(dq, own)


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gain_of_one_side(which, accumulate):
    """Gains of the queries or of the keys alone: the bits of each side by itself."""
    n, D, heads = 200, 128, {"q": 5, "k": 2}
    g = torch.Generator(device="cuda").manual_seed(6)
    x, do = ({nm: torch.randn(n, h, D, device="cuda", generator=g) for nm, h in heads.items()} for _ in range(2))
    gain, acc = torch.rand(D, device="cuda", generator=g) + 0.5, torch.randn(D, device="cuda", generator=g)
    rope = dev(rope_table(n, D))
    kw = {"g_" + which: gain}
    out = {nm: torch.empty(n, h, D, device="cuda") for nm, h in heads.items()}
    dx, dg = {nm: torch.empty_like(t) for nm, t in x.items()}, acc.clone()
    R.repro_qk_norm_rope_fwd(x["q"], x["k"], rope, out["q"], out["k"], **kw)
    R.repro_qk_norm_rope_bwd(do["q"], do["k"], x["q"], x["k"], rope, dx["q"], dx["k"], accumulate=accumulate,
                             **kw, **{"dg_" + which: dg})
    for nm in heads:
        has = nm == which
        o, d, e = torch.empty_like(out[nm]), torch.empty_like(x[nm]), acc.clone()
        R.repro_qk_norm_rope_fwd(x[nm], None, rope, o, None, g_q=gain if has else None)
        R.repro_qk_norm_rope_bwd(do[nm], None, x[nm], None, rope, d, None, g_q=gain if has else None,
                                 dg_q=e if has else None, accumulate=accumulate)
        assert torch.equal(out[nm], o) and torch.equal(dx[nm], d)
        assert not has or torch.equal(dg, e)
