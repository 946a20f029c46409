"""GPU: a training step of a block's feed-forward half -- norms, codes, products in three layouts,
SwiGLU out of its 8-bit copy -- bit for bit against the oracle's calls in the same order; captured
into a graph, on two streams at once, token by token, and with the tensor cores off."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import bitwise_reproducible_int8_gb300 as R  # noqa: E402
from bitwise_reproducible_int8_gb300.ffn_step import Ffn, FfnStep, host_inputs  # noqa: E402
from gpu_helpers import assert_bits_equal, host  # noqa: E402

pytestmark = pytest.mark.gpu
CASES = [Ffn(tokens=70, width=64, ffn=200), Ffn(tokens=33, width=50, ffn=131, alpha=0.75), Ffn(tokens=300, width=128, ffn=256)]


def oracle_step(orc, s, h):
    """(H2, dx, dattn, gradients by name) from the oracle."""
    wq, sw = {}, {}
    for k in ("gate_up", "down"):
        wq[k], sw[k] = orc.quant_rows(h[k])
    norm = dict(gate=h["gate"], g_post=h["post"], g_pre=h["pre"], alpha=s.alpha, post=True)
    hh, u, st = orc.block_norm_fwd(h["x"], h["attn"], **norm)
    uq, us = orc.quant_rows(u)
    gu = orc.matmul_i8(uq, wq["gate_up"], us, sw["gate_up"])
    a, codes, scales = orc.swiglu_fwd(gu)
    aq, as_ = orc.quant_rows(a)
    y = orc.matmul_i8(aq, wq["down"], as_, sw["down"])
    h2, _, st2 = orc.block_norm_fwd(hh, y, alpha=s.alpha, beta=s.beta, want_u=False)
    g = {}

    def linear_bwd(dy, k, xq, xs):
        q, qs = orc.quant_rows(dy, sw[k])
        dx = orc.matmul_i8(q, wq[k], qs, None, False, True)
        q, qs = orc.quant_rows(dy, xs, True)
        g[k] = orc.matmul_i8(q, xq, qs, None, True, True)
        return dx

    dh, dy, *_ = orc.block_norm_bwd(h["dout"], None, None, y, st2, alpha=s.alpha, beta=s.beta)
    da = linear_bwd(dy, "down", aq, as_)
    dgu = orc.swiglu_bwd(da, codes=codes, scales=scales)
    du = linear_bwd(dgu, "gate_up", uq, us)
    dx, dattn, g["gate"], g["post"], g["pre"] = orc.block_norm_bwd(dh, du, hh, h["attn"], st, **norm)
    return h2, dx, dattn, g


def check(step, exp):
    h2, dx, dattn, g = exp
    assert_bits_equal(host(step.h2), h2, "h2")
    assert_bits_equal(host(step.dx), dx, "dx")
    assert_bits_equal(host(step.dattn), dattn, "dattn")
    for k, e in g.items():
        assert_bits_equal(host(step.dp[k]), e, k)


@pytest.mark.parametrize("s", CASES)
def test_step(orc, s):
    h = host_inputs(s)
    exp = oracle_step(orc, s, h)
    step, st = FfnStep(s, h), torch.cuda.Stream()
    step.run(st)
    st.synchronize()
    check(step, exp)
    graph = step.capture(st)
    for t in (step.h2, step.dx, step.dattn, step.grad, step.codes):
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(2):
        with torch.cuda.stream(st):
            graph.replay()
    st.synchronize()
    check(step, exp)
    assert R.repro_device_check(st) == R.REPRO_OK


def test_tokens_alone_give_the_batch_s_bits():
    s = CASES[2]
    step, st = FfnStep(s), torch.cuda.Stream()
    step.weights(st)
    step.forward(st)
    st.synchronize()
    batch = host(step.h2).copy()
    for rows in (slice(0, 1), slice(7, 8), slice(100, 116), slice(20, 57), slice(299, 300)):
        step.h2.fill_(7.0)
        torch.cuda.synchronize()
        got = step.forward(st, rows)
        st.synchronize()
        assert_bits_equal(host(got), batch[rows], str(rows))


def test_two_steps_at_once_and_without_tensor_cores():
    """Two steps whose calls overlap on two streams, and one on the CUDA cores: one digest."""
    s = CASES[0]
    digests = []
    steps, streams = [FfnStep(s) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for step, st in zip(steps, streams):
            step.run(st)
    digests += [step.state_digest(st) for step, st in zip(steps, streams)]
    for hook in (dict(fwd_path=0), dict(fwd_selftest=1)):
        R.repro_set_launch_cfg(**hook)
        steps[0].grad.zero_()
        torch.cuda.synchronize()
        steps[0].run(streams[0])
        digests.append(steps[0].state_digest(streams[0]))
        R.repro_set_launch_cfg(reset=True)
    R.repro_device_check(streams[0])                         # takes the forced failure's report
    assert len(set(digests)) == 1


def test_a_few_updates():
    step, st = FfnStep(CASES[0]), torch.cuda.Stream()
    seen = set()
    for t in range(1, 4):
        step.run(st)
        step.update(t, st)
        seen.add(step.state_digest(st))
    assert len(seen) == 3
    assert bool(torch.isfinite(step.flat).all())
