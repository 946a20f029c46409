"""GPU: a whole training step of a small student -- embedding, QKV linear, head norm
with rotation, attention, output and head linears, distillation loss, and back --
bit for bit against the oracle's calls in the same order; captured into a graph; and
trained for a few steps."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import bitwise_reproducible_int8_gb300 as R  # noqa: E402
from bitwise_reproducible_int8_gb300.distill_step import DistillStep, Student, host_inputs  # noqa: E402
from gpu_helpers import assert_bits_equal, host  # noqa: E402

pytestmark = pytest.mark.gpu
SMALL = Student(vocab=301, width=64, heads_q=2, heads_kv=1, sequences=2, seq_len=70, window=48, top=5)


def oracle_step(orc, s, h):
    """(loss, gradients by name) from the oracle."""
    B, T, Hq, Hkv, n = s.sequences, s.seq_len, s.heads_q, s.heads_kv, s.tokens
    D, sc = 128, float(np.float32(s.width ** 0.5))
    sw = {k: orc.wscale(h[k], 0) for k in ("qkv", "out", "head")}
    wq = {k: orc.quant_i8(h[k], sw[k]) for k in sw}

    def codes(x):
        a = orc.wscale(x, 1)
        return orc.quant_i8(x, a), a

    x = orc.embed_fwd(h["embed"], h["tokens"], sc)
    xq, sx = codes(x)
    y = orc.linear_fwd(xq, wq["qkv"], sx, sw["qkv"]).reshape(n, -1, D)
    yq, yk, v = y[:, :Hq], y[:, Hq:Hq + Hkv], np.ascontiguousarray(y[:, Hq + Hkv:]).reshape(B, T, Hkv, D)
    pos = np.tile(np.arange(T, dtype=np.int32), B)
    q = orc.qk_fwd(yq, h["rope"], pos, h["gain_q"]).reshape(B, T, Hq, D)
    k = orc.qk_fwd(yk, h["rope"], pos, h["gain_k"]).reshape(B, T, Hkv, D)
    vq, sv = codes(v)
    o, m, l = orc.attn_fwd(q, k, vq, sv, s.window)
    oq, so = codes(o.reshape(n, -1))
    hid = orc.grad_accum(x, orc.linear_fwd(oq, wq["out"], so, sw["out"]))
    hq, sh = codes(hid)
    z = orc.linear_fwd(hq, wq["head"], sh, sw["head"])
    loss, stats = orc.distill_fwd(z, h["t_idx"], h["t_logits"], h["labels"], **s.loss_args)
    dz = orc.distill_bwd(z, h["t_idx"], stats, h["g"], h["labels"], **s.loss_args)
    dh = orc.linear_bwd_dx(dz, wq["head"], sw["head"])
    g = {"head": orc.linear_bwd_dw(dz, hq, sh), "out": orc.linear_bwd_dw(dh, oq, so)}
    do = orc.linear_bwd_dx(dh, wq["out"], sw["out"]).reshape(o.shape)
    dq, dk, dv = orc.attn_bwd(q, k, vq, sv, o, do, m, l, s.window)
    dyq, g["gain_q"] = orc.qk_bwd(dq.reshape(n, Hq, D), yq, h["rope"], pos, h["gain_q"])
    dyk, g["gain_k"] = orc.qk_bwd(dk.reshape(n, Hkv, D), yk, h["rope"], pos, h["gain_k"])
    dy = np.concatenate([dyq, dyk, dv.reshape(n, Hkv, D)], 1).reshape(n, -1)
    g["qkv"] = orc.linear_bwd_dw(dy, xq, sx)
    dx = orc.grad_accum(orc.linear_bwd_dx(dy, wq["qkv"], sw["qkv"]), dh)
    g["embed"] = orc.embed_bwd(dx, h["tokens"], s.vocab, sc)
    return loss, g


@pytest.fixture(scope="module")
def expected(orc):
    h = host_inputs(SMALL)
    return h, *oracle_step(orc, SMALL, h)


def check(step, loss, grads, what):
    assert_bits_equal(host(step.loss), loss, what + " loss")
    for k, g in grads.items():
        assert_bits_equal(host(step.dp[k]), g, what + " d" + k)


def test_step_matches_oracle(expected):
    h, loss, grads = expected
    step = DistillStep(SMALL, h)
    st = torch.cuda.Stream()
    step.run(st)
    check(step, loss, grads, "eager")
    assert R.repro_device_check(st) == 0


def test_graph_beside_an_eager_step(expected):
    """Captured while another step's buffers and results live; replays give the eager
    bits, also after the buffers were overwritten."""
    h, loss, grads = expected
    st = torch.cuda.Stream()
    other = DistillStep(SMALL, h)
    other.run(st)
    step = DistillStep(SMALL, h)
    step.run(st)
    st.synchronize()
    graph = step.capture(st)
    for _ in range(2):
        step.grad.fill_(float("nan"))
        step.loss.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            graph.replay()
        check(step, loss, grads, "graph")
    check(other, loss, grads, "eager")
    assert R.repro_device_check(st) == 0


def test_training_repeats_and_learns():
    st = torch.cuda.Stream()
    runs = []
    for _ in range(2):
        step = DistillStep(Student(vocab=500, sequences=1, seq_len=130))
        out = []
        for t in range(1, 7):
            step.run(st)
            out.append((step.state_digest(st), float(step.loss.mean().item())))
            step.update(t, st)
        runs.append(out)
    assert runs[0] == runs[1]
    assert runs[0][-1][1] < runs[0][0][1]
    assert R.repro_device_check(st) == 0
