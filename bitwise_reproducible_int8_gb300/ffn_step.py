"""One training step of the feed-forward half of a decoder block, through the C ABI: the norms
around it, 8-bit products with a scale for each token and each channel in all three layouts, and
the gated activation whose inputs are kept in 8 bits for the backward.

  x, attention's output -> norm behind the attention, gate, residual -> H -> norm -> U
  U -> codes by token -> gate and up product -> SwiGLU (8-bit copy) -> codes by token
    -> down product -> Y;  H2 = H (+) residual scale Y
  and back: Y's gradient as codes by token against W_down for the activation's, as codes by
    channel against the activation's codes for W_down's; SwiGLU out of its 8-bit copy; the
    same two products around W_gate_up; the norms' backward with the gains and the gate.

A linear's weights get their codes with a scale for each output channel; a gradient takes the
other side's scales in before it becomes codes, so every product is one of integers.  What the
backward needs of the activations is kept in 8 bits: the codes of U and of the activation, and
the copy of gate and up.  Nothing depends on the run or on the other tokens of the batch: a
token alone gives the bits that it has in a batch.

  python -m bitwise_reproducible_int8_gb300.ffn_step [--steps N] [--graph]
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

import numpy as np
import torch

from . import inputs
from . import repro as R


@dataclass(frozen=True)
class Ffn:
    tokens: int = 512
    width: int = 256
    ffn: int = 704
    alpha: float = 1.0            # residual scales of both additions
    beta: float = 0.5
    seed: int = 900

    def shapes(self) -> dict:
        d, f = self.width, self.ffn
        return {"gate_up": (2 * f, d), "down": (d, f), "post": (d,), "pre": (d,), "gate": (d,)}


def host_inputs(s: Ffn) -> dict:
    """Seeded parameters, one batch and the gradient of its output, on the host."""
    h = {k: inputs.normal(s.seed + i, inputs.S_W, v, 0.02) for i, (k, v) in enumerate(s.shapes().items())}
    for k in ("post", "pre", "gate"):
        h[k] = (1.0 + h[k]).astype(np.float32)
    rows = (s.tokens, s.width)
    h["x"] = inputs.normal(s.seed, inputs.S_X, rows)
    h["attn"] = inputs.normal(s.seed + 1, inputs.S_X, rows, 0.5)
    h["dout"] = inputs.normal(s.seed, inputs.S_DY, rows, 1e-3)
    return h


class FfnStep:
    """Device buffers and the calls of one step."""

    def __init__(self, s: Ffn, host: dict | None = None, device: str = "cuda"):
        self.s = s
        host = host if host is not None else host_inputs(s)
        dev = torch.device(device)
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        e = lambda *shape, dt=torch.float32: torch.empty(shape, dtype=dt, device=dev)  # noqa: E731
        n, d, f, i8 = s.tokens, s.width, s.ffn, torch.int8
        G = -(-f // R.REPRO_SWIGLU_GROUP)
        offs, total = {}, 0
        for k, shape in s.shapes().items():
            offs[k] = total
            total += (int(np.prod(shape)) + 3) // 4 * 4
        self.flat, self.grad = torch.zeros(total, device=dev), torch.zeros(total, device=dev)
        view = lambda b, k: b[offs[k]:offs[k] + int(np.prod(s.shapes()[k]))].view(s.shapes()[k])  # noqa: E731
        self.p, self.dp = {k: view(self.flat, k) for k in offs}, {k: view(self.grad, k) for k in offs}
        for k in offs:
            self.p[k].copy_(torch.from_numpy(host[k]))
        self.x, self.attn, self.dout = t(host["x"]), t(host["attn"]), t(host["dout"])
        self.wq = {k: e(*self.p[k].shape, dt=i8) for k in ("gate_up", "down")}
        self.ws_ = {k: e(self.p[k].shape[0]) for k in ("gate_up", "down")}       # a scale per output channel
        self.h, self.u, self.stats = e(n, d), e(n, d), e(n, 2)
        self.uq, self.us, self.gu = e(n, d, dt=i8), e(n), e(n, 2 * f)
        self.a, self.aq, self.as_ = e(n, f), e(n, f, dt=i8), e(n)
        self.codes, self.scales = e(n, 2, G, R.REPRO_SWIGLU_GROUP, dt=i8), e(n, 2, G)
        self.y, self.h2, self.stats2 = e(n, d), e(n, d), e(n, 2)
        # gradients; codes of one at a time
        self.dh, self.dy, self.da, self.dgu, self.du = e(n, d), e(n, d), e(n, f), e(n, 2 * f), e(n, d)
        self.dx, self.dattn = e(n, d), e(n, d)
        wide = max(d, 2 * f)
        self.gq, self.gs = e(n * wide, dt=i8), e(max(n, wide))
        self.digest = e(32, dt=torch.uint8)
        w = lambda b: torch.empty(max(int(b), 16), dtype=torch.uint8, device=dev)  # noqa: E731
        mm = R.repro_matmul_i8_ws_bytes
        self.space = {
            "mm": w(max(mm(n, 2 * f, d), mm(n, d, f), mm(n, f, d, trans_b=True), mm(n, d, 2 * f, trans_b=True),
                        mm(d, f, n, True, True), mm(2 * f, d, n, True, True))),
            "quant": w(R.repro_quant_rows_i8_ws_bytes(n, wide, columns=True)),
            "norm": w(R.repro_block_norm_bwd_ws_bytes(n, d)),
            "sumsq": w(R.repro_sumsq_ws_bytes(total)),
            "hash": w(R.repro_state_hash_ws_bytes([self.flat, self.grad])),
        }
        self.adam, self.sumsq = [torch.zeros_like(self.flat), torch.zeros_like(self.flat)], e(1)
        torch.cuda.synchronize(dev)

    def weights(self, st) -> None:
        """Codes and scales of the weights, once per update."""
        for k in ("gate_up", "down"):
            R.repro_quant_rows_i8(self.p[k], self.wq[k], self.ws_[k], stream=st)

    def forward(self, st, rows: slice | None = None) -> torch.Tensor:
        """H2 of these tokens (all of them by default); what the backward needs stays in the buffers."""
        s, p, mm = self.s, self.p, self.space["mm"]
        c = lambda t: t if rows is None else t[rows]  # noqa: E731
        norm = dict(alpha=s.alpha, stream=st)
        R.repro_block_norm_fwd(c(self.x), c(self.attn), c(self.h), c(self.u), stats=c(self.stats), gate=p["gate"],
                               g_post=p["post"], g_pre=p["pre"], post=True, **norm)
        R.repro_quant_rows_i8(c(self.u), c(self.uq), c(self.us), stream=st)
        R.repro_matmul_i8(c(self.uq), self.wq["gate_up"], c(self.gu), c(self.us), self.ws_["gate_up"], ws=mm, stream=st)
        R.repro_swiglu_fwd(c(self.gu), c(self.a), c(self.codes), c(self.scales), stream=st)
        R.repro_quant_rows_i8(c(self.a), c(self.aq), c(self.as_), stream=st)
        R.repro_matmul_i8(c(self.aq), self.wq["down"], c(self.y), c(self.as_), self.ws_["down"], ws=mm, stream=st)
        R.repro_block_norm_fwd(c(self.h), c(self.y), c(self.h2), None, stats=c(self.stats2), beta=s.beta, **norm)
        return c(self.h2)

    def _linear_bwd(self, dy, k, xq, xs, dx, st) -> None:
        """dx and the weight gradient of linear k from dy [n, N], the codes xq and scales xs of its input."""
        n, N = dy.shape
        q, mm = self.gq[:n * N].view(n, N), self.space["mm"]
        R.repro_quant_rows_i8(dy, q, self.gs[:n], mul=self.ws_[k], stream=st)
        R.repro_matmul_i8(q, self.wq[k], dx, s_a=self.gs[:n], trans_b=True, ws=mm, stream=st)
        R.repro_quant_rows_i8(dy, q, self.gs[:N], mul=xs, columns=True, ws=self.space["quant"], stream=st)
        R.repro_matmul_i8(q, xq, self.dp[k], s_a=self.gs[:N], trans_a=True, trans_b=True, ws=mm, stream=st)

    def backward(self, st) -> None:
        s, p, dp = self.s, self.p, self.dp
        R.repro_block_norm_bwd(self.dout, None, None, self.y, self.stats2, self.dh, self.dy, alpha=s.alpha, beta=s.beta,
                               stream=st)
        self._linear_bwd(self.dy, "down", self.aq, self.as_, self.da, st)
        R.repro_swiglu_bwd(self.da, self.dgu, codes=self.codes, scales=self.scales, stream=st)
        self._linear_bwd(self.dgu, "gate_up", self.uq, self.us, self.du, st)
        R.repro_block_norm_bwd(self.dh, self.du, self.h, self.attn, self.stats, self.dx, self.dattn, gate=p["gate"],
                               dgate=dp["gate"], g_post=p["post"], g_pre=p["pre"], dg_post=dp["post"], dg_pre=dp["pre"],
                               post=True, alpha=s.alpha, ws=self.space["norm"], stream=st)

    def run(self, stream: torch.cuda.Stream) -> None:
        """Enqueue the weights' codes, forward and backward on `stream`."""
        self.weights(stream)
        self.forward(stream)
        self.backward(stream)

    def update(self, t: int, stream: torch.cuda.Stream, lr: float = 1e-3) -> None:
        """Clip to the global norm and apply AdamW step t (1, 2, ..)."""
        R.repro_sumsq(self.grad, self.sumsq, ws=self.space["sumsq"], stream=stream)
        R.repro_adamw_step(self.flat, *self.adam, self.grad, self.sumsq, t, lr=lr, stream=stream)

    def capture(self, stream: torch.cuda.Stream) -> "torch.cuda.CUDAGraph":
        """Forward and backward as one CUDA graph (run() once before)."""
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            self.run(stream)
        return g

    def state_digest(self, stream: torch.cuda.Stream) -> str:
        """Merkle root of parameters and gradients, as hex.  Synchronises."""
        R.repro_state_hash([self.flat, self.grad], self.digest, ws=self.space["hash"], stream=stream)
        stream.synchronize()
        return bytes(self.digest.cpu().numpy()).hex()


def main() -> None:
    ap = argparse.ArgumentParser(description="train the feed-forward half of a block on a fixed output gradient")
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--graph", action="store_true", help="replay forward and backward as one CUDA graph")
    args = ap.parse_args()
    st = torch.cuda.Stream()
    step = FfnStep(Ffn())
    step.run(st)                     # the first tensor-core call checks its exactness
    st.synchronize()
    graph = step.capture(st) if args.graph else None
    for t in range(1, args.steps + 1):
        if graph is not None:
            with torch.cuda.stream(st):
                graph.replay()
        else:
            step.run(st)
        digest = step.state_digest(st)
        print(f"step {t}: output along its gradient {(step.h2 * step.dout).sum().item():.6f} state {digest}")
        step.update(t, st)
    st.synchronize()
    status = R.repro_device_check(st)
    if status != R.REPRO_OK:
        raise SystemExit(R.repro_status_str(status))


if __name__ == "__main__":
    main()
