"""One training step of a small student on a teacher's top logits, from tokens to
gradients, through the C ABI: the calls around the decoder blocks together with
the ones inside.

  tokens -> embedding (x sqrt(d)) -> X
  X -> int8 QKV linear -> norm of the query and key heads with the rotation
    -> int8 P.V attention -> int8 output linear -> H = X (+) A
  H -> int8 head linear -> logits -> loss against the teacher's top logits, the
    labels and the log-partition penalty; the logits' gradient in their place
  and back: head, output linear, attention, rotation and norm, QKV linear, and the
    embedding's gradient from the sum of both paths into X.

Every gradient lies in one flat buffer (embedding, QKV, output, head, the two
gains), so that clip + AdamW and the state hash take it as they take any other.
All arithmetic happens in librepro.so; this module allocates device memory, copies
and enqueues calls.  Nothing depends on the run: the same inputs give the same
digest.

  python -m bitwise_reproducible_int8_gb300.distill_step [--steps N] [--graph]
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

import numpy as np
import torch

from . import inputs
from . import repro as R


@dataclass(frozen=True)
class Student:
    vocab: int = 2000
    width: int = 256
    heads_q: int = 4
    heads_kv: int = 2
    sequences: int = 2
    seq_len: int = 192
    window: int = 64
    theta: float = 500000.0
    top: int = 16             # teacher entries per position
    tau: float = 2.0
    w_kd: float = 0.9
    w_ce: float = 0.1
    w_z: float = 1e-4
    seed: int = 700

    @property
    def tokens(self) -> int:
        return self.sequences * self.seq_len

    @property
    def qkv_rows(self) -> int:
        return (self.heads_q + 2 * self.heads_kv) * inputs.HEAD_DIM

    @property
    def loss_args(self) -> dict:
        return dict(tau=self.tau, w_kd=self.w_kd, w_ce=self.w_ce, w_z=self.w_z)

    def shapes(self) -> dict:
        d, a = self.width, self.heads_q * inputs.HEAD_DIM
        return {"embed": (self.vocab, d), "qkv": (self.qkv_rows, d), "out": (d, a), "head": (self.vocab, d),
                "gain_q": (inputs.HEAD_DIM,), "gain_k": (inputs.HEAD_DIM,)}


def rope_table(positions: int, width: int, theta: float = 500000.0) -> np.ndarray:
    """[positions, width] float32: width / 2 cosines, then width / 2 sines, of
    position * theta^(-2j / width), taken in 64 bits and rounded once."""
    j = np.arange(width // 2, dtype=np.float64)
    ang = np.arange(positions, dtype=np.float64)[:, None] * theta ** (-2.0 * j / max(width, 1))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def host_inputs(s: Student) -> dict:
    """Seeded parameters and one batch, on the host."""
    g = np.random.default_rng(s.seed)
    h = {k: (0.02 * g.standard_normal(v)).astype(np.float32) for k, v in s.shapes().items()}
    for k in ("gain_q", "gain_k"):
        h[k] = (1.0 + h[k]).astype(np.float32)
    p = 1.0 / (np.arange(s.vocab) + 2.0)
    h["tokens"] = g.choice(s.vocab, s.tokens, p=p / p.sum()).astype(np.int32)
    h["tokens"][-3:] = -1                                    # the end of the batch is padding
    h["t_idx"] = np.stack([g.permutation(s.vocab)[:s.top] for _ in range(s.tokens)]).astype(np.int32)
    h["t_logits"] = (6.0 - 1.5 * np.log1p(np.arange(s.top)) + 0.3 * g.standard_normal((s.tokens, s.top))).astype(np.float32)
    h["labels"] = h["t_idx"][:, 0].copy()
    h["labels"][-3:] = -100
    h["t_idx"][-3:] = -1
    h["rope"] = rope_table(s.seq_len, inputs.HEAD_DIM, s.theta)
    h["g"] = np.float32([1.0 / s.tokens])
    return h


class DistillStep:
    """Device buffers and the calls of one step."""

    def __init__(self, s: Student, host: dict | None = None, device: str = "cuda"):
        self.s = s
        host = host if host is not None else host_inputs(s)
        dev = torch.device(device)
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        e = lambda *shape, dt=torch.float32: torch.empty(shape, dtype=dt, device=dev)  # noqa: E731
        n, d, D = s.tokens, s.width, inputs.HEAD_DIM
        B, T, Hq, Hkv = s.sequences, s.seq_len, s.heads_q, s.heads_kv
        # parameters and gradients as views of flat buffers, each on 16 bytes
        self.flat, self.grad, self.p, self.dp = self._flat(s, host, dev)
        self.batch = {k: t(host[k]) for k in ("tokens", "t_idx", "t_logits", "labels", "rope", "g")}
        i8 = torch.int8
        self.wq = {k: e(*self.p[k].shape, dt=i8) for k in ("qkv", "out", "head")}
        self.scale = {k: e(1) for k in ("w_qkv", "w_out", "w_head", "x", "o", "h", "v")}
        self.x, self.xq, self.y = e(n, d), e(n, d, dt=i8), e(n, s.qkv_rows)
        self.q, self.k, self.v = e(B, T, Hq, D), e(B, T, Hkv, D), e(B, T, Hkv, D)
        self.vq = e(B, T, Hkv, D, dt=i8)
        self.o, self.m, self.l = e(B, T, Hq, D), e(B, T, Hq), e(B, T, Hq)
        self.oq, self.h, self.hq = e(n, Hq * D, dt=i8), e(n, d), e(n, d, dt=i8)
        self.a, self.z = e(n, d), e(n, s.vocab)
        self.loss, self.stats = e(n), e(n, R.REPRO_DISTILL_STATS + s.top)
        self.dh, self.do = e(n, d), e(B, T, Hq, D)
        self.dq, self.dk, self.dv = e(B, T, Hq, D), e(B, T, Hkv, D), e(B, T, Hkv, D)
        self.dy, self.dx = e(n, s.qkv_rows), e(n, d)
        self.digest = e(32, dt=torch.uint8)
        # workspaces, one per use: nothing is allocated in a step
        w = lambda b: torch.empty(max(int(b), 16), dtype=torch.uint8, device=dev)  # noqa: E731
        largest = max(x.numel() for x in (*self.p.values(), self.x, self.h, self.o, self.v))
        lin = [(n, s.qkv_rows, d), (n, d, Hq * D), (n, s.vocab, d)]
        self.ws = {
            "scale": w(R.repro_wscale_ws_bytes(largest)),
            "fwd": w(max(R.repro_linear_fwd_ws_bytes(*g) for g in lin)),
            "bwd": w(max(R.repro_linear_bwd_ws_bytes(*g) for g in lin)),
            "attn": w(R.repro_attn_fwd_ws_bytes(B, T, Hq, s.window)),
            "attn_bwd": w(R.repro_attn_bwd_ws_bytes(B, T, Hq, s.window)),
            "qk": w(R.repro_qk_norm_rope_bwd_ws_bytes(n, Hq, Hkv, D)),
            "embed": w(R.repro_embed_bwd_ws_bytes(n, s.vocab, d)),
            "distill": w(R.repro_distill_ws_bytes(n, s.vocab)),
            "sumsq": w(R.repro_sumsq_ws_bytes(self.grad.numel())),
            "hash": w(R.repro_state_hash_ws_bytes([self.flat, self.grad])),
        }
        self.adam = [torch.zeros_like(self.flat), torch.zeros_like(self.flat)]
        self.sumsq = e(1)
        torch.cuda.synchronize(dev)

    @staticmethod
    def _flat(s: Student, host: dict, dev):
        offs, total = {}, 0
        for k, shape in s.shapes().items():
            offs[k] = total
            total += (int(np.prod(shape)) + 3) // 4 * 4
        flat, grad = torch.zeros(total, device=dev), torch.zeros(total, device=dev)
        view = lambda b, k: b[offs[k]:offs[k] + int(np.prod(s.shapes()[k]))].view(s.shapes()[k])  # noqa: E731
        p, dp = {k: view(flat, k) for k in offs}, {k: view(grad, k) for k in offs}
        for k in offs:
            p[k].copy_(torch.from_numpy(host[k]))
        return flat, grad, p, dp

    def _codes(self, x, name, out, st) -> torch.Tensor:
        """Activation scale and int8 codes of x."""
        R.repro_wscale(x, R.REPRO_SCALE_ACT_AMAX, self.scale[name], ws=self.ws["scale"], stream=st)
        R.repro_quant_i8(x, self.scale[name], out, stream=st)
        return out

    def _heads(self, t, lo, count):
        """Heads [lo, lo + count) of the fused QKV rows, as [B, T, count, D]."""
        s, D = self.s, inputs.HEAD_DIM
        return t.view(s.sequences, s.seq_len, -1, D)[:, :, lo:lo + count]

    def run(self, stream: torch.cuda.Stream) -> None:
        """Enqueue forward and backward on `stream`."""
        s, b, st = self.s, self.batch, stream
        Hq, Hkv = s.heads_q, s.heads_kv
        with torch.cuda.stream(st):
            for k in ("qkv", "out", "head"):
                R.repro_wscale(self.p[k], R.REPRO_SCALE_WEIGHT_MEANABS, self.scale["w_" + k], ws=self.ws["scale"],
                               stream=st)
                R.repro_quant_i8(self.p[k], self.scale["w_" + k], self.wq[k], stream=st)
            # forward
            R.repro_embed_fwd(self.p["embed"], b["tokens"], self.x, scale=s.width ** 0.5, stream=st)
            self._codes(self.x, "x", self.xq, st)
            R.repro_linear_fwd(self.xq, self.wq["qkv"], self.scale["x"], self.scale["w_qkv"], self.y,
                               ws=self.ws["fwd"], stream=st)
            q, k, v = self._heads(self.y, 0, Hq), self._heads(self.y, Hq, Hkv), self._heads(self.y, Hq + Hkv, Hkv)
            norm = dict(g_q=self.p["gain_q"], g_k=self.p["gain_k"])
            R.repro_qk_norm_rope_fwd(q, k, b["rope"], self.q, self.k, **norm, stream=st)
            self.v.copy_(v)
            self._codes(self.v, "v", self.vq, st)
            R.repro_attn_fwd(self.q, self.k, self.vq, self.scale["v"], self.o, self.m, self.l, s.window,
                             ws=self.ws["attn"], stream=st)
            self._codes(self.o.view(s.tokens, -1), "o", self.oq, st)
            R.repro_linear_fwd(self.oq, self.wq["out"], self.scale["o"], self.scale["w_out"], self.a,
                               ws=self.ws["fwd"], stream=st)
            self.h.copy_(self.x)
            R.repro_grad_accum(self.h, self.a, stream=st)
            self._codes(self.h, "h", self.hq, st)
            R.repro_linear_fwd(self.hq, self.wq["head"], self.scale["h"], self.scale["w_head"], self.z,
                               ws=self.ws["fwd"], stream=st)
            R.repro_distill_fwd(self.z, b["t_idx"], b["t_logits"], self.loss, self.stats, labels=b["labels"],
                                ws=self.ws["distill"], **s.loss_args, stream=st)
            # backward; the logits make room for their gradient
            R.repro_distill_bwd(self.z, b["t_idx"], self.stats, b["g"], self.z, labels=b["labels"], **s.loss_args,
                                stream=st)
            lin = dict(ws=self.ws["bwd"], stream=st)
            R.repro_linear_bwd(self.z, self.hq, self.wq["head"], self.scale["h"], self.scale["w_head"], self.dh,
                               self.dp["head"], **lin)
            R.repro_linear_bwd(self.dh, self.oq, self.wq["out"], self.scale["o"], self.scale["w_out"],
                               self.do.view(s.tokens, -1), self.dp["out"], **lin)
            R.repro_attn_bwd(self.q, self.k, self.vq, self.scale["v"], self.o, self.do, self.m, self.l, self.dq,
                             self.dk, self.dv, s.window, ws=self.ws["attn_bwd"], fwd_ws=self.ws["attn"], stream=st)
            R.repro_qk_norm_rope_bwd(self.dq, self.dk, q, k, b["rope"], self._heads(self.dy, 0, Hq),
                                     self._heads(self.dy, Hq, Hkv), **norm, dg_q=self.dp["gain_q"],
                                     dg_k=self.dp["gain_k"], ws=self.ws["qk"], stream=st)
            self._heads(self.dy, Hq + Hkv, Hkv).copy_(self.dv)
            R.repro_linear_bwd(self.dy, self.xq, self.wq["qkv"], self.scale["x"], self.scale["w_qkv"], self.dx,
                               self.dp["qkv"], **lin)
            R.repro_grad_accum(self.dx, self.dh, stream=st)      # both paths into X
            R.repro_embed_bwd(self.dx, b["tokens"], self.dp["embed"], scale=s.width ** 0.5, ws=self.ws["embed"],
                              stream=st)

    def update(self, t: int, stream: torch.cuda.Stream, lr: float = 1e-3) -> None:
        """Clip to the global norm and apply AdamW step t (1, 2, ..)."""
        R.repro_sumsq(self.grad, self.sumsq, ws=self.ws["sumsq"], stream=stream)
        R.repro_adamw_step(self.flat, *self.adam, self.grad, self.sumsq, t, lr=lr, stream=stream)

    def capture(self, stream: torch.cuda.Stream) -> "torch.cuda.CUDAGraph":
        """Forward and backward as one CUDA graph (run() once before)."""
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            self.run(stream)
        return g

    def state_digest(self, stream: torch.cuda.Stream) -> str:
        """Merkle root of parameters and gradients, as hex.  Synchronises."""
        R.repro_state_hash([self.flat, self.grad], self.digest, ws=self.ws["hash"], stream=stream)
        stream.synchronize()
        return bytes(self.digest.cpu().numpy()).hex()


def main() -> None:
    ap = argparse.ArgumentParser(description="train a small student on a teacher's top logits")
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--graph", action="store_true", help="replay forward and backward as one CUDA graph")
    args = ap.parse_args()
    st = torch.cuda.Stream()
    step = DistillStep(Student())
    step.run(st)                     # the first tensor-core calls check their exactness
    st.synchronize()
    graph = step.capture(st) if args.graph else None
    for t in range(1, args.steps + 1):
        if graph is not None:
            with torch.cuda.stream(st):
                graph.replay()
        else:
            step.run(st)
        digest = step.state_digest(st)
        print(f"step {t}: loss {step.loss.mean().item():.6f} state {digest}")
        step.update(t, st)
    st.synchronize()
    status = R.repro_device_check(st)
    if status != R.REPRO_OK:
        raise SystemExit(R.repro_status_str(status))


if __name__ == "__main__":
    main()
