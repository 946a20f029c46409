"""The feed-forward half of a decoder block around its 8-bit products, as it is measured.

  norm     RMS norms behind and before a block, with the block's gate and the residual
           scales between them, and their backward
  quant    8-bit codes with a scale for each token or each channel
  matmul   the product of 8-bit codes with scales for tokens and channels, in the three
           layouts of a training step (outputs, input gradients, weight gradients)
  swiglu   the gated activation, its inputs kept in 8 bits, and its backward from those

`own` False: plain torch operations.  `own` True: the library's calls.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
EPS = 1e-6
GROUP = 128      # neighbours that share a scale in the 8-bit copy of the activation's inputs


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one 16,384-token micro-batch at the model width: the attention's output is normed and
        # added to the residual stream, and the stream normed for the feed-forward half
        dict(name="norm_fwd_16k", op="norm_fwd", n=16384, D=2048, x="f32", u="f32", y=True, post=True,
             gate="none", alpha=1.0, beta=1.0),
        # one token of a model served in narrow types, its block gated element by element: latency
        dict(name="norm_fwd_1tok", op="norm_fwd", n=1, D=2048, x="bf16", u="bf16", y=True, post=True,
             gate="token", alpha=1.0, beta=1.0),
        # the micro-batch's backward with both gains
        dict(name="norm_bwd_16k", op="norm_bwd", n=16384, D=2048, x="f32", u="f32", y=True, post=True,
             gate="none", alpha=1.0, beta=1.0),
        # an odd width and token count, a scale per channel on the block, residual scales
        dict(name="norm_bwd_ragged", op="norm_bwd", n=1023, D=1001, x="bf16", u="f32", y=True, post=False,
             gate="channel", alpha=0.9, beta=0.25),
        # the down projection's input, a scale for each token
        dict(name="quant_tokens_16k", op="quant", n=16384, D=5632, x="f32", columns=False, mul=False),
        # the gradient of the outputs for the weights' gradient: a scale for each channel, each
        # token's activation scale folded in
        dict(name="quant_channels_ragged", op="quant", n=4099, D=2003, x="f32", columns=True, mul=True),
        # the fused gate and up projection of a micro-batch
        dict(name="matmul_gate_up_16k", op="matmul", M=16384, N=11264, K=2048, ta=False, tb=False, y="f32",
             accumulate=False),
        # the down projection of one token
        dict(name="matmul_1tok", op="matmul", M=1, N=2048, K=5632, ta=False, tb=False, y="f32",
             accumulate=False),
        # the down projection's weight gradient, summed over the micro-batch's tokens
        dict(name="matmul_dw_16k", op="matmul", M=2048, N=5632, K=16384, ta=True, tb=True, y="f32",
             accumulate=True),
        # the micro-batch's activation and its 8-bit copy
        dict(name="swiglu_fwd_16k", op="swiglu_fwd", n=16384, F=5632, x="f32", a="f32", keep=True),
        # a short ragged batch of an odd width in narrow types
        dict(name="swiglu_fwd_ragged", op="swiglu_fwd", n=301, F=1001, x="bf16", a="bf16", keep=True),
        # the micro-batch's backward out of the 8-bit copy
        dict(name="swiglu_bwd_16k", op="swiglu_bwd", n=16384, F=5632, x="f32", a="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Any width, or a multiple of 64."""
    w = _log_int(rng, lo, hi)
    return w if rng.random() < 0.5 else max(64, w // 64 * 64)


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "quant", "matmul", "matmul", "swiglu_fwd", "swiglu_bwd"])
    kind = rng.choice(["f32", "f32", "bf16"])
    if op.startswith("norm"):
        D = _width(rng, 33, 8192)
        y = rng.random() < 0.8
        return dict(op=op, n=_log_int(rng, 1, max(1, 16384 * 2048 // D)), D=D, x=kind,
                    u="bf16" if kind == "bf16" else rng.choice(["f32", "bf16"]), y=y, post=y and rng.random() < 0.6,
                    gate=rng.choice(["none", "channel", "token"]) if y else "none",
                    alpha=rng.choice([1.0, 0.75]) if y else 1.0, beta=rng.choice([1.0, 0.25]) if y else 1.0)
    if op == "quant":
        D = _width(rng, 20, 12000)
        return dict(op=op, n=_log_int(rng, 1, max(1, min(40000, 16384 * 5632 // D))), D=D, x=kind,
                    columns=rng.random() < 0.5, mul=rng.random() < 0.5)
    if op == "matmul":
        ta, tb = rng.choice([(False, False), (False, False), (False, True), (True, True)])
        N, K = _width(rng, 64, 12000), _width(rng, 64, 12000)
        M = _log_int(rng, 1, max(1, min(16384, 16384 * 11264 * 2048 // (N * K))))
        if ta:      # summed over the tokens
            M, K = max(64, min(N, K)), max(64, M)
        y = rng.choice(["f32", "f32", "bf16"])
        return dict(op=op, M=M, N=N, K=K, ta=ta, tb=tb, y=y, accumulate=y == "f32" and ta and rng.random() < 0.5)
    F = _width(rng, 60, 8192)
    c = dict(op=op, n=_log_int(rng, 1, max(1, 16384 * 5632 // F)), F=F, x=kind, a=rng.choice(["f32", "f32", "bf16"]))
    if op == "swiglu_fwd":
        c["keep"] = rng.random() < 0.7
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    t = torch.empty(shape, device="cuda", dtype=torch.float32)
    t.normal_(0.0, std, generator=g)
    return t.to(dtype)


def _scales(g, n, std):
    """Quantiser steps of n rows of that deviation: their largest values over 127."""
    return (std * 3.5 / 127.0) * (0.7 + 0.6 * torch.rand(n, generator=g, device="cuda"))


def _ceil_div(a, b):
    return -(-a // b)


def _ws(nbytes):
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    c, g, op = case, _gen(seed), case["op"]
    s = {"case": dict(case)}
    if op.startswith("norm"):
        n, D, t = c["n"], c["D"], DT[c["x"]]
        s["x"] = _randn(g, n, D, std=1.5, dtype=t)
        s["y"] = _randn(g, n, D, std=0.7, dtype=t) if c["y"] else None
        s["g_pre"] = 1.0 + _randn(g, D, std=0.1)
        s["g_post"] = 0.5 + _randn(g, D, std=0.1) if c["post"] else None
        s["gate"] = {"none": lambda: None, "channel": lambda: 0.3 + _randn(g, D, std=0.1),
                     "token": lambda: torch.sigmoid(_randn(g, n, D)).to(t)}[c["gate"]]()
        if op == "norm_bwd":
            s["dh"] = _randn(g, n, D, std=1e-3, dtype=t)
            s["du"] = _randn(g, n, D, std=1e-3, dtype=DT[c["u"]])
            # what the forward left: the stream it wrote and its rows' statistics
            s["h"], _, s["stats"] = _plain_norm_fwd(s)
            if own:
                from bitwise_reproducible_int8_gb300 import repro as R
                s["ws"] = _ws(R.repro_block_norm_bwd_ws_bytes(n, D))
    elif op == "quant":
        s["x"] = _randn(g, c["n"], c["D"], std=1.0 if not c["columns"] else 1e-3, dtype=DT[c["x"]])
        s["mul"] = _scales(g, c["n"] if c["columns"] else c["D"], 1.0) if c["mul"] else None
        if own:
            from bitwise_reproducible_int8_gb300 import repro as R
            s["ws"] = _ws(R.repro_quant_rows_i8_ws_bytes(c["n"], c["D"], columns=c["columns"]))
    elif op == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        for nm, rows, t in (("a", M, c["ta"]), ("b", N, c["tb"])):
            # codes of normal values at 3.5 deviations over 127
            q = _randn(g, *((K, rows) if t else (rows, K)), std=127.0 / 3.5)
            s[nm] = q.round_().clamp_(-127, 127).to(torch.int8)
            del q
        s["s_a"], s["s_b"] = _scales(g, M, 1.0), _scales(g, N, 0.02)
        s["y0"] = _randn(g, M, N, std=1.0) if c["accumulate"] else None
        if own:
            from bitwise_reproducible_int8_gb300 import repro as R
            s["ws"] = _ws(R.repro_matmul_i8_ws_bytes(M, N, K, trans_a=c["ta"], trans_b=c["tb"]))
    else:
        n, F = c["n"], c["F"]
        gu = _randn(g, n, 2 * F, dtype=DT[c["x"]])
        if op == "swiglu_fwd":
            s["gu"] = gu
        else:
            s["da"] = _randn(g, n, F, std=1e-3, dtype=DT[c["a"]])
            s["codes"], s["scales"] = _plain_keep(c, gu)
    return s


# ------------------------------------------------------------------ the plain forms

def _rms(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _plain_norm_fwd(s):
    c = s["case"]
    t, h, r1 = DT[c["x"]], s["x"].float(), None
    if c["y"]:
        p = s["y"].float()
        if c["post"]:
            r1 = _rms(p)
            p = p * r1 * s["g_post"]
        if s["gate"] is not None:
            p = p * s["gate"].float()
        h = (c["alpha"] * h + c["beta"] * p).to(t).float()     # the norm reads the stream as it is stored
    r2 = _rms(h)
    u = (h * r2 * s["g_pre"]).to(DT[c["u"]])
    stats = torch.cat([torch.zeros_like(r2) if r1 is None else r1, r2], 1)
    return [h.to(t), u, stats]


def _plain_norm_bwd(s):
    c = s["case"]
    t = DT[c["x"]]
    r1, r2 = s["stats"][:, :1], s["stats"][:, 1:]
    out = []
    du, hh = s["du"].float(), s["h"].float() * r2
    dg_pre = (du * hh).double().sum(0).float()
    v = du * s["g_pre"]
    dh = s["dh"].float() + r2 * (v - hh * (v * hh).mean(-1, keepdim=True))
    out.append((c["alpha"] * dh).to(t))
    if c["y"]:
        y, db = s["y"].float(), c["beta"] * dh
        yh = y * r1 if c["post"] else y
        p = yh * s["g_post"] if c["post"] else y
        dp = db
        dgate = dg_post = None
        if s["gate"] is not None:
            dgate = (db * p).double().sum(0).float() if c["gate"] == "channel" else (db * p).to(t)
            dp = db * s["gate"].float()
        if c["post"]:
            dg_post = (dp * yh).double().sum(0).float()
            w = dp * s["g_post"]
            dp = r1 * (w - yh * (w * yh).mean(-1, keepdim=True))
        out += [dp.to(t)] + [x for x in (dgate, dg_post) if x is not None]
    return out + [dg_pre]


def _codes(x, s):
    """x over its steps s, to the nearest whole number (ties to even); steps of 0 give 0."""
    q = torch.where(s > 0, x / torch.where(s > 0, s, 1.0), 0.0)
    return q.round_().clamp_(-127, 127).to(torch.int8)


def _plain_quant(s):
    c = s["case"]
    x = s["x"].float()
    if c["mul"]:
        x = x * (s["mul"][:, None] if c["columns"] else s["mul"])
    top = torch.full((1,), 127.0, device="cuda")      # a tensor: a quotient, not a product by 1 / 127
    st = x.abs().amax(0 if c["columns"] else 1, keepdim=True) / top
    return [_codes(x, st), st.flatten()]


def _plain_matmul(s):
    c = s["case"]
    a, b = s["a"].float(), s["b"].float()
    y = (a.t() if c["ta"] else a) @ (b if c["tb"] else b.t())
    y = y * s["s_a"][:, None] * s["s_b"]
    return (y + s["y0"] if c["accumulate"] else y).to(DT[c["y"]])


def _plain_keep(c, gu):
    """Codes [n, 2, G, 128] and steps [n, 2, G] of the activation's inputs; the last group is filled up with 0."""
    n, F = c["n"], c["F"]
    G = _ceil_div(F, GROUP)
    x = torch.zeros((n, 2, G * GROUP), device="cuda")
    x[..., :F] = gu.view(n, 2, F)
    x = x.view(n, 2, G, GROUP)
    st = x.abs().amax(-1, keepdim=True) / torch.full((1,), 127.0, device="cuda")
    return _codes(x, st), st[..., 0].contiguous()


def _plain_swiglu_fwd(s):
    c = s["case"]
    g, u = (v.float() for v in s["gu"].view(c["n"], 2, c["F"]).unbind(1))
    a = (g / (1.0 + torch.exp(-g)) * u).to(DT[c["a"]])
    return [a, *_plain_keep(c, s["gu"])] if c["keep"] else [a]


def _plain_swiglu_bwd(s):
    c = s["case"]
    x = (s["codes"].float() * s["scales"][..., None]).flatten(2)[..., :c["F"]]
    g, u = x.unbind(1)
    da = s["da"].float()
    sg = 1.0 / (1.0 + torch.exp(-g))
    dg = da * u * sg * (1.0 + g * (1.0 - sg))
    return torch.stack([dg, da * (g * sg)], 1).flatten(1).to(DT[c["x"]])


# ------------------------------------------------------------------ the library's calls

def _own(s):
    from bitwise_reproducible_int8_gb300 import repro as R
    c, op = s["case"], s["case"]["op"]
    if op == "norm_fwd":
        h = torch.empty_like(s["x"]) if c["y"] else None
        u = torch.empty(s["x"].shape, dtype=DT[c["u"]], device="cuda")
        stats = torch.empty((c["n"], 2), device="cuda")
        R.repro_block_norm_fwd(s["x"], s["y"], h, u, stats=stats, gate=s["gate"], g_post=s["g_post"],
                               g_pre=s["g_pre"], post=c["post"], alpha=c["alpha"], beta=c["beta"], eps=EPS)
        return [h if c["y"] else s["x"], u, stats]
    if op == "norm_bwd":
        dx = torch.empty_like(s["h"])
        dy = torch.empty_like(s["h"]) if c["y"] else None
        dgate = torch.empty_like(s["gate"]) if s["gate"] is not None else None
        dg_post = torch.empty_like(s["g_post"]) if c["post"] else None
        dg_pre = torch.empty_like(s["g_pre"])
        R.repro_block_norm_bwd(s["dh"], s["du"], s["h"], s["y"], s["stats"], dx, dy, gate=s["gate"], dgate=dgate,
                               g_post=s["g_post"], g_pre=s["g_pre"], dg_post=dg_post, dg_pre=dg_pre,
                               post=c["post"], alpha=c["alpha"], beta=c["beta"], ws=s["ws"])
        return [v for v in (dx, dy, dgate, dg_post, dg_pre) if v is not None]
    if op == "quant":
        q = torch.empty(s["x"].shape, dtype=torch.int8, device="cuda")
        st = torch.empty(c["D"] if c["columns"] else c["n"], device="cuda")
        R.repro_quant_rows_i8(s["x"], q, st, mul=s["mul"], columns=c["columns"], ws=s["ws"])
        return [q, st]
    if op == "matmul":
        y = s["y0"].clone() if c["accumulate"] else torch.empty((c["M"], c["N"]), dtype=DT[c["y"]], device="cuda")
        R.repro_matmul_i8(s["a"], s["b"], y, s_a=s["s_a"], s_b=s["s_b"], trans_a=c["ta"], trans_b=c["tb"],
                          accumulate=c["accumulate"], ws=s["ws"])
        return y
    n, F = c["n"], c["F"]
    if op == "swiglu_fwd":
        a = torch.empty((n, F), dtype=DT[c["a"]], device="cuda")
        if not c["keep"]:
            R.repro_swiglu_fwd(s["gu"], a)
            return [a]
        G = _ceil_div(F, GROUP)
        codes = torch.empty((n, 2, G, GROUP), dtype=torch.int8, device="cuda")
        scales = torch.empty((n, 2, G), device="cuda")
        R.repro_swiglu_fwd(s["gu"], a, codes, scales)
        return [a, codes, scales]
    dgu = torch.empty((n, 2 * F), dtype=DT[c["x"]], device="cuda")
    R.repro_swiglu_bwd(s["da"], dgu, codes=s["codes"], scales=s["scales"])
    return dgu


_PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "quant": _plain_quant, "matmul": _plain_matmul,
          "swiglu_fwd": _plain_swiglu_fwd, "swiglu_bwd": _plain_swiglu_bwd}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ the work

def work(case):
    c, op = case, case["op"]
    if op.startswith("norm"):
        e, x, u = c["n"] * c["D"], SIZE[c["x"]], SIZE[c["u"]]
        gate = e * x if c["gate"] == "token" else 4 * c["D"] if c["gate"] == "channel" else 0
        gains = 4 * c["D"] * (2 if c["post"] else 1)
        if op == "norm_fwd":    # the stream and the block's output in, the stream and the normed stream out
            return {"bytes": e * (x + (2 * x if c["y"] else 0) + u) + 8 * c["n"] + gate + gains, "flops": 10 * e}
        b = e * (x + u + x + x + (2 * x if c["y"] else 0)) + 8 * c["n"] + 2 * (gate + gains)
        return {"bytes": b, "flops": 20 * e}
    if op == "quant":
        e, rows, mul = c["n"] * c["D"], c["n"], c["D"]
        if c["columns"]:
            rows, mul = mul, rows
        return {"bytes": e * (SIZE[c["x"]] + 1) + 4 * rows + (4 * mul if c["mul"] else 0), "flops": 3 * e}
    if op == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        out = M * N * SIZE[c["y"]] * (2 if c["accumulate"] else 1)
        return {"bytes": M * K + N * K + out + 4 * (M + N), "flops": 2 * M * N * K}
    e = c["n"] * c["F"]
    kept = c["n"] * 2 * c["F"] + c["n"] * 2 * _ceil_div(c["F"], GROUP) * 4
    b = e * (2 * SIZE[c["x"]] + SIZE[c["a"]])
    if op == "swiglu_bwd" or c["keep"]:
        b += kept
    return {"bytes": b, "flops": e * (12 if op == "swiglu_fwd" else 16)}


# ------------------------------------------------------------------ the definitions in 64 bits

def _by_rows(n, width, f):
    """f over slices of the rows, so that the 64-bit copies stay small; its results end to end."""
    step = max(1, (1 << 26) // width)
    parts = [f(slice(lo, min(n, lo + step))) for lo in range(0, n, step)]
    return [torch.cat(p) for p in zip(*parts)]


def _unit(v):
    """(rows over their root mean square, the reciprocal of that)."""
    inv = (torch.einsum("nd,nd->n", v, v) / v.shape[1] + EPS).pow(-0.5)
    return v * inv[:, None], inv


def _exact_norm_fwd(c, s):
    gate = s["gate"]

    def part(r):
        h, post = s["x"][r].double(), torch.zeros(len(range(*r.indices(c["n"]))), dtype=torch.float64, device="cuda")
        if c["y"]:
            b = s["y"][r].double()
            if c["post"]:
                b, post = _unit(b)
                b = b * s["g_post"].double()
            if gate is not None:
                b = b * (gate if c["gate"] == "channel" else gate[r]).double()
            h = torch.add(h * c["alpha"], b, alpha=c["beta"]).to(DT[c["x"]]).double()
        nh, pre = _unit(h)
        return h, nh * s["g_pre"].double(), torch.stack([post, pre], 1)

    return _by_rows(c["n"], c["D"], part)


def _through_norm(d, unit, inv):
    """The gradient d of a row over its root mean square, taken back to the row."""
    along = torch.einsum("nd,nd->n", d, unit) / d.shape[1]
    return inv[:, None] * (d - unit * along[:, None])


def _exact_norm_bwd(c, s):
    z = lambda: torch.zeros(c["D"], dtype=torch.float64, device="cuda")  # noqa: E731
    sums = {"gate": z(), "post": z(), "pre": z()}

    def part(r):
        st = s["stats"][r].double()
        d, u = s["du"][r].double(), s["h"][r].double() * st[:, 1:]
        sums["pre"] += torch.einsum("nd,nd->d", d, u)
        dh = s["dh"][r].double() + _through_norm(d * s["g_pre"].double(), u, st[:, 1])
        got = [dh * c["alpha"]]
        if c["y"]:
            y, d = s["y"][r].double(), dh * c["beta"]
            unit = y * st[:, :1]
            rows = []
            if s["gate"] is not None:
                out = unit * s["g_post"].double() if c["post"] else y
                if c["gate"] == "channel":
                    sums["gate"] += torch.einsum("nd,nd->d", d, out)
                    d = d * s["gate"].double()
                else:
                    rows.append(d * out)
                    d = d * s["gate"][r].double()
            if c["post"]:
                sums["post"] += torch.einsum("nd,nd->d", d, unit)
                d = _through_norm(d * s["g_post"].double(), unit, st[:, 0])
            got += [d] + rows
        return got

    got = _by_rows(c["n"], c["D"], part)
    if c["gate"] == "channel":
        got.append(sums["gate"])
    if c["post"]:
        got.append(sums["post"])
    return got + [sums["pre"]]


def _exact_codes(v, st):
    """The quotient is rounded to 32 bits and then to a whole number."""
    q = (v / st).to(torch.float32).double().masked_fill(st == 0, 0.0)
    return torch.round(q).clamp(-127, 127).to(torch.int8)


def _exact_quant(c, s):
    if not c["columns"]:
        def part(r):
            v = s["x"][r].double()
            v = (v * s["mul"].double()).to(torch.float32).double() if c["mul"] else v
            st = (v.abs().max(1, keepdim=True).values / 127.0).to(torch.float32).double()
            return _exact_codes(v, st), st[:, 0]
        return _by_rows(c["n"], c["D"], part)
    v = s["x"].double()
    if c["mul"]:
        v = (v * s["mul"].double()[:, None]).to(torch.float32).double()
    st = (v.abs().max(0).values / 127.0).to(torch.float32).double()
    return [_exact_codes(v, st), st]


def _exact_matmul(c, s):
    a, b = s["a"].double(), s["b"].double()
    y = torch.einsum("km,kn->mn" if c["ta"] and c["tb"] else "mk,kn->mn" if c["tb"] else "mk,nk->mn", a, b)
    y *= torch.outer(s["s_a"].double(), s["s_b"].double())
    return y.add_(s["y0"]) if c["accumulate"] else y


def _exact_swiglu_fwd(c, s):
    F = c["F"]

    def part(r):
        gu = s["gu"][r].double()
        got = [torch.nn.functional.logsigmoid(gu[:, :F]).exp() * gu[:, :F] * gu[:, F:]]
        if c["keep"]:
            fill = _ceil_div(F, GROUP) * GROUP - F
            v = torch.nn.functional.pad(gu.reshape(-1, 2, F), (0, fill)).unflatten(2, (-1, GROUP))
            st = (v.abs().max(3).values / 127.0).to(torch.float32).double()
            got += [_exact_codes(v, st[..., None]), st]
        return got

    return _by_rows(c["n"], 2 * F, part)


def _exact_swiglu_bwd(c, s):
    F = c["F"]

    def part(r):
        kept = torch.einsum("nhgi,nhg->nhgi", s["codes"][r].double(), s["scales"][r].double())
        g, u = kept[:, 0].flatten(1)[:, :F], kept[:, 1].flatten(1)[:, :F]
        sg = torch.nn.functional.logsigmoid(g).exp()
        slope = sg + g * sg * torch.nn.functional.logsigmoid(-g).exp()
        d = s["da"][r].double()
        return [torch.cat([d * u * slope, d * g * sg], 1)]

    return _by_rows(c["n"], 2 * F, part)[0]


_EXACT = {"norm_fwd": _exact_norm_fwd, "norm_bwd": _exact_norm_bwd, "quant": _exact_quant, "matmul": _exact_matmul,
          "swiglu_fwd": _exact_swiglu_fwd, "swiglu_bwd": _exact_swiglu_bwd}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return _EXACT[case["op"]](case, s)
