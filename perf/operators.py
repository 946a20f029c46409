"""The operators around the decoder blocks of a training step, as they are measured.

Three pairs, each a forward and a backward call:

  embed    token embedding lookup with a scale, and the table's gradient
  qknorm   RMS norm of every query and key head followed by the position rotation
  distill  loss against a teacher's top logits (with the label's cross entropy and
           the log-partition penalty), and the logits' gradient

`own` False: plain torch operations.  `own` True: the library's calls.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6
THETA = 500000.0


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one 16,384-token micro-batch at the model width: the step's first call
        dict(name="embed_fwd_16k", op="embed_fwd", n=16384, V=32768, D=2048, table="f32", out="f32",
             scale=1.0, pad=False),
        # a ragged batch with padding, a quantised table, an odd width, narrow outputs
        dict(name="embed_fwd_i8_ragged", op="embed_fwd", n=4099, V=50001, D=1001, table="i8", out="bf16",
             scale=31.6, pad=True),
        # the micro-batch's gradient of the whole table
        dict(name="embed_bwd_16k", op="embed_bwd", n=16384, V=32768, D=2048, dout="f32", scale=1.0,
             pad=False, accumulate=False),
        # a short ragged batch added into an existing gradient: latency
        dict(name="embed_bwd_small_acc", op="embed_bwd", n=301, V=2003, D=1001, dout="bf16", scale=31.6,
             pad=True, accumulate=True),
        # the micro-batch's queries and keys, 4 x 4096 tokens, gainless, out of the fused projection
        dict(name="qknorm_fwd_16k", op="qknorm_fwd", B=4, T=4096, Hq=16, Hkv=4, D=128, R=128, x="f32",
             gain=False, interleaved=False, far=False),
        # one token at a far position: latency
        dict(name="qknorm_fwd_1tok", op="qknorm_fwd", B=1, T=1, Hq=16, Hkv=4, D=128, R=128, x="f32",
             gain=True, interleaved=False, far=True),
        # the micro-batch's backward with trained gains
        dict(name="qknorm_bwd_16k", op="qknorm_bwd", B=4, T=4096, Hq=16, Hkv=4, D=128, R=128, x="f32",
             gain=True, interleaved=False, far=False),
        # odd token count, narrow inputs, a partly rotated head of another width, neighbour pairs
        dict(name="qknorm_bwd_ragged", op="qknorm_bwd", B=1, T=1023, Hq=5, Hkv=1, D=80, R=40, x="bf16",
             gain=True, interleaved=True, far=True),
        # half a micro-batch of student logits, softened targets mixed with labels
        dict(name="distill_fwd_8k", op="distill_fwd", n=8192, V=32768, K=64, z="f32", tau=2.0, w_kd=0.9,
             w_ce=0.1, w_z=1e-4, logprobs=False),
        # few rows: the vocabulary has to be split over the card
        dict(name="distill_fwd_few", op="distill_fwd", n=5, V=50001, K=17, z="f32", tau=1.0, w_kd=1.0,
             w_ce=0.0, w_z=0.0, logprobs=True),
        # the gradient of the same half micro-batch at temperature one
        dict(name="distill_bwd_8k", op="distill_bwd", n=8192, V=32768, K=64, z="f32", tau=1.0, w_kd=0.9,
             w_ce=0.1, w_z=1e-4, logprobs=False),
        # narrow logits over a long, odd vocabulary, softened
        dict(name="distill_bwd_bf16_ragged", op="distill_bwd", n=1021, V=130001, K=33, z="bf16", tau=1.5,
             w_kd=1.0, w_ce=0.0, w_z=0.0, logprobs=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "qknorm_fwd", "qknorm_bwd", "distill_fwd", "distill_bwd"])
    if op.startswith("embed"):
        V = _log_int(rng, 500, 60000)
        D = rng.choice([_log_int(rng, 33, 2048), 8 * _log_int(rng, 8, 256)])
        n = _log_int(rng, 1, 16384)
        c = dict(op=op, n=n, V=V, D=D, scale=rng.choice([1.0, round(math.sqrt(D), 3)]),
                 pad=rng.random() < 0.5)
        if op == "embed_fwd":
            c.update(table=rng.choice(["f32", "bf16", "i8"]), out=rng.choice(["f32", "f32", "bf16"]))
        else:
            c.update(dout=rng.choice(["f32", "f32", "bf16"]), accumulate=rng.random() < 0.4)
        return c
    if op.startswith("qknorm"):
        D = rng.choice([32, 64, 80, 96, 128, 128, 192, 256, 2 * rng.randint(8, 128)])
        R = D if rng.random() < 0.6 else 2 * rng.randint(1, D // 2)
        G = rng.choice([1, 2, 4, 5])
        Hkv = rng.choice([1, 2, 4])
        B = rng.choice([1, 1, 2, 3])
        most = 4 * 4096 * 20 * 128 // (B * (G + 1) * Hkv * D)
        return dict(op=op, B=B, T=_log_int(rng, 1, max(1, min(16384, most))), Hq=G * Hkv, Hkv=Hkv, D=D, R=R,
                    x=rng.choice(["f32", "f32", "bf16"]), gain=rng.random() < 0.5,
                    interleaved=rng.random() < 0.4, far=rng.random() < 0.5)
    V = _log_int(rng, 100, 140000)
    n = _log_int(rng, 1, max(1, min(16384, 8192 * 32768 // V)))
    K = min(V // 2, rng.randint(1, 100))
    ce = rng.random() < 0.5
    return dict(op=op, n=n, V=V, K=K, z=rng.choice(["f32", "f32", "bf16"]),
                tau=rng.choice([1.0, 1.0, 1.5, 2.0, 4.0]), w_kd=0.9 if ce else 1.0, w_ce=0.1 if ce else 0.0,
                w_z=1e-4 if rng.random() < 0.5 else 0.0, logprobs=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    t = torch.empty(shape, device="cuda", dtype=torch.float32)
    t.normal_(0.0, std, generator=g)
    return t.to(dtype)


def _zipf(V):
    """Token frequencies of text: the r-th most frequent token goes like 1 / (r + 2)."""
    p = 1.0 / (np.arange(V, dtype=np.float64) + 2.0)
    return p / p.sum()


def _tokens(g, n, V, pad):
    cdf = torch.from_numpy(np.cumsum(_zipf(V))).cuda()
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.searchsorted(cdf, u).clamp_(max=V - 1)
    names = torch.randperm(V, generator=g, device="cuda")
    tok = names[rank]
    if pad:   # the end of the batch is filled up with the padding token 0
        tok[n - n // 8:] = 0
    return tok


def _rope(P, R):
    """[P, R] cosines then sines of position * THETA^(-2j / R), rounded once."""
    j = torch.arange(R // 2, dtype=torch.float64, device="cuda")
    ang = torch.arange(P, dtype=torch.float64, device="cuda")[:, None] * torch.pow(THETA, -2.0 * j / R)[None]
    return torch.cat([torch.cos(ang), torch.sin(ang)], 1).float()


def prepare(case, seed):
    c, g, op = case, _gen(seed), case["op"]
    s = {"case": dict(case)}
    if op.startswith("embed"):
        n, V, D = c["n"], c["V"], c["D"]
        s["tokens"] = _tokens(g, n, V, c["pad"])
        if op == "embed_fwd":
            if c["table"] == "i8":
                s["table"] = torch.randint(-127, 128, (V, D), generator=g, device="cuda", dtype=torch.int8)
                s["s_w"] = torch.rand(1, generator=g, device="cuda") * 1e-3 + 1e-3
            else:
                s["table"] = _randn(g, V, D, std=0.02, dtype=DT[c["table"]])
                s["s_w"] = None
        else:
            s["dout"] = _randn(g, n, D, std=1e-3, dtype=DT[c["dout"]])
            s["grad"] = _randn(g, V, D, std=1e-3) if c["accumulate"] else None
            if own:
                from bitwise_reproducible_int8_gb300 import repro as R
                s["ws"] = torch.empty(max(R.repro_embed_bwd_ws_bytes(n, V, D), 16), dtype=torch.uint8,
                                      device="cuda")
    elif op.startswith("qknorm"):
        B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
        # queries, keys and values side by side, as the fused projection leaves them
        qkv = _randn(g, B, T, (Hq + 2 * Hkv) * D, std=1.3, dtype=DT[c["x"]])
        s["qkv"] = qkv
        off = 120000 if c["far"] else 0
        s["positions"] = (torch.arange(T, device="cuda", dtype=torch.int32) + off).repeat(B)
        s["rope"] = _rope(off + T, c["R"])
        for nm, H in (("q", Hq), ("k", Hkv)):
            s["g_" + nm] = 1.0 + _randn(g, D, std=0.1) if c["gain"] else None
            if op == "qknorm_bwd":
                s["do_" + nm] = _randn(g, B, T, H, D, std=1e-3)
        if own and op == "qknorm_bwd":
            from bitwise_reproducible_int8_gb300 import repro as R
            s["ws"] = torch.empty(max(R.repro_qk_norm_rope_bwd_ws_bytes(B * T, Hq, Hkv, D), 16),
                                  dtype=torch.uint8, device="cuda")
    else:
        n, V, K = c["n"], c["V"], c["K"]
        # K distinct columns a row; the teacher's logits fall off from the first on
        start = torch.randint(0, V, (n, 1), generator=g, device="cuda")
        step = max(1, V // K)
        idx = (start + torch.arange(K, device="cuda")[None] * step) % V
        t = 11.0 - 1.6 * torch.log(torch.arange(K, device="cuda", dtype=torch.float32) + 1.0)[None]
        t = t + _randn(g, n, K, std=0.5)
        z = _randn(g, n, V, std=1.5)
        z.scatter_(1, idx, t + _randn(g, n, K, std=0.7))
        # a few rows have fewer teacher entries than the others
        short = torch.rand(n, 1, generator=g, device="cuda") < 0.1
        idx = torch.where(short & (torch.arange(K, device="cuda")[None] >= (K + 1) // 2), -1, idx)
        if c["logprobs"]:   # the teacher's own log-probabilities: the listed ones hold part of the mass
            t = t - torch.logsumexp(t, 1, keepdim=True) - 0.2
        s["t_idx"], s["t_logits"] = idx.to(torch.int32), t
        lab = idx[:, 0].clone()
        lab[torch.rand(n, generator=g, device="cuda") < 0.05] = -100
        s["labels"] = lab.to(torch.int32) if c["w_ce"] else None
        s["logits"] = z.to(DT[c["z"]])
        del z
        if op == "distill_bwd":
            s["g"] = torch.full((1,), 1.0 / n, device="cuda")
        if own:
            from bitwise_reproducible_int8_gb300 import repro as R
            s["ws"] = torch.empty(max(R.repro_distill_ws_bytes(n, V), 16), dtype=torch.uint8, device="cuda")
            s["hp"] = dict(tau=c["tau"], w_kd=c["w_kd"], w_ce=c["w_ce"], w_z=c["w_z"], logprobs=c["logprobs"])
            if op == "distill_bwd":   # the forward's row statistics, kept for the backward
                s["stats"] = torch.empty((n, R.REPRO_DISTILL_STATS + K), device="cuda")
                R.repro_distill_fwd(s["logits"], s["t_idx"], s["t_logits"], torch.empty(n, device="cuda"),
                                    s["stats"], labels=s["labels"], ws=s["ws"], **s["hp"])
        elif op == "distill_bwd":
            s["stats"] = _plain_stats(c, s)
    return s


# ------------------------------------------------------------------ the plain forms

def _split(case, qkv):
    B, T, Hq, Hkv, D = (case[k] for k in ("B", "T", "Hq", "Hkv", "D"))
    x = qkv.view(B, T, Hq + 2 * Hkv, D)
    return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]


def _pairs(x, R, interleaved):
    if interleaved:
        return x[..., 0:R:2], x[..., 1:R:2]
    return x[..., :R // 2], x[..., R // 2:R]


def _unpair(a, b, rest, interleaved):
    ab = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([ab, rest], -1)


def _cos_sin(s):
    c = s["case"]
    rows = s["rope"][s["positions"].long()].view(c["B"], c["T"], 1, c["R"])
    return rows[..., :c["R"] // 2], rows[..., c["R"] // 2:]


def _plain_qknorm_fwd(s):
    c, out = s["case"], []
    cos, sin = _cos_sin(s)
    for x, g in zip(_split(c, s["qkv"]), (s["g_q"], s["g_k"])):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        if g is not None:
            y = y * g
        a, b = _pairs(y, c["R"], c["interleaved"])
        out.append(_unpair(a * cos - b * sin, b * cos + a * sin, y[..., c["R"]:], c["interleaved"]))
    return out


def _plain_qknorm_bwd(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    dxs, dgs = [], []
    for x, g, do in zip(_split(c, s["qkv"]), (s["g_q"], s["g_k"]), (s["do_q"], s["do_k"])):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xh = x * r
        a, b = _pairs(do, c["R"], c["interleaved"])
        dy = _unpair(a * cos + b * sin, b * cos - a * sin, do[..., c["R"]:], c["interleaved"])
        if g is not None:
            dgs.append((dy * xh).double().sum((0, 1, 2)).float())
            dy = dy * g
        dx = r * (dy - xh * (dy * xh).mean(-1, keepdim=True))
        dxs.append(dx.to(DT[c["x"]]))
    return dxs + dgs


def _plain_embed_fwd(s):
    c, tok = s["case"], s["tokens"]
    y = s["table"][tok].float()
    if s["s_w"] is not None:
        y = y * s["s_w"]
    y = y * c["scale"]
    if c["pad"]:
        y = torch.where((tok == 0)[:, None], 0.0, y)
    return y.to(DT[c["out"]])


def _plain_embed_bwd(s):
    c, tok = s["case"], s["tokens"]
    d = s["dout"].double()
    if c["pad"]:
        d = torch.where((tok == 0)[:, None], 0.0, d)
    w = torch.zeros(c["V"], c["D"], device="cuda", dtype=torch.float64).index_add_(0, tok, d) * c["scale"]
    return (w + s["grad"] if c["accumulate"] else w).float()


def _plain_teacher(c, s):
    """The teacher's weights (0 where an entry is padding) and the columns they stand for."""
    ok = s["t_idx"] >= 0
    t = torch.where(ok, s["t_logits"].float(), -math.inf)
    if c["logprobs"]:
        logp = t
    else:
        t = t / c["tau"]
        m = t.max(1, keepdim=True).values
        logp = t - (m + torch.log(torch.exp(t - m).sum(1, keepdim=True)))
    return ok, torch.where(ok, torch.exp(logp), 0.0), logp, s["t_idx"].clamp(min=0).long()


def _lse(u):
    m = u.max(1, keepdim=True).values
    return m + torch.log(torch.exp(u - m).sum(1, keepdim=True))


def _plain_stats(c, s):
    z = s["logits"].float()
    return _lse(z / c["tau"]), _lse(z)


def _plain_distill_fwd(s):
    c = s["case"]
    ok, p, logp, idx = _plain_teacher(c, s)
    z = s["logits"].float()
    lse_t = _lse(z / c["tau"])
    logq = torch.gather(z, 1, idx) / c["tau"] - lse_t
    kd = torch.where(p > 0, p * (logp - logq), 0.0).sum(1)
    loss = c["w_kd"] * c["tau"] ** 2 * kd
    if c["w_ce"] or c["w_z"]:
        lse = _lse(z)
        if c["w_ce"]:
            lab = s["labels"].long()
            ce = lse[:, 0] - torch.gather(z, 1, lab.clamp(min=0)[:, None])[:, 0]
            loss = loss + c["w_ce"] * torch.where(lab >= 0, ce, 0.0)
        loss = loss + c["w_z"] * lse[:, 0] ** 2
    return [loss, lse_t[:, 0]]


def _plain_distill_bwd(s):
    c = s["case"]
    ok, p, logp, idx = _plain_teacher(c, s)
    z, (lse_t, lse) = s["logits"].float(), s["stats"]
    w = c["w_kd"] * c["tau"]
    dz = torch.exp(z / c["tau"] - lse_t) * (w * p.sum(1, keepdim=True))
    dz.scatter_add_(1, idx, -w * p)
    if c["w_ce"] or c["w_z"]:
        coef = 2.0 * c["w_z"] * lse
        if c["w_ce"]:
            hit = (s["labels"] >= 0).float()[:, None]
            coef = coef + c["w_ce"] * hit
        dz += torch.exp(z - lse) * coef
        if c["w_ce"]:
            dz.scatter_add_(1, s["labels"].clamp(min=0).long()[:, None], -c["w_ce"] * hit)
    return (dz * s["g"]).to(DT[c["z"]])


# ------------------------------------------------------------------ the library's calls

def _own(s):
    from bitwise_reproducible_int8_gb300 import repro as R
    c, op, dev = s["case"], s["case"]["op"], "cuda"
    if op == "embed_fwd":
        out = torch.empty((c["n"], c["D"]), dtype=DT[c["out"]], device=dev)
        R.repro_embed_fwd(s["table"], s["tokens"], out, scale=c["scale"], s_w=s["s_w"],
                          pad=0 if c["pad"] else -1)
        return out
    if op == "embed_bwd":
        dw = s["grad"].clone() if c["accumulate"] else torch.empty((c["V"], c["D"]), device=dev)
        R.repro_embed_bwd(s["dout"], s["tokens"], dw, scale=c["scale"], pad=0 if c["pad"] else -1,
                          accumulate=c["accumulate"], ws=s["ws"])
        return dw
    if op.startswith("qknorm"):
        q, k = _split(c, s["qkv"])
        kw = dict(g_q=s["g_q"], g_k=s["g_k"], positions=s["positions"], eps=EPS, interleaved=c["interleaved"])
        if op == "qknorm_fwd":
            qo = torch.empty(q.shape, dtype=torch.float32, device=dev)
            ko = torch.empty(k.shape, dtype=torch.float32, device=dev)
            R.repro_qk_norm_rope_fwd(q, k, s["rope"], qo, ko, **kw)
            return [qo, ko]
        dq, dk = torch.empty(q.shape, dtype=q.dtype, device=dev), torch.empty(k.shape, dtype=k.dtype, device=dev)
        dg = [torch.empty(c["D"], device=dev) if c["gain"] else None for _ in range(2)]
        R.repro_qk_norm_rope_bwd(s["do_q"], s["do_k"], q, k, s["rope"], dq, dk, dg_q=dg[0], dg_k=dg[1],
                                 ws=s["ws"], **kw)
        return [dq, dk] + (dg if c["gain"] else [])
    if op == "distill_fwd":
        loss = torch.empty(c["n"], device=dev)
        stats = torch.empty((c["n"], R.REPRO_DISTILL_STATS + c["K"]), device=dev)
        R.repro_distill_fwd(s["logits"], s["t_idx"], s["t_logits"], loss, stats, labels=s["labels"],
                            ws=s["ws"], **s["hp"])
        return [loss, stats[:, R.REPRO_DISTILL_STAT_LSE]]
    dz = torch.empty_like(s["logits"])
    R.repro_distill_bwd(s["logits"], s["t_idx"], s["stats"], s["g"], dz, labels=s["labels"], **s["hp"])
    return dz


_PLAIN = {"embed_fwd": _plain_embed_fwd, "embed_bwd": _plain_embed_bwd, "qknorm_fwd": _plain_qknorm_fwd,
          "qknorm_bwd": _plain_qknorm_bwd, "distill_fwd": _plain_distill_fwd, "distill_bwd": _plain_distill_bwd}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ the work

_SIZE = {"f32": 4, "bf16": 2, "i8": 1}


def _distinct(n, V):
    """Distinct tokens to be expected among n."""
    return float((1.0 - np.power(1.0 - _zipf(V), n)).sum())


def work(case):
    c, op = case, case["op"]
    if op == "embed_fwd":
        rows = _distinct(c["n"], c["V"])
        return {"bytes": rows * c["D"] * _SIZE[c["table"]] + c["n"] * (8 + c["D"] * _SIZE[c["out"]]),
                "flops": c["n"] * c["D"]}
    if op == "embed_bwd":
        b = c["n"] * (8 + c["D"] * _SIZE[c["dout"]])
        # the table's gradient is written whole; one that is added to is read as well
        b += c["V"] * c["D"] * 4 * (2 if c["accumulate"] else 1)
        return {"bytes": b, "flops": c["n"] * c["D"]}
    if op.startswith("qknorm"):
        n, H = c["B"] * c["T"], c["Hq"] + c["Hkv"]
        e = n * H * c["D"]
        per = _SIZE[c["x"]] + 4 if op == "qknorm_fwd" else 2 * _SIZE[c["x"]] + 4
        gains = (4 * c["D"] * (2 if op == "qknorm_fwd" else 4)) if c["gain"] else 0
        return {"bytes": e * per + c["T"] * c["R"] * 4 + n * 4 + gains,
                "flops": e * (8 if op == "qknorm_fwd" else 16)}
    n, V, K = c["n"], c["V"], c["K"]
    e = n * V
    two = 2 if c["tau"] != 1.0 and (c["w_ce"] or c["w_z"]) else 1
    b = e * _SIZE[c["z"]] * (1 if op == "distill_fwd" else 2) + n * K * 8 + n * 8
    return {"bytes": b, "flops": e * (3 if op == "distill_fwd" else 4) * two}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_qknorm(case, s):
    """Heads as rows of a matrix; the rotation as a complex product."""
    c = case
    n, D, R = c["B"] * c["T"], c["D"], c["R"]
    tab = s["rope"].double()[s["positions"].long()]
    w = torch.complex(tab[:, :R // 2], tab[:, R // 2:])[:, None, :]

    def rotate(v, w):
        v = v.clone()
        ia = torch.arange(R // 2, device="cuda") * (2 if c["interleaved"] else 1)
        ib = ia + (1 if c["interleaved"] else R // 2)
        r = torch.complex(v[..., ia], v[..., ib]) * w
        v[..., ia], v[..., ib] = r.real, r.imag
        return v

    res, gains = [], []
    lo = 0
    x_all = s["qkv"].view(n, -1)
    for nm, H in (("q", c["Hq"]), ("k", c["Hkv"])):
        x = x_all[:, lo:lo + H * D].double().view(n, H, D)
        lo += H * D
        g = s["g_" + nm].double() if c["gain"] else torch.ones(D, dtype=torch.float64, device="cuda")
        inv = 1.0 / torch.sqrt(torch.einsum("nhd,nhd->nh", x, x) / D + EPS)[..., None]
        if c["op"] == "qknorm_fwd":
            res.append(rotate(x * inv * g, w).view(c["B"], c["T"], H, D))
            continue
        dy = rotate(s["do_" + nm].double().view(n, H, D), w.conj())
        if c["gain"]:
            gains.append(torch.einsum("nhd,nhd->d", dy, x * inv))
        dn = dy * g
        dx = inv * dn - x * inv ** 3 * torch.einsum("nhd,nhd->nh", dn, x)[..., None] / D
        res.append(dx.view(c["B"], c["T"], H, D))
    return res + gains


def _exact_embed(case, s):
    c, tok = case, s["tokens"]
    if c["op"] == "embed_fwd":
        f = c["scale"] * (1.0 if s["s_w"] is None else s["s_w"].double())
        y = torch.index_select(s["table"], 0, tok).double() * f
        if c["pad"]:
            y[tok == 0] = 0.0
        return y
    d = s["dout"].double()
    order = torch.argsort(tok, stable=True)
    sums = torch.zeros(c["n"] + 1, c["D"], dtype=torch.float64, device="cuda")
    count = torch.bincount(tok, minlength=c["V"])
    end = torch.cumsum(count, 0)
    # segments as differences of running sums: 64 bits hold them far below a binary32 step
    torch.cumsum(d[order], 0, out=sums[1:])
    w = (sums[end] - sums[end - count]) * c["scale"]
    if c["pad"]:
        w[0] = 0.0
    return w + s["grad"].double() if c["accumulate"] else w


def _exact_distill(case, s):
    c = case
    n, tau, out, part = c["n"], c["tau"], [], []
    need = c["w_ce"] != 0.0 or c["w_z"] != 0.0
    step = max(1, (1 << 27) // c["V"])
    for lo in range(0, n, step):
        rows = slice(lo, min(n, lo + step))
        z = s["logits"][rows].double()
        idx, t = s["t_idx"][rows].long(), s["t_logits"][rows].double()
        logp = t if c["logprobs"] else torch.log_softmax((t / tau).masked_fill(idx < 0, -math.inf), 1)
        p = logp.exp().masked_fill(idx < 0, 0.0)
        here = idx.clamp(min=0)
        logq = torch.log_softmax(z / tau, 1)
        lse = torch.logsumexp(z, 1) if need else None
        lab = s["labels"][rows].long() if c["w_ce"] else None
        if c["op"] == "distill_fwd":
            d = (logp - logq.gather(1, here)).masked_fill(idx < 0, 0.0)
            loss = c["w_kd"] * tau * tau * (p * d).sum(1)
            if lab is not None:
                ce = lse - z.gather(1, lab.clamp(min=0)[:, None]).squeeze(1)
                loss += c["w_ce"] * ce * (lab >= 0)
            if c["w_z"]:
                loss += c["w_z"] * lse.square()
            out.append(loss)
            part.append(torch.logsumexp(z / tau, 1))
            continue
        dz = logq.exp_().mul_(p.sum(1, keepdim=True)).scatter_add_(1, here, -p).mul_(c["w_kd"] * tau)
        if need:
            k = torch.full_like(lse, 0.0)
            if lab is not None:
                k = k + c["w_ce"] * (lab >= 0)
            k = k + 2.0 * c["w_z"] * lse
            dz.addcmul_(torch.softmax(z, 1), k[:, None])
            if lab is not None:
                dz.scatter_add_(1, lab.clamp(min=0)[:, None], -c["w_ce"] * (lab >= 0).double()[:, None])
        out.append(dz.mul_(s["g"].double()))
    return [torch.cat(out), torch.cat(part)] if part else torch.cat(out)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"].startswith("embed"):
        return _exact_embed(case, s)
    if case["op"].startswith("qknorm"):
        return _exact_qknorm(case, s)
    return _exact_distill(case, s)
