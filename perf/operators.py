"""The operators beside the quantized head, as cases to measure and check.

Embedding lookup from the packed table and its gradient, layer norm (and its
uncentred form) and its gradient, and the distillation loss of the head
against a teacher's top logits with its gradient into the hidden states.
`run` computes them in plain torch operations, or, with `own` set, through
the package's public calls.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6

# Table shapes are the ones the package's workloads use: V = 262144, H = 2560,
# 4-bit, soft cap 30, and V = 131072, H = 1536, 8-bit.
GEMMA = dict(V=262144, H=2560, bits=4)
MID8 = dict(V=131072, H=1536, bits=8)


def listed():
    return [
        # a verify window's 5 tokens enter the model: latency
        dict(name="embed_window", op="embed", M=5, out="bf16", scale=50.596, masked=False, **GEMMA),
        # a training batch of 8 sequences of 1024 tokens, prompt padding masked
        dict(name="embed_batch", op="embed", M=8192, out="bf16", scale=50.596, masked=True, **GEMMA),
        # a long prefill of an odd number of tokens into a float32 residual stream
        dict(name="embed_prefill_f32", op="embed", M=65537, out="f32", scale=1.0, masked=False, **MID8),
        # the embedding's gradient by itself: every row of dW is written
        dict(name="embed_grad", op="embed_bwd", M=8192, dy="bf16", scale=50.596, masked=True, add=False, **GEMMA),
        # tied table: added into the head's dW, float32 gradients of a long batch
        dict(name="embed_grad_tied", op="embed_bwd", M=32768, dy="f32", scale=1.0, masked=False, add=True, **MID8),
        # the final norm before the head: a verify window, and a float32 stream of odd width
        dict(name="norm_window", op="norm", M=5, H=2560, x="bf16", y="bf16", center=False, bias=False, pad=0),
        dict(name="norm_odd_f32", op="norm", M=20001, H=2563, x="f32", y="f32", center=True, bias=True, pad=5),
        # its gradient from the head's float32 dh, and in bf16 throughout
        dict(name="norm_grad", op="norm_bwd", M=8192, H=2560, x="bf16", y="f32", center=True, bias=True, pad=0),
        dict(name="norm_grad_long", op="norm_bwd", M=65536, H=1536, x="bf16", y="bf16", center=False, bias=False, pad=0),
        # distillation steps: a few rows, 512 rows of the capped 4-bit head,
        # and the 8-bit head's training batch with masked prompts
        dict(name="distill_few", op="distill", M=13, K=20, cap=30.0, temp=1.0, t="f32", masked=False, **GEMMA),
        dict(name="distill_512", op="distill", M=512, K=64, cap=30.0, temp=1.0, t="bf16", masked=False, **GEMMA),
        dict(name="distill_batch8", op="distill", M=8192, K=32, cap=0.0, temp=2.0, t="f32", masked=True, **MID8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_bwd", "norm", "norm_bwd", "distill", "distill"])
    c = dict(op=op)
    if op in ("norm", "norm_bwd"):
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            H = (H + 7) // 8 * 8
        c.update(H=H, M=_log_int(rng, 1, 100_000_000 // H), x=rng.choice(["bf16", "f16", "f32"]),
                 y=rng.choice(["bf16", "f32"]), center=rng.random() < 0.5, bias=rng.random() < 0.5,
                 pad=rng.choice([0, 0, 8, 3]))
        return c
    H = 128 * rng.randint(2, 20)
    c.update(H=H, bits=rng.choice([4, 8]))
    if op == "distill":
        c.update(V=_log_int(rng, 3000, 262144), K=_log_int(rng, 1, 128), cap=rng.choice([0.0, 30.0]),
                 temp=rng.choice([1.0, 1.0, 2.0, 3.5]), t=rng.choice(["f32", "bf16"]), masked=rng.random() < 0.5)
        c["M"] = _log_int(rng, 1, max(64, min(4096, 300_000_000_000 // (c["V"] * H))))
        return c
    c.update(V=_log_int(rng, 2000, 262144), M=_log_int(rng, 1, 32768), masked=rng.random() < 0.5,
             scale=rng.choice([1.0, round(math.sqrt(H), 3)]))
    if op == "embed":
        c.update(out=rng.choice(["bf16", "f32"]))
    else:
        c.update(dy=rng.choice(["bf16", "f32"]), add=rng.random() < 0.5)
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _table(c, g):
    """Uniform codes; scales and biases as the package's synthetic heads have them."""
    V, H, bits = c["V"], c["H"], c["bits"]
    wq = torch.randint(-2 ** 31, 2 ** 31, (V, H * bits // 32), device=DEV, generator=g, dtype=torch.int64).to(torch.int32)
    u = torch.rand(V, H // 64, device=DEV, generator=g)
    if bits == 4:
        s = 1e-3 + 9e-3 * u
        b = -8.0 * s + 1e-3 * torch.randn(V, H // 64, device=DEV, generator=g)
    else:
        s = 1e-4 + 9e-4 * u
        b = -128.0 * s
    return wq, s.half(), b.half()


def _tokens(c, g):
    """Token ids of a text: the id is the rank in frequency, frequency ~ 1 / rank."""
    u = torch.rand(c["M"], device=DEV, generator=g, dtype=torch.float64)
    return ((u * math.log(c["V"] + 1)).exp() - 1).long().clamp(0, c["V"] - 1).to(torch.int32)


def _mask(c):
    """Sequences of 1024 tokens whose first 307 are the prompt (off)."""
    if not c["masked"]:
        return None
    return (torch.arange(c["M"], device=DEV) % 1024 >= 307) | (c["M"] <= 307)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = dict(c=c)
    if c["op"] in ("norm", "norm_bwd"):
        M, H = c["M"], c["H"]
        # a residual stream: rows of their own size and offset, a few strong channels
        x = torch.randn(M, H + c["pad"], device=DEV, generator=g)
        x *= 0.5 + 2.0 * torch.rand(M, 1, device=DEV, generator=g)
        x += 0.3 * torch.randn(M, 1, device=DEV, generator=g)
        x[:, :: max(1, H // 4)] *= 8.0
        s["x"] = x.to(DT[c["x"]])[:, :H]
        s["w"] = (1.0 + 0.1 * torch.randn(H, device=DEV, generator=g)).to(DT[c["x"]])
        s["b"] = (0.1 * torch.randn(H, device=DEV, generator=g)).to(DT[c["x"]]) if c["bias"] else None
        if c["op"] == "norm_bwd":
            xf = s["x"].double()
            s["mean"] = xf.mean(1).float() if c["center"] else None
            xc = xf - xf.mean(1, keepdim=True) if c["center"] else xf
            s["rstd"] = (xc.square().mean(1) + EPS).rsqrt().float()
            s["dy"] = (1e-2 * torch.randn(M, H, device=DEV, generator=g)).to(DT[c["y"]])
        return s
    s["wq"], s["s"], s["b"] = _table(c, g)
    if c["op"] in ("embed", "embed_bwd"):
        s["tokens"], s["mask"] = _tokens(c, g), _mask(c)
        if c["op"] == "embed_bwd":
            s["dy"] = (1e-2 * torch.randn(c["M"], c["H"], device=DEV, generator=g)).to(DT[c["dy"]])
            s["dw"] = 1e-2 * torch.randn(c["V"], c["H"], device=DEV, generator=g) if c["add"] else None
        return s
    # A student near its teacher: the hidden state is a sum of the K tokens'
    # rows, so that their logits fall off like log-frequencies from a peak
    # that differs from row to row; the teacher's logits differ by noise.
    M, K, V = c["M"], c["K"], c["V"]
    K = min(K, V)
    stride = V // K
    ids = torch.arange(K, device=DEV) * stride + torch.randint(0, stride, (M, K), device=DEV, generator=g)
    ids = ids.gather(1, torch.rand(M, K, device=DEV, generator=g).argsort(1))
    peak = 12.0 + 6.0 * torch.rand(M, 1, device=DEV, generator=g)
    t = peak - 1.2 * torch.log1p(torch.arange(K, device=DEV).float()) + 0.3 * torch.randn(M, K, device=DEV, generator=g)
    # One row in eight kept fewer of the teacher's tokens (those that carry its
    # mass; -1 fills the row up), and the student gives the others none either.
    short = (torch.arange(M, device=DEV) % 8 == 7)[:, None] & (torch.arange(K, device=DEV) >= (K + 1) // 2)[None]
    rows = _dequant(s["wq"][ids.view(-1)], s["s"][ids.view(-1)], s["b"][ids.view(-1)], c["bits"]).view(M, K, -1)
    raw = t if c["cap"] <= 0 else c["cap"] * torch.atanh((t / c["cap"]).clamp(-0.9, 0.9))
    h = torch.einsum("mk,mkh->mh", (raw / rows.square().sum(2)).masked_fill(short, 0.0), rows)
    s["h"] = (h + 0.3 * h.std() * torch.randn(M, c["H"], device=DEV, generator=g)).to(torch.bfloat16)
    s["t"] = (t + 0.7 * torch.randn(M, K, device=DEV, generator=g)).to(DT[c["t"]])
    s["ids"] = ids.masked_fill(short, -1).to(torch.int32)
    s["mask"] = _mask(c)
    s["dloss"] = (0.5 + torch.rand(M, device=DEV, generator=g)) / M
    return s


# ------------------------------------------------------------------ plain forms

def _dequant(wq, sc, bi, bits):
    """Rows of packed codes -> float32 rows."""
    k = torch.arange(32 // bits, device=wq.device, dtype=torch.int32) * bits
    q = ((wq[:, :, None] >> k) & (2 ** bits - 1)).view(wq.shape[0], -1, 64).float()
    return (sc.float()[:, :, None] * q + bi.float()[:, :, None]).view(wq.shape[0], -1)


def _embed(s):
    c = s["c"]
    t = s["tokens"].long()
    y = _dequant(s["wq"][t], s["s"][t], s["b"][t], c["bits"]) * c["scale"]
    if s["mask"] is not None:
        y = y * s["mask"][:, None]
    return y.to(DT[c["out"]])


def _embed_bwd(s):
    c = s["c"]
    dy = s["dy"].float() * c["scale"]
    if s["mask"] is not None:
        dy = dy * s["mask"][:, None]
    dw = s["dw"] if c["add"] else torch.zeros(c["V"], c["H"], device=DEV)
    return dw.index_add_(0, s["tokens"], dy)


def _norm(s):
    c = s["c"]
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    xc = x - mean if c["center"] else x
    rstd = (xc.square().mean(1, keepdim=True) + EPS).rsqrt()
    y = xc * rstd * s["w"].float()
    if c["bias"]:
        y = y + s["b"].float()
    return {"y": y.to(DT[c["y"]]), "mean": mean[:, 0] if c["center"] else None, "rstd": rstd[:, 0]}


def _norm_bwd(s):
    c = s["c"]
    x, dy = s["x"].float(), s["dy"].float()
    rstd = s["rstd"][:, None]
    xh = (x - s["mean"][:, None] if c["center"] else x) * rstd
    g = dy * s["w"].float()
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if c["center"]:
        dx = dx - g.mean(1, keepdim=True)
    return {"dx": (dx * rstd).to(DT[c["x"]]), "dw": (dy * xh).sum(0), "db": dy.sum(0) if c["bias"] else None}


def _distill(s):
    c = s["c"]
    T, cap = c["temp"], c["cap"]
    W = _dequant(s["wq"], s["s"], s["b"], c["bits"])
    raw = s["h"].float() @ W.t()
    z = cap * torch.tanh(raw / cap) if cap > 0 else raw
    zs = z / T
    top = zs.amax(1, keepdim=True)
    lse = top + (zs - top).exp().sum(1, keepdim=True).log()
    has = s["ids"] >= 0
    ids = s["ids"].clamp_min(0).long()
    t = (s["t"].float() / T).masked_fill(~has, -math.inf)
    lp = t - t.amax(1, keepdim=True)
    lp = lp - lp.exp().sum(1, keepdim=True).log()
    p = lp.exp()
    zk = z.gather(1, ids)
    loss = (p * (lp - zk / T + lse)).masked_fill(~has, 0.0).sum(1)
    coef = (zs - lse).exp().scatter_add_(1, ids, -p)
    if cap > 0:
        coef = coef * (1.0 - (z / cap).square())
    gr = s["dloss"][:, None] / T
    lse = lse[:, 0]
    if s["mask"] is not None:
        loss, lse, gr = loss * s["mask"], lse * s["mask"], gr * s["mask"][:, None]
    return {"loss": loss, "lse": lse, "dh": ((coef * gr) @ W).to(torch.bfloat16)}


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["c"]
    op = c["op"]
    if not own:
        return {"embed": _embed, "embed_bwd": _embed_bwd, "norm": _norm, "norm_bwd": _norm_bwd, "distill": _distill}[op](s)
    from verify_vocab_blocked_gb300 import qhead
    if op == "norm":
        y, mean, rstd = qhead.layer_norm(s["x"], s["w"], s["b"], EPS, center=c["center"], out_dtype=DT[c["y"]])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        dx, dw, db = qhead.layer_norm_bwd(s["x"], s["w"], s["mean"], s["rstd"], s["dy"], want_dbias=c["bias"])
        return {"dx": dx, "dw": dw, "db": db}
    head = qhead.Head(s["wq"], s["s"], s["b"], c["bits"], softcap=c.get("cap", 0.0))
    if op == "embed":
        return qhead.embed(head, s["tokens"], c["scale"], s["mask"], out_dtype=DT[c["out"]])
    if op == "embed_bwd":
        return qhead.embed_bwd(head, s["tokens"], s["dy"], c["scale"], s["mask"], dw=s["dw"])
    loss, lse, zk = qhead.distill_fwd(head, s["h"], s["ids"], s["t"], c["temp"], s["mask"])
    dh = qhead.distill_bwd(head, s["h"], s["ids"], s["t"], zk, lse, s["dloss"], c["temp"], s["mask"])
    return {"loss": loss, "lse": lse, "dh": dh}


# ------------------------------------------------------------------ definitions in 64 bits

def _codes64(wq, sc, bi, bits):
    """The table in 64 bits, code by code from the words' bytes."""
    by = wq.contiguous().view(torch.uint8)
    q = by if bits == 8 else torch.stack((by % 16, by // 16), dim=2).flatten(1)
    G = sc.shape[1]
    return sc.double().repeat_interleave(64, 1)[:, : G * 64] * q.double() + bi.double().repeat_interleave(64, 1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op = c["op"]
    if op in ("norm", "norm_bwd"):
        x, w = s["x"].double(), s["w"].double()
        b = s["b"].double() if c["bias"] else None
        if op == "norm":
            mean = x.mean(1)
            var = (x.var(1, correction=0) if c["center"] else (x * x).mean(1)) + EPS
            y = (x - mean[:, None] * c["center"]) / var.sqrt()[:, None] * w
            return {"y": y if b is None else y + b, "mean": mean if c["center"] else None, "rstd": 1.0 / var.sqrt()}
        # through the given (rounded) statistics, term by term
        dy, r = s["dy"].double(), s["rstd"].double()
        xh = torch.addcmul(-s["mean"].double()[:, None] * r[:, None], x, r[:, None]) if c["center"] else x * r[:, None]
        n = c["H"]
        c2 = torch.einsum("mh,mh,h->m", dy, xh, w) / n
        c1 = (dy @ w) / n if c["center"] else torch.zeros_like(c2)
        dx = r[:, None] * (dy * w - c1[:, None] - c2[:, None] * xh)
        return {"dx": dx, "dw": torch.einsum("mh,mh->h", dy, xh), "db": torch.ones_like(r) @ dy if c["bias"] else None}
    if op == "embed":
        t = s["tokens"].long()
        y = c["scale"] * _codes64(s["wq"][t], s["s"][t], s["b"][t], c["bits"])
        return y if s["mask"] is None else torch.where(s["mask"][:, None], y, 0.0)
    if op == "embed_bwd":
        keep = torch.arange(c["M"], device=DEV) if s["mask"] is None else s["mask"].nonzero()[:, 0]
        dw = s["dw"].double() if c["add"] else torch.zeros(c["V"], c["H"], device=DEV, dtype=torch.float64)
        uniq, inv = s["tokens"].long()[keep].unique(return_inverse=True)
        part = torch.zeros(len(uniq), c["H"], device=DEV, dtype=torch.float64)
        part.index_put_((inv,), s["dy"][keep].double(), accumulate=True)
        dw[uniq] += c["scale"] * part
        return dw
    # 64-bit products run at about 1 TFLOP/s
    if 6.0 * c["M"] * c["V"] * c["H"] > 1.2e13:
        return None
    T, cap = c["temp"], c["cap"]
    keep = torch.arange(c["M"], device=DEV) if s["mask"] is None else s["mask"].nonzero()[:, 0]
    W = _codes64(s["wq"], s["s"], s["b"], c["bits"])
    with torch.enable_grad():
        h = s["h"][keep].double().requires_grad_(True)
        z = h @ W.t()
        if cap > 0:
            z = torch.tanh(z / cap) * cap
        lse = torch.logsumexp(z / T, 1)
        ids = s["ids"][keep].long()
        ok = ids >= 0
        p = torch.softmax(torch.where(ok, s["t"][keep].double() / T, -math.inf), 1)
        plogp = torch.special.xlogy(p, p)
        zk = z.gather(1, ids * ok)
        loss = (plogp - p * (zk / T - lse[:, None])).sum(1)
        dh, = torch.autograd.grad((loss * s["dloss"][keep].double()).sum(), h)
    full = lambda v: torch.zeros(c["M"], *v.shape[1:], device=DEV, dtype=torch.float64).index_copy_(0, keep, v.detach())  # noqa: E731
    return {"loss": full(loss), "lse": full(lse), "dh": full(dh)}


# ------------------------------------------------------------------ work

def _distinct(c, M):
    """Expected number of distinct tokens among M draws of _tokens."""
    v = torch.arange(c["V"], dtype=torch.float64)
    p = torch.log((v + 2) / (v + 1)) / math.log(c["V"] + 1)
    return float((1 - (1 - p) ** M).sum())


def work(case):
    c = case
    M, H = c["M"], c["H"]
    if c["op"] == "norm":
        return {"bytes": M * H * (SIZE[c["x"]] + SIZE[c["y"]]) + 8 * M, "flops": 8 * M * H}
    if c["op"] == "norm_bwd":
        return {"bytes": M * H * (2 * SIZE[c["x"]] + SIZE[c["y"]]) + 8 * M + 12 * H, "flops": 14 * M * H}
    V, row = c["V"], c["H"] * c["bits"] // 8 + 4 * (c["H"] // 64)
    live = M * 717 / 1024 if c["masked"] and M > 307 else M
    if c["op"] == "embed":
        return {"bytes": _distinct(c, live) * row + M * (4 + H * SIZE[c["out"]]), "flops": 3 * live * H}
    if c["op"] == "embed_bwd":
        dw = 8 * H * _distinct(c, live) if c["add"] else 4 * V * H
        return {"bytes": live * H * SIZE[c["dy"]] + 4 * M + dw, "flops": 2 * live * H}
    # the logits once and the contraction with the table once
    return {"bytes": V * row + live * (4 * H + c["K"] * (4 + SIZE[c["t"]])) + 8 * M, "flops": 4 * live * V * H}
