"""The trainable block beside the quantized head, as cases to measure and check.

A matrix product with bias, activation and residual in its epilogue, its
gradient and its form on 8-bit operands; the residual's addition with the norm
behind it, its gradient and its 8-bit output with row scales; and the global
gradient norm over many tensors, with clipping.  `run` computes them in plain
torch operations, or, with `own` set, through the package's public calls.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
E4M3 = torch.float8_e4m3fn
EPS = 1e-6


def listed():
    # H = 2560 and 1536 and the row counts 5, 512 and 8192 are the package's
    # workloads'; 4 H is the usual inner width of a block.
    return [
        # a draft block on a verify window's rows, h + silu(W h + b): latency
        dict(name="linear_window", op="linear", M=5, K=2560, N=2560, t="bf16", act="silu", bias="bf16", res="bf16", out="bf16", pad=0),
        # a ragged batch through odd widths, rows of a wider tensor, float32 out
        dict(name="linear_ragged", op="linear", M=301, K=1541, N=2563, t="f16", act="gelu_tanh", bias="f32", res="", out="f32", pad=3),
        # the training batch through a block's first product
        dict(name="linear_up", op="linear", M=8192, K=2560, N=10240, t="bf16", act="gelu_tanh", bias="bf16", res="", out="bf16", pad=0),
        # serving from 8-bit weights: a verify window, and a long prompt back into the stream
        dict(name="linear8_window", op="linear8", M=5, K=2560, N=10240, act="silu", bias="bf16", res="", out="bf16"),
        dict(name="linear8_prompt", op="linear8", M=8192, K=10240, N=2560, act="none", bias="", res="bf16", out="bf16"),
        # training steps of the block: forward, and gradients into x, W and b
        dict(name="linear_step", op="linear_step", M=8192, K=2560, N=2560, t="bf16", act="silu", bias="bf16", res="bf16", out="bf16", pad=0),
        dict(name="linear_step_515", op="linear_step", M=515, K=1536, N=6144, t="f16", act="gelu", bias="f16", res="", out="f16", pad=0),
        # the residual and the norm behind it: a verify window; 8 bits out for the product above
        dict(name="add_norm_window", op="add_norm", M=5, H=2560, x="bf16", r="bf16", y="bf16", center=False, bias=False, pad=0),
        dict(name="norm8_batch", op="norm8", M=8192, H=2560, x="bf16", r="bf16", center=False, bias=False, pad=0),
        # both directions over a long batch with a float32 stream
        dict(name="add_norm_step", op="add_norm_step", M=32768, H=1536, x="bf16", r="f32", y="bf16", center=True, bias=True, pad=0),
        # gradients of a tied table and of the blocks beside it, clipped into 16 bits' place
        dict(name="clip_table", op="clip", n=40, total=230_000_000, t="mix", flat=False, factor=0.5, out=True),
        # a few small tensors within the limit, in one flat buffer
        dict(name="clip_small", op="clip", n=48, total=120_001, t="f32", flat=True, factor=2.0, out=False),
    ]


ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear8", "linear_step", "add_norm", "norm8", "add_norm_step", "clip"])
    c = dict(op=op)
    if op == "clip":
        factor = rng.choice([0.1, 0.7, 3.0])
        c.update(n=_log_int(rng, 1, 60), total=_log_int(rng, 1000, 200_000_000), t=rng.choice(["f32", "bf16", "mix"]),
                 flat=rng.random() < 0.4, factor=factor, out=factor < 1 or rng.random() < 0.5)
        return c
    if op in ("add_norm", "norm8", "add_norm_step"):
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            H = (H + 7) // 8 * 8
        c.update(H=H, M=_log_int(rng, 1, 40_000_000 // H), x=rng.choice(["bf16", "f16", "f32"]), r=rng.choice(["bf16", "f32", "f16"]),
                 center=rng.random() < 0.5, bias=rng.random() < 0.5, pad=rng.choice([0, 0, 8, 3]))
        if op != "norm8":
            c.update(y=rng.choice(["bf16", "f16", "f32"]))
        elif rng.random() < 0.3:
            c.update(r="")
        return c
    c.update(K=_log_int(rng, 64, 10240), N=_log_int(rng, 64, 10240), act=rng.choice(ACTS), bias=rng.choice(["", "bf16", "f32"]),
             res=rng.choice(["", "bf16", "f32"]), out=rng.choice(["bf16", "bf16", "f32"]))
    if rng.random() < 0.6:
        c.update(K=(c["K"] + 15) // 16 * 16, N=(c["N"] + 15) // 16 * 16)
    c["M"] = _log_int(rng, 1, max(64, min(16384, 60_000_000_000 // (c["K"] * c["N"]))))
    if op != "linear8":
        c.update(t=rng.choice(["bf16", "bf16", "f16"]), pad=rng.choice([0, 0, 8, 3]))
    if op == "linear_step":
        c.update(out=c["t"], bias=c["t"] if c["bias"] else "")
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def _quantized(v):
    """Rows in 8 bits with a scale each, as a program stores its weights."""
    scale = v.abs().amax(1).clamp_min(1e-30) / 448.0
    return (v / scale[:, None]).to(E4M3), scale


def _sizes(c):
    """Tensor sizes that fall off like 1 / rank, one of them of a single element."""
    w = [1.0 / (i + 1) for i in range(c["n"])]
    return [max(1, int(c["total"] * v / sum(w))) for v in w[:-1]] + [1]


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = dict(c=c)
    if c["op"] == "clip":
        sizes = _sizes(c)
        types = [torch.float32 if c["t"] == "f32" or c["t"] == "mix" and i % 2 == 0 else torch.bfloat16 for i in range(len(sizes))]
        if c["flat"] and c["t"] != "mix":  # back to back in one buffer: starts of any alignment
            s["grads"] = list((1e-3 * _randn(g, sum(sizes))).to(types[0]).split(sizes))
        else:
            s["grads"] = [(1e-3 * _randn(g, n)).to(t) for n, t in zip(sizes, types)]
        s["max_norm"] = c["factor"] * 1e-3 * math.sqrt(sum(sizes))
        s["out"] = [torch.empty(n, device=DEV, dtype=torch.bfloat16) for n in sizes] if c["out"] else None
        return s
    M = c["M"]
    if "H" in c:
        H = c["H"]
        # a residual stream: rows of their own size and offset, a few strong channels
        r = _randn(g, M, H + c["pad"]) * (0.5 + 2.0 * torch.rand(M, 1, device=DEV, generator=g)) + 0.3 * _randn(g, M, 1)
        r[:, :: max(1, H // 4)] *= 8.0
        s["x"] = (0.5 * _randn(g, M, H + c["pad"])).to(DT[c["x"]])[:, :H]
        s["r"] = r.to(DT[c["r"]])[:, :H] if c["r"] else None
        s["w"] = (1.0 + 0.1 * _randn(g, H)).to(DT[c["x"]])
        s["b"] = (0.1 * _randn(g, H)).to(DT[c["x"]]) if c["bias"] else None
        if c["op"] == "add_norm_step":
            s["dy"] = (1e-2 * _randn(g, M, H)).to(DT[c["y"]])
            s["dt"] = (1e-2 * _randn(g, M, H)).to(DT[c["r"]])
        return s
    K, N = c["K"], c["N"]
    x, w = _randn(g, M, K + c.get("pad", 0)), _randn(g, N, K) / math.sqrt(K)
    if c["op"] == "linear8":
        s["x"], s["xs"] = _quantized(x)
        s["w"], s["ws"] = _quantized(w)
    else:
        s["x"], s["w"] = x.to(DT[c["t"]])[:, :K], w.to(DT[c["t"]])
    s["b"] = (0.1 * _randn(g, N)).to(DT[c["bias"]]) if c["bias"] else None
    s["r"] = _randn(g, M, N).to(DT[c["res"]]) if c["res"] else None
    if c["op"] == "linear_step":
        s["dy"] = (1e-2 * _randn(g, M, N)).to(DT[c["t"]])
    return s


# ------------------------------------------------------------------ plain forms

def _act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _linear(s):
    """(y, pre-activation), float32."""
    c = s["c"]
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.t()
    if c["op"] == "linear8":
        z = z * s["xs"][:, None] * s["ws"]
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, c["act"])
    return (y if s["r"] is None else y + s["r"].float()), z


def _linear_step(s):
    c = s["c"]
    t = DT[c["t"]]
    y, z = _linear(s)
    dz = s["dy"].float() * _act_grad(z, c["act"])
    return {"y": y.to(t), "dx": (dz @ s["w"].float()).to(t), "dw": (dz.t() @ s["x"].float()).to(t),
            "db": dz.sum(0).to(t) if s["b"] is not None else None}


def _norm(s):
    """(y, sum, mean, rstd), float32."""
    c = s["c"]
    v = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
    mean = v.mean(1, keepdim=True)
    vc = v - mean if c["center"] else v
    rstd = (vc.square().mean(1, keepdim=True) + EPS).rsqrt()
    y = vc * rstd * s["w"].float()
    return (y if s["b"] is None else y + s["b"].float()), v, mean, rstd


def _add_norm(s):
    c = s["c"]
    y, v, mean, rstd = _norm(s)
    return {"y": y.to(DT[c["y"]]), "sum": v.to(DT[c["r"]]), "mean": mean[:, 0] if c["center"] else None, "rstd": rstd[:, 0]}


def _norm8(s):
    c = s["c"]
    y, v, _, _ = _norm(s)
    codes, scale = _quantized(y)
    return {"codes": codes, "scale": scale, "sum": v.to(DT[c["r"]]) if c["r"] else None}


def _add_norm_step(s):
    c = s["c"]
    out = _add_norm(s)
    _, v, mean, rstd = _norm(s)
    dy = s["dy"].float()
    xh = (v - mean if c["center"] else v) * rstd
    g = dy * s["w"].float()
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if c["center"]:
        dx = dx - g.mean(1, keepdim=True)
    out["dx"] = (dx * rstd + s["dt"].float()).to(DT[c["r"]])
    # (16 bits, as the parameters' gradients are kept: the sum that the backward reads is rounded)
    out["dw"] = (dy * xh).sum(0).to(DT["bf16"])
    out["db"] = dy.sum(0) if c["bias"] else None
    return out


def _clip(s):
    norm = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]]).sum().sqrt()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    if s["out"] is not None:
        return {"norm": norm.float(), "grads": [o.copy_(t.float() * coef) for o, t in zip(s["out"], s["grads"])]}
    return {"norm": norm.float(), "grads": [t.mul_(coef) for t in s["grads"]]}


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["c"]
    op = c["op"]
    if not own:
        if op in ("linear", "linear8"):
            return _linear(s)[0].to(DT[c["out"]])
        return {"linear_step": _linear_step, "add_norm": _add_norm, "norm8": _norm8, "add_norm_step": _add_norm_step, "clip": _clip}[op](s)
    from verify_vocab_blocked_gb300 import qhead
    if op == "linear":
        return qhead.linear(s["x"], s["w"], s["b"], c["act"], s["r"], out_dtype=DT[c["out"]])
    if op == "linear8":
        return qhead.linear(s["x"], s["w"], s["b"], c["act"], s["r"], x_scale=s["xs"], w_scale=s["ws"], out_dtype=DT[c["out"]])
    if op == "linear_step":
        y, pre = qhead.linear(s["x"], s["w"], s["b"], c["act"], s["r"], want_pre=True)
        dx, dw, db = qhead.linear_bwd(s["x"], s["w"], s["dy"], pre, c["act"], want_dbias=s["b"] is not None)
        return {"y": y, "dx": dx, "dw": dw, "db": db}
    if op == "norm8":
        codes, scale, total = qhead.norm_8bit(s["x"], s["w"], s["b"], EPS, residual=s["r"], center=c["center"])
        return {"codes": codes, "scale": scale, "sum": total}
    if op == "clip":
        norm = qhead.clip_grads(s["grads"], s["max_norm"], out=s["out"])
        return {"norm": norm, "grads": s["grads"] if s["out"] is None else s["out"]}
    y, total, mean, rstd = qhead.add_norm(s["x"], s["r"], s["w"], s["b"], EPS, center=c["center"], out_dtype=DT[c["y"]])
    out = {"y": y, "sum": total, "mean": mean, "rstd": rstd}
    if op == "add_norm_step":
        out["dx"], dw, out["db"] = qhead.add_norm_bwd(total, s["w"], mean, rstd, s["dy"], s["dt"], want_dbias=c["bias"])
        out["dw"] = dw.to(DT["bf16"])
    return out


# ------------------------------------------------------------------ definitions in 64 bits

def exact(case, seed):
    c, s = case, prepare(case, seed)
    op = c["op"]
    if op == "clip":
        norm = torch.cat([t.double().norm().reshape(1) for t in s["grads"]]).norm()
        k = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
        return {"norm": norm, "grads": [t.double() * k for t in s["grads"]]}
    if "H" in c:
        x = s["x"].double() + (s["r"].double() if s["r"] is not None else 0.0)
        w, b = s["w"].double().requires_grad_(True), torch.zeros_like(s["w"], dtype=torch.float64).requires_grad_(True)
        if s["b"] is not None:
            b = s["b"].double().requires_grad_(True)
        x.requires_grad_(op == "add_norm_step")
        var, mean = torch.var_mean(x, 1, correction=0)
        std = ((var if c["center"] else var + mean.square()) + EPS).sqrt()
        y = torch.addcmul(b, (x - mean[:, None] * float(c["center"])) / std[:, None], w)
        if op == "norm8":
            scale = y.abs().amax(1) / 448.0
            return {"codes": (y / scale[:, None]).detach(), "scale": scale.detach(), "sum": x if c["r"] else None}
        out = {"y": y.detach(), "sum": x.detach(), "mean": mean.detach() if c["center"] else None, "rstd": (1.0 / std).detach()}
        if op == "add_norm_step":
            dx, dw, db = torch.autograd.grad(y, (x, w, b), s["dy"].double())
            out |= {"dx": dx + s["dt"].double(), "dw": dw, "db": db if c["bias"] else None}
        return out
    x, w = s["x"].double(), s["w"].double()
    if op == "linear8":
        x, w = x * s["xs"].double()[:, None], w * s["ws"].double()[:, None]
    b = torch.zeros(c["N"], device=DEV, dtype=torch.float64) if s["b"] is None else s["b"].double()
    leaves = [v.requires_grad_(op == "linear_step") for v in (x, w, b)]
    f = torch.nn.functional
    act = {"none": lambda z: z, "relu": f.relu, "silu": f.silu, "gelu": f.gelu, "gelu_tanh": lambda z: f.gelu(z, approximate="tanh")}[c["act"]]
    y = act(torch.addmm(b, x, w.t()))
    if s["r"] is not None:
        y = y + s["r"].double()
    if op != "linear_step":
        return y
    dx, dw, db = torch.autograd.grad(y, leaves, s["dy"].double())
    return {"y": y.detach(), "dx": dx, "dw": dw, "db": db if s["b"] is not None else None}


# ------------------------------------------------------------------ work

def work(case):
    c = case
    op = c["op"]
    if op == "clip":
        sizes = _sizes(c)
        item = [4 if c["t"] == "f32" or c["t"] == "mix" and i % 2 == 0 else 2 for i in range(len(sizes))]
        read = sum(n * k for n, k in zip(sizes, item))
        return {"bytes": read + (2 * sum(sizes) if c["out"] else read if c["factor"] < 1 else 0), "flops": 3 * sum(sizes)}
    M = c["M"]
    if "H" in c:
        H, r = c["H"], SIZE.get(c["r"], 0)
        row = SIZE[c["x"]] + 2 * r + (1 if op == "norm8" else SIZE[c["y"]])
        if op == "add_norm_step":
            row += SIZE[c["y"]] + 3 * r
        return {"bytes": M * H * row + 8 * M, "flops": (25 if op == "add_norm_step" else 10) * M * H}
    K, N = c["K"], c["N"]
    t = 1 if op == "linear8" else SIZE[c["t"]]
    size = t * (M * K + N * K) + M * N * (SIZE[c["out"]] + SIZE.get(c["res"], 0))
    if op == "linear_step":  # dy read, dx and dw written; x and W are still at hand
        return {"bytes": size + t * (2 * M * K + 2 * N * K + M * N), "flops": 6 * M * N * K}
    return {"bytes": size, "flops": 2 * M * N * K}
