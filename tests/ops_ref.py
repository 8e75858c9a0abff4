"""Plain 64-bit forms of the operators beside the head, and small inputs for
their tests."""
import torch

U = 2.0 ** -24                       # half a step of fp32


def half_step(dtype):
    """The largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the smallest subnormal step (roundings near zero)."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make_table(V, H, bits, seed, sb=torch.float16):
    """(wq int32, scales, biases) on the GPU: uniform codes."""
    g = gen(seed)
    wq = torch.randint(-2 ** 31, 2 ** 31, (V, H * bits // 32), device="cuda", generator=g,
                       dtype=torch.int64).to(torch.int32)
    s = (1e-3 + 9e-3 * torch.rand(V, H // 64, device="cuda", generator=g)) * (16 / 2 ** bits)
    b = -(2 ** (bits - 1)) * s + 1e-3 * torch.randn(V, H // 64, device="cuda", generator=g)
    return wq, s.to(sb), b.to(sb)


def table64(wq, s, b, bits):
    by = wq.contiguous().view(torch.uint8)
    q = by if bits == 8 else torch.stack((by & 15, by >> 4), dim=2).flatten(1)
    return s.double().repeat_interleave(64, 1) * q.double() + b.double().repeat_interleave(64, 1)


def norm64(x, w, b, eps, center):
    x, w = x.double(), w.double()
    mean = x.mean(1, keepdim=True)
    xc = x - mean if center else x
    rstd = (xc.square().mean(1, keepdim=True) + eps).rsqrt()
    y = xc * rstd * w
    return y + b.double() if b is not None else y


def distill64(W, h, ids, t, T, cap, mask=None):
    """Per-row loss and lse (float64) with autograd into h (float64)."""
    z = h @ W.t()
    if cap > 0:
        z = cap * torch.tanh(z / cap)
    lse = torch.logsumexp(z / T, 1)
    ok = ids >= 0
    tt = torch.where(ok, t.double() / T, -float("inf"))
    some = torch.isfinite(tt).any(1)
    p = torch.softmax(torch.where(some[:, None], tt, 0.0), 1) * some[:, None]
    zk = z.gather(1, ids.clamp_min(0).long())
    loss = (torch.special.xlogy(p, p) - torch.where(p > 0, p * (zk / T - lse[:, None]), 0.0)).sum(1)
    if mask is not None:
        on = mask.bool()
        loss, lse = torch.where(on, loss, 0.0), torch.where(on, lse, 0.0)
    return loss, lse, z, p
