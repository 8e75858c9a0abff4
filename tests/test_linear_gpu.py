"""The matrix product with its epilogue, and its gradient, against 64 bits.

Tolerances.  The products of 16-bit (8-bit) operands are exact in fp32; a sum of
K of them is formed 16 (32) at a time with at most a whole step of fp32, 2^-23 of
the sum of magnitudes, lost at each.  Scales, bias and the activation's function
add a few steps; its derivative is below 1.13 and its argument enters the
exponential with a relative half step, so that 2^-20 (1 + |z|) covers it.  Every
output adds one rounding to its type.  The gradient is checked as the function of
the given pre that it is documented to be; its products take dz rounded once."""
import pytest
import torch

from ops_ref import gen, half_step, tiny
from verify_vocab_blocked_gb300 import build as qbuild
from verify_vocab_blocked_gb300 import qhead

pytestmark = pytest.mark.gpu
BF, HF, F, E8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
ACTS = {
    "none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
    "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh"),
}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qhead.lib()


def accumulated(K, mag, per=16):
    return (K / per + 16) * 2.0 ** -23 * mag


def operands(M, K, N, t, seed, pad=0, padw=0):
    g = gen(seed)
    x = torch.randn(M, K + pad, device="cuda", generator=g)
    w = torch.randn(N, K + padw, device="cuda", generator=g) / K ** 0.5
    if t != E8:
        return x.to(t)[:, :K], w.to(t)[:, :K], None, None
    xs, ws = x[:, :K].abs().amax(1) / 448, w[:, :K].abs().amax(1) / 448
    return (x / xs[:, None]).to(E8)[:, :K], (w / ws[:, None]).to(E8)[:, :K], xs, ws


def check(x, w, xs, ws, b, act, r, out, want_pre=False):
    got = qhead.linear(x, w, b, act, r, x_scale=xs, w_scale=ws, out_dtype=out, want_pre=want_pre)
    y, pre = got if want_pre else (got, None)
    xd, wd = x.double(), w.double()
    if xs is not None:
        xd, wd = xd * xs.double()[:, None], wd * ws.double()[:, None]
    z = xd @ wd.t()
    mag = xd.abs() @ wd.abs().t()
    if b is not None:
        z, mag = z + b.double(), mag + b.double().abs()
    ref = ACTS[act](z)
    e = accumulated(x.shape[1], mag, 16 if xs is None else 32)
    tol = 1.13 * e + 2.0 ** -20 * (1 + z.abs()) * (act != "none")
    if r is not None:
        ref = ref + r.double()
    tol = tol + (half_step(out or x.dtype) + 2.0 ** -23) * ref.abs() + tiny(out or x.dtype)
    assert y.dtype == (out or x.dtype) and y.shape == ref.shape
    bad = ((y.double() - ref).abs() > 1.01 * tol).sum().item()
    assert bad == 0, (bad, ((y.double() - ref).abs() / tol).max().item())
    if want_pre:
        assert ((pre.double() - z).abs() <= 1.01 * (e + (2.0 ** -11 + 2.0 ** -23) * z.abs() + tiny(HF))).all()
    return y, pre


@pytest.mark.parametrize("M,K,N,t,pad,padw,act,bias,res,out", [
    # few tokens: each tile, cluster splits of 1 to 8, ragged edges
    (1, 64, 128, BF, 0, 0, "none", None, None, None),
    (1, 2560, 2560, BF, 0, 0, "silu", BF, BF, BF),
    (5, 2560, 10240, HF, 0, 0, "gelu", F, None, F),
    (16, 192, 200, BF, 0, 0, "relu", HF, F, BF),
    (17, 1536, 4096, BF, 0, 0, "none", None, None, BF),
    (33, 8, 129, HF, 0, 0, "gelu_tanh", None, BF, HF),
    (64, 4096, 40000, BF, 0, 0, "none", BF, None, BF),
    (65, 1000, 1000, BF, 0, 0, "silu", BF, None, F),
    (128, 2560, 2560, HF, 0, 0, "none", None, F, F),
    # lengths of one, odd widths, strides
    (1, 1, 1, BF, 0, 0, "none", F, F, F),
    (3, 7, 5, HF, 1, 0, "gelu", HF, None, F),
    (40, 77, 130, BF, 3, 2, "silu", BF, BF, BF),
    (70, 200, 96, BF, 8, 16, "relu", None, None, BF),
    # pairs
    (129, 64, 64, BF, 0, 0, "none", None, None, BF),
    (200, 128, 256, HF, 0, 0, "gelu_tanh", BF, HF, HF),
    (257, 576, 513, BF, 0, 0, "silu", BF, BF, BF),
    (301, 1541, 2563, HF, 3, 0, "gelu_tanh", F, None, F),
    (1000, 72, 1000, BF, 8, 8, "relu", F, F, F),
    (2049, 1536, 2560, BF, 0, 0, "gelu", BF, BF, BF),
    # tiles whose reduction is shared, alone and behind full rounds; ragged, unaligned
    (300, 4096, 600, BF, 0, 0, "silu", BF, BF, BF),
    (300, 4100, 601, HF, 4, 0, "gelu", F, HF, HF),
    (257, 3000, 520, BF, 0, 8, "none", None, F, F),
    (2500, 2560, 2600, BF, 0, 0, "silu", F, F, BF),
    # every count of parts of few rows, and several tiles of 64
    (7, 192, 300, BF, 0, 0, "none", BF, None, BF),
    (12, 1000, 20000, HF, 0, 0, "relu", None, HF, HF),
    (100, 2560, 700, BF, 0, 0, "gelu_tanh", BF, BF, BF),
    (190, 2000, 1300, BF, 8, 0, "silu", BF, F, F),
    (256, 576, 1001, HF, 0, 0, "none", F, None, HF),
])
def test_forward(M, K, N, t, pad, padw, act, bias, res, out):
    x, w, xs, ws = operands(M, K, N, t, M + K + N, pad, padw)
    g = gen(M)
    b = torch.randn(N, device="cuda", generator=g).to(bias) if bias else None
    r = torch.randn(M, N + pad, device="cuda", generator=g).to(res)[:, :N] if res else None
    check(x, w, xs, ws, b, act, r, out, want_pre=True)


@pytest.mark.parametrize("M,K,N,pad,act,bias,res,out", [
    (1, 2560, 2560, 0, "silu", BF, BF, BF),
    (5, 128, 300, 0, "none", None, None, F),
    (9, 16, 17, 0, "gelu", F, None, BF),
    (3, 5, 6, 2, "none", None, None, None),
    (100, 10240, 256, 0, "none", BF, None, F),
    (130, 256, 256, 0, "none", None, None, F),
    (515, 1536, 2563, 0, "gelu_tanh", BF, F, F),
    (300, 1001, 520, 7, "relu", None, BF, HF),
    (300, 4096, 600, 0, "silu", F, BF, BF),
    (200, 4000, 700, 0, "none", BF, None, F),
])
def test_forward_of_8_bits(M, K, N, pad, act, bias, res, out):
    x, w, xs, ws = operands(M, K, N, E8, M + K + N, pad)
    g = gen(M)
    b = torch.randn(N, device="cuda", generator=g).to(bias) if bias else None
    r = torch.randn(M, N, device="cuda", generator=g).to(res) if res else None
    check(x, w, xs, ws, b, act, r, out or BF)


def act_grad64(z, act):
    if act == "none":
        return torch.ones_like(z)
    z = z.clone().requires_grad_(True)
    return torch.autograd.grad(ACTS[act](z).sum(), z)[0]


def check_bwd(M, K, N, t, act, dt, pad=0, padw=0, seed=0):
    x, w, _, _ = operands(M, K, N, t, seed + M + K + N, pad, padw)
    g = gen(seed + 3)
    _, pre = qhead.linear(x, w, torch.randn(N, device="cuda", generator=g), act, want_pre=True)
    dy = torch.randn(M, N + pad, device="cuda", generator=g).to(dt)[:, :N]
    dx, dw, db = qhead.linear_bwd(x, w, dy, pre, act)
    again = qhead.linear_bwd(x, w, dy, pre, act)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))
    z = pre.double()
    grad = act_grad64(z, act)
    dz = dy.double() * grad
    # the derivative: below 1.13, its parts off by a few steps of (1 + |z|)
    e_dz = dy.double().abs() * 2.0 ** -20 * (1 + z.abs()) * (act != "none")
    as_is = act == "none" and dt == t
    r_dz = e_dz + (0 if as_is else (half_step(t) * dz.abs() + tiny(t)))
    wd, xd = w.double(), x.double()
    for got, ref, e, mag, n in (
            (dx, dz @ wd, r_dz @ wd.abs(), dz.abs() @ wd.abs(), N),
            (dw, dz.t() @ xd, r_dz.t() @ xd.abs(), dz.abs().t() @ xd.abs(), M)):
        tol = e + accumulated(n, mag * 1.01) + half_step(t) * ref.abs() + tiny(t)
        assert got.dtype == t and got.shape == ref.shape
        assert ((got.double() - ref).abs() <= 1.01 * tol).all(), ((got.double() - ref).abs() / tol).max().item()
    ref = dz.sum(0)
    tol = e_dz.sum(0) + M * 2.0 ** -24 * dz.abs().sum(0) + half_step(t) * ref.abs() + tiny(t)
    assert ((db.double() - ref).abs() <= 1.01 * tol).all()
    return x, w, dy, pre, dx, dw, db


@pytest.mark.parametrize("M,K,N,t,act,dt,pad,padw", [
    (1, 1, 1, BF, "silu", F, 0, 0),
    (5, 2560, 2560, BF, "silu", BF, 0, 0),
    (64, 100, 72, HF, "gelu", HF, 0, 0),
    (70, 77, 131, BF, "gelu_tanh", F, 3, 1),
    (130, 256, 384, BF, "none", BF, 0, 0),
    (130, 256, 383, BF, "none", BF, 1, 0),
    (200, 640, 136, HF, "relu", BF, 8, 8),
    (515, 1536, 1030, BF, "silu", BF, 0, 0),
    (2000, 520, 264, BF, "none", F, 0, 0),
    (4100, 128, 2563, HF, "gelu", HF, 0, 0),
    (5000, 600, 300, BF, "silu", BF, 0, 0),       # shared reductions: over 5000 rows,
    (300, 264, 4200, HF, "none", HF, 0, 0),       # over 4200 columns
    (190, 300, 1000, BF, "gelu_tanh", BF, 0, 0),  # few rows, weights down their rows
])
def test_gradient(M, K, N, t, act, dt, pad, padw):
    check_bwd(M, K, N, t, act, dt, pad, padw)


def test_gradient_parts_and_none():
    x, w, dy, pre, dx, dw, db = check_bwd(90, 64, 80, BF, "silu", BF)
    got = qhead.linear_bwd(x, w, dy, pre, "silu", want_dx=False, want_dbias=False)
    assert got[0] is None and got[2] is None and torch.equal(got[1], dw)
    got = qhead.linear_bwd(x, w, dy, pre, "silu", want_dw=False, want_dx=False)
    assert got[:2] == (None, None) and torch.equal(got[2], db)
    assert torch.equal(qhead.linear_bwd(x, w, dy, pre, "silu", want_dw=False)[0], dx)
    none = qhead.linear_bwd(x[:0], w, dy[:0], pre[:0], "silu")
    assert none[0].shape == (0, 64) and not none[1].any() and not none[2].any()
    assert qhead.linear(x[:0], w).shape == (0, 80)


@pytest.mark.parametrize("act", list(ACTS))
def test_gradient_against_differences(act):
    """The loss sum(dy y) along random directions of x, W and b: the 64-bit
    function's central difference over a step of 1e-4, off by its third
    derivative (1e-8 of the loss's scale) and, of the gradients, by the roundings of
    dz and of the output, 2^-11 each of the sum of magnitudes; relu's kink is kept
    away from."""
    M, K, N = 40, 96, 72
    x, w, _, _ = operands(M, K, N, HF, 4)
    g = gen(5)
    b = torch.randn(N, device="cuda", generator=g)
    dy = torch.randn(M, N, device="cuda", generator=g)
    if act == "relu":  # no gradient through values that the step may carry past the kink
        z = x.double() @ w.double().t() + b.double()
        dy = torch.where(z.abs() > 0.02, dy, 0.0)
    _, pre = qhead.linear(x, w, b, act, want_pre=True)
    dx, dw, db = (v.double() for v in qhead.linear_bwd(x, w, dy, pre, act))

    def loss(xx, ww, bb):
        return (ACTS[act](xx @ ww.t() + bb) * dy.double()).sum()

    xd, wd, bd, step = x.double(), w.double(), b.double(), 1e-4
    for k, grad in ((0, dx), (1, dw), (2, db)):
        v = torch.randn(grad.shape, device="cuda", generator=g, dtype=torch.float64)
        at = [xd, wd, bd]
        up, down = list(at), list(at)
        up[k], down[k] = at[k] + step * v, at[k] - step * v
        diff = (loss(*up) - loss(*down)) / (2 * step)
        dzm = dy.double().abs() * 1.13
        mag = (dzm @ wd.abs(), dzm.t() @ xd.abs(), dzm.sum(0))[k]
        # pre's own rounding (2^-11 of it, times a second derivative below 1.2) beside them
        tol = 4 * 2.0 ** -11 * (mag * v.abs()).sum() + 1e-5 * mag.sum()
        assert abs((grad * v).sum() - diff) <= tol


def test_values_that_are_not_finite_stay_in_their_row():
    x, w, _, _ = operands(20, 64, 40, BF, 8)
    x, w = x.contiguous(), w.contiguous()
    x[3, 5], x[7, 0], x[9, :] = float("nan"), float("inf"), 0
    for act in ACTS:
        y, pre = qhead.linear(x, w, None, act, want_pre=True)
        rest = [i for i in range(20) if i not in (3, 7)]
        assert torch.isnan(y[3]).all() and torch.isfinite(y[rest]).all() and (y[9] == 0).all()
        assert torch.isnan(pre[3]).all() and (pre[7].abs() == 65504).all()
    wide = torch.full((1, 64), 3e4, device="cuda", dtype=BF)   # beyond fp16
    y, pre = qhead.linear(wide, wide, None, "gelu", want_pre=True)
    assert torch.isfinite(y).all() and (pre == 65504).all()
    assert torch.equal(qhead.linear_bwd(wide, wide, y, pre, "gelu")[2], y[0])


def test_a_captured_call_and_another_stream():
    x, w, _, _ = operands(300, 200, 264, BF, 1)
    b = torch.randn(264, device="cuda").to(BF)
    few = x[:9].contiguous()
    _, pre = qhead.linear(x, w, b, "silu", want_pre=True)
    dy = torch.randn(300, 264, device="cuda", generator=gen(2))

    def every(stream=None):
        return (qhead.linear(x, w, b, "silu", stream=stream), qhead.linear(few, w, b, "gelu", stream=stream),
                *qhead.linear_bwd(x, w, dy, pre, "silu", stream=stream))

    ref = every()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = every(s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = every()
    x.neg_()
    few.copy_(x[:9])
    graph.replay()
    now = every()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(kept, now)) and not torch.equal(kept[0], ref[0])


@pytest.mark.parametrize("M", [5, 300])
def test_a_wait_that_expires(M):
    """No loads are issued: the outputs come back NaN after the limit, and the next
    call is right."""
    import time
    x, w, _, _ = operands(M, 256, 300, BF, 6)
    ref = qhead.linear(x, w)
    torch.cuda.synchronize()
    t0 = time.monotonic()
    qhead.test_stall_next_call(True)
    y = qhead.linear(x, w)
    torch.cuda.synchronize()
    assert 1.5 <= time.monotonic() - t0 < 60
    assert torch.isnan(y).all()
    assert torch.equal(qhead.linear(x, w), ref)


@pytest.mark.parametrize("M,K,N,t,pad,padw,act,bias,res,out", [
    # 17 to 512 rows in several tiles of 32, 64 and 128, the reduction in 1 to 8 parts
    (20, 128, 3000, BF, 0, 0, "none", None, None, BF),
    (96, 2560, 2560, BF, 0, 0, "gelu", F, BF, BF),
    (192, 6144, 1536, HF, 0, 0, "silu", HF, F, F),
    (301, 1536, 1536, BF, 0, 0, "silu", BF, BF, BF),
    (384, 4096, 520, BF, 0, 0, "none", None, F, F),
    (400, 640, 1003, HF, 3, 5, "gelu_tanh", F, HF, HF),
    (512, 1000, 1000, BF, 8, 0, "relu", BF, BF, F),
    # columns that end inside a strip, 4 and 1 of them; more tiles than fit at once
    (45, 512, 900, BF, 0, 0, "silu", BF, BF, BF),
    (6, 512, 129, HF, 0, 0, "gelu", None, HF, HF),
    (5, 256, 70000, BF, 0, 0, "silu", BF, BF, BF),
    (40, 64, 50001, BF, 0, 0, "none", None, None, BF),
    # pairs: short reductions, shared tiles of ragged and unaligned rows
    (100, 64, 40000, BF, 0, 0, "silu", None, BF, BF),
    (600, 4096, 600, BF, 0, 0, "silu", BF, BF, BF),
    (600, 4100, 601, HF, 4, 0, "gelu", F, HF, HF),
    (700, 3000, 520, BF, 0, 8, "none", None, F, F),
    (515, 10240, 300, BF, 0, 0, "gelu_tanh", BF, None, F),
])
def test_forward_of_middle_sizes(M, K, N, t, pad, padw, act, bias, res, out):
    test_forward(M, K, N, t, pad, padw, act, bias, res, out)


@pytest.mark.parametrize("M,K,N,t,act,dt,pad,padw", [
    (301, 1536, 1536, BF, "silu", BF, 0, 0),
    (512, 260, 2100, HF, "none", HF, 4, 0),
    (700, 600, 4200, BF, "gelu", BF, 0, 0),
    (640, 1001, 515, BF, "silu", F, 1, 0),
])
def test_gradient_of_middle_sizes(M, K, N, t, act, dt, pad, padw):
    check_bwd(M, K, N, t, act, dt, pad, padw)


@pytest.mark.parametrize("M,K,N", [(130, 5120, 256), (600, 4096, 600), (2048, 2560, 2560)])
def test_a_wait_that_expires_in_shared_sums(M, K, N):
    """... where several CTAs share a tile's reduction."""
    x, w, _, _ = operands(M, K, N, BF, 7)
    ref = qhead.linear(x, w)
    qhead.test_stall_next_call(True)
    y = qhead.linear(x, w)
    torch.cuda.synchronize()
    assert torch.isnan(y).all()
    assert torch.equal(qhead.linear(x, w), ref)


def test_few_rows_many_times_over():
    """Sums sent between CTAs: the same bits call after call, with calls in flight on two
    streams."""
    x, w, _, _ = operands(64, 2560, 2560, BF, 8)
    x2, w2, _, _ = operands(16, 2560, 4096, BF, 9)
    ref, ref2 = qhead.linear(x, w, None, "silu"), qhead.linear(x2, w2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, got2 = [], []
    for _ in range(100):
        got.append(qhead.linear(x, w, None, "silu"))
        got2.append(qhead.linear(x2, w2, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(ref, y) for y in got) and all(torch.equal(ref2, y) for y in got2)
