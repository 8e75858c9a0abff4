"""Layer norm, its uncentred form and their gradient against the plain 64-bit
forms.

Tolerances.  A sum along a row runs through at most 40 elements per thread, 5
shuffle steps and 32 warps; D = 128 half steps of the sum of magnitudes
cover it with the few operations around it.  A column sum over M rows in any
grouping is off by at most M half steps of its magnitudes.  Every output adds
one rounding to its type."""
import pytest
import torch

from ops_ref import U, gen, half_step, norm64, tiny
from verify_vocab_blocked_gb300 import build as qbuild
from verify_vocab_blocked_gb300 import qhead

pytestmark = pytest.mark.gpu
D = 128
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qhead.lib()


def _inputs(M, H, xt, wt, seed, offset=0.0, pad=0):
    g = gen(seed)
    x = torch.randn(M, H + pad, device="cuda", generator=g) * 2 + offset
    w = 1 + 0.2 * torch.randn(H, device="cuda", generator=g)
    b = torch.randn(H, device="cuda", generator=g)
    return x.to(xt)[:, :H], w.to(wt), b.to(wt)


def _check_fwd(x, w, b, eps, center, out):
    y, mean, rstd = qhead.layer_norm(x, w, b, eps, center=center, out_dtype=out)
    xd, wd = x.double(), w.double()
    m = xd.mean(1, keepdim=True) if center else torch.zeros_like(xd[:, :1])
    xc = xd - m
    r = (xc.square().mean(1, keepdim=True) + eps).rsqrt()
    ref = norm64(x, w, b, eps, center)
    mx = xd.abs().mean(1, keepdim=True) if center else torch.zeros_like(r)
    # an error e of the mean moves xc by e and the mean square by its square
    e_mean = D * U * mx
    rel_r = D * U + (e_mean * r).square()
    tol = (r * wd).abs() * (e_mean + U * (xd.abs() if center else 0)) \
        + (ref - (b.double() if b is not None else 0)).abs() * (rel_r + 4 * U) \
        + (half_step(out) + 2 * U) * ref.abs() + tiny(out)
    assert y.dtype == out
    assert ((y.double() - ref).abs() <= 1.01 * tol).all()
    assert ((rstd.double() - r[:, 0]).abs() <= (r * (rel_r + 4 * U))[:, 0]).all()
    if center:
        assert ((mean.double() - m[:, 0]).abs() <= e_mean[:, 0] + 1e-40).all()
    else:
        assert mean is None


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("M,H,xt,wt,out,bias,pad", [
    (1, 1, F, F, F, True, 0),
    (1, 2560, BF, BF, BF, True, 0),
    (5, 2560, BF, F, BF, False, 0),
    (3, 8192, HF, HF, BF, True, 0),
    (2, 8191, BF, BF, F, True, 0),
    (70, 4096, F, BF, HF, True, 8),
    (9, 4104, F, F, F, True, 0),
    (2050, 256, HF, F, BF, True, 0),
    (2051, 1536, F, F, F, False, 16),
    (300, 2563, F, F, F, True, 5),
    (257, 1000, BF, BF, BF, True, 3),
    (64, 7, HF, HF, HF, True, 1),
    (40, 1029, BF, F, F, False, 0),
    (17, 3000, F, F, BF, True, 0),
    (17, 512, F, F, BF, True, 0),
    (17, 1024, BF, BF, BF, True, 0),
    (17, 2048, BF, BF, BF, True, 0),
])
def test_forward(center, M, H, xt, wt, out, bias, pad):
    x, w, b = _inputs(M, H, xt, wt, M + H, pad=pad)
    _check_fwd(x, w, b if bias else None, 1e-5, center, out)


def test_large_mean_and_unaligned_views():
    x, w, b = _inputs(33, 1024, F, F, 1, offset=1000.0)
    _check_fwd(x, w, b, 1e-6, True, F)
    big = torch.randn(33, 1025, device="cuda", generator=gen(2)).to(BF)
    wide = torch.randn(1025, device="cuda", generator=gen(3)).to(BF)
    _check_fwd(big[:, 1:], wide[1:], wide[:-1], 1e-6, True, BF)   # 2-byte aligned rows
    flat = torch.randn(8 * 512 + 1, device="cuda", generator=gen(4))
    _check_fwd(flat[1:].view(8, 512), torch.ones(512, device="cuda"), None, 1e-6, False, F)
    _check_fwd(big.contiguous()[:1, :1024], torch.ones(1024, device="cuda"), None, 1e-6, True, BF)


def test_constant_and_extreme_rows():
    H = 512
    x = torch.zeros(4, H, device="cuda")
    x[1] = 3.0
    x[2] = float("inf")
    x[3, 5] = float("nan")
    w, b = torch.ones(H, device="cuda"), torch.full((H,), 0.5, device="cuda")
    y, _, _ = qhead.layer_norm(x, w, b, 1e-5)
    assert (y[:2] == 0.5).all()          # no spread: the bias
    assert torch.isnan(y[2:]).all()      # only their own rows
    assert torch.isnan(qhead.layer_norm(x[:1], w, None, 0.0)[0]).all()


def _check_bwd(M, H, xt, dt, wt, center, pad=0, seed=0, want_dbias=True):
    x, w, _ = _inputs(M, H, xt, wt, seed + M + H, offset=0.5, pad=pad)
    dy = (torch.randn(M, H + pad, device="cuda", generator=gen(seed + 9)) * 1e-2).to(dt)[:, :H]
    _, mean, rstd = qhead.layer_norm(x, w, None, 1e-5, center=center)
    dx, dw, db = qhead.layer_norm_bwd(x, w, mean, rstd, dy, want_dbias=want_dbias)
    again = qhead.layer_norm_bwd(x, w, mean, rstd, dy, want_dbias=want_dbias)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    xd, wd, dd = x.double(), w.double(), dy.double()
    m = mean.double()[:, None] if center else 0.0
    r = rstd.double()[:, None]
    xh, g = (xd - m) * r, dd * wd
    c1 = g.mean(1, keepdim=True) if center else torch.zeros_like(r)
    c2 = (g * xh).mean(1, keepdim=True)
    ref = r * (g - c1 - xh * c2)
    xm = (xd.abs() + (m.abs() if center else 0.0)) * r     # bounds xh before cancellation
    mag = r * (g.abs() + g.abs().mean(1, keepdim=True) * (1 if center else 0)
               + xm * (g.abs() * xm).mean(1, keepdim=True))
    tol = 2 * D * U * mag + half_step(xt) * ref.abs() + tiny(xt)
    assert dx.dtype == xt
    assert ((dx.double() - ref).abs() <= 1.01 * tol).all()
    tol = (M + 8) * U * (dd.abs() * xm).sum(0)
    assert ((dw.double() - (dd * xh).sum(0)).abs() <= 1.01 * tol + 1e-40).all()
    if want_dbias:
        assert ((db.double() - dd.sum(0)).abs() <= 1.01 * M * U * dd.abs().sum(0) + 1e-40).all()
    else:
        assert db is None


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("M,H,xt,dt,wt,pad", [
    (1, 1, F, F, F, 0),
    (1, 2560, BF, F, BF, 0),
    (5, 2560, BF, BF, BF, 0),
    (611, 2560, BF, F, F, 0),
    (1300, 256, HF, BF, F, 8),
    (700, 4096, F, F, F, 0),
    (333, 8192, BF, BF, BF, 0),
    (100, 8191, F, F, F, 0),
    (50, 4097, HF, F, HF, 1),
    (411, 2563, F, F, F, 5),
    (2000, 7, F, HF, F, 0),
    (90, 3001, BF, BF, BF, 2),
])
def test_backward(center, M, H, xt, dt, wt, pad):
    _check_bwd(M, H, xt, dt, wt, center, pad)


def test_backward_without_dbias_and_empty():
    _check_bwd(37, 640, BF, F, F, True, want_dbias=False)
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    e = torch.empty(0, device="cuda")
    y, mean, rstd = qhead.layer_norm(x, w)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    dx, dw, db = qhead.layer_norm_bwd(x, w, e, e, x)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("center", [True, False])
def test_gradient_against_differences(center):
    """dx, dw and db contracted with a direction against the central
    difference of sum(y dy) in 64 bits."""
    M, H, eps = 6, 320, 1e-3
    x, w, b = _inputs(M, H, F, F, 11)
    dy = torch.randn(M, H, device="cuda", generator=gen(12))
    _, mean, rstd = qhead.layer_norm(x, w, b, eps, center=center)
    dx, dw, db = qhead.layer_norm_bwd(x, w, mean, rstd, dy)
    g = gen(13)
    ex, ew, eb = (torch.randn(s, device="cuda", generator=g, dtype=torch.float64)
                  for s in ((M, H), (H,), (H,)))

    def f(e):
        return (norm64(x.double() + e * ex, w.double() + e * ew, b.double() + e * eb, eps, center)
                * dy.double()).sum().item()

    e = 1e-4
    quot = (f(e) - f(-e)) / (2 * e)
    got = ((dx * ex).sum() + (dw * ew).sum() + (db * eb).sum()).item()
    mag = ((dx * ex).abs().sum() + (dw * ew).abs().sum() + (db * eb).abs().sum()).item()
    # the kernel's roundings (2 D half steps) and e^2 / 6 of third derivatives of order 10
    assert abs(quot - got) <= (4 * D * U + 10 * e * e) * mag


def test_graph_and_stream():
    x, w, b = _inputs(300, 768, BF, F, 21)
    dy = torch.randn(300, 768, device="cuda", generator=gen(22))

    def both():
        y, m, r = qhead.layer_norm(x, w, b)
        return (y, *qhead.layer_norm_bwd(x, w, m, r, dy))

    first = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = both()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(p, q) for p, q in zip(first, second))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = both()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, third))
