"""The residual's addition and the norm behind it, its 8-bit output and its
gradient, against 64 bits.

Tolerances are the norm's own (a sum along a row: 128 half steps of its
magnitudes) with the addition's rounding, a half step of fp32, beside them.  A code
is off by its rounding (half a step of e4m3: 2^-4 relative, 2^-10 at the least) and
by the error of y over the scale."""
import pytest
import torch

from ops_ref import U, gen, half_step, tiny
from verify_vocab_blocked_gb300 import build as qbuild
from verify_vocab_blocked_gb300 import qhead

pytestmark = pytest.mark.gpu
D = 128
BF, HF, F, E8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qhead.lib()


def inputs(M, H, xt, rt, wt, seed, pad=0, padr=0):
    g = gen(seed)
    x = (torch.randn(M, H + pad, device="cuda", generator=g) * 0.5).to(xt)[:, :H]
    r = (torch.randn(M, H + padr, device="cuda", generator=g) * 2 + 0.5).to(rt)[:, :H]
    w = (1 + 0.2 * torch.randn(H, device="cuda", generator=g)).to(wt)
    b = torch.randn(H, device="cuda", generator=g).to(wt)
    return x, r, w, b


def norm_and_tol(x, r, w, b, eps, center):
    """(t, y, tolerance of y, mean, its, 1/rstd's relative one, rstd) in 64 bits."""
    t = x.double() + (0 if r is None else r.double())
    m = t.mean(1, keepdim=True) if center else torch.zeros_like(t[:, :1])
    c = t - m
    rs = (c.square().mean(1, keepdim=True) + eps).rsqrt()
    wd = w.double()
    y0 = c * rs * wd
    y = y0 if b is None else y0 + b.double()
    e_mean = D * U * t.abs().mean(1, keepdim=True) if center else torch.zeros_like(rs)
    rel = D * U + (e_mean * rs).square()
    tol = (rs * wd).abs() * (e_mean + 2 * U * t.abs()) + y0.abs() * (rel + 4 * U) + 2 * U * y.abs()
    return t, y, tol, m, e_mean, rel, rs


SHAPES = [
    (1, 1, F, F, F, True, 0, 0), (5, 2560, BF, BF, BF, False, 0, 0), (3, 8192, HF, F, HF, True, 0, 0),
    (2, 8191, BF, BF, BF, True, 0, 0), (70, 4096, F, BF, BF, True, 8, 16), (9, 4104, F, F, F, True, 0, 0),
    (2050, 256, HF, F, F, True, 0, 0), (2049, 512, BF, HF, BF, True, 0, 8), (2051, 1536, BF, F, F, False, 16, 0),
    (300, 2563, F, F, F, True, 5, 0), (257, 1000, BF, BF, BF, True, 0, 3), (64, 7, HF, HF, HF, True, 1, 2),
    (2100, 1024, BF, BF, BF, True, 0, 0), (33, 1032, F, HF, BF, True, 0, 0), (40, 1029, BF, F, F, False, 0, 0),
    (17, 6150, BF, BF, BF, True, 0, 0), (13, 1544, F, F, F, True, 0, 0),
]


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("M,H,xt,rt,wt,bias,pad,padr", SHAPES)
def test_forward(center, M, H, xt, rt, wt, bias, pad, padr):
    x, r, w, b = inputs(M, H, xt, rt, wt, M + H, pad, padr)
    b = b if bias else None
    for out in (BF, F):
        y, total, mean, rstd = qhead.add_norm(x, r, w, b, 1e-5, center=center, out_dtype=out)
        t, ref, tol, m, e_mean, rel, rs = norm_and_tol(x, r, w, b, 1e-5, center)
        assert y.dtype == out and total.dtype == rt
        assert ((total.double() - t).abs() <= 1.01 * (half_step(rt) + U) * t.abs() + tiny(rt)).all()
        assert ((y.double() - ref).abs() <= 1.01 * (tol + half_step(out) * ref.abs()) + tiny(out)).all()
        assert ((rstd.double() - rs[:, 0]).abs() <= (rs * (rel + 4 * U))[:, 0]).all()
        if center:
            assert ((mean.double() - m[:, 0]).abs() <= 1.01 * e_mean[:, 0] + 1e-40).all()
        else:
            assert mean is None


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("M,H,xt,rt,wt,bias,pad,padr", SHAPES)
def test_8_bits(center, M, H, xt, rt, wt, bias, pad, padr):
    x, r, w, b = inputs(M, H, xt, rt, wt, M + H + 1, pad, padr)
    b = b if bias else None
    for res in (r, None):
        codes, scale, total = qhead.norm_8bit(x, w, b, 1e-5, residual=res, center=center)
        t, ref, tol, *_ = norm_and_tol(x, res, w, b, 1e-5, center)
        top = ref.abs().amax(1)
        e_top = (tol + half_step(F) * top[:, None]).amax(1)
        assert codes.dtype == E8 and scale.dtype == F
        assert ((scale.double() * 448 - top).abs() <= 1.01 * (e_top + 2 * U * top) + 1e-30).all()
        got = codes.double() * scale.double()[:, None]
        s = (top / 448)[:, None]
        assert ((got - ref).abs() <= 1.01 * (tol + e_top[:, None] + 2.0 ** -4 * ref.abs() + 2.0 ** -10 * s)).all()
        assert (codes.double().abs() <= 448).all()
        if res is None:
            assert total is None
        else:
            assert torch.equal(total, qhead.add_norm(x, r, w, b, 1e-5, center=center)[1])


def test_rows_without_spread_or_of_no_value():
    H = 512
    x, r = torch.zeros(5, H, device="cuda"), torch.zeros(5, H, device="cuda")
    r[1], r[2], r[3, 5] = 3.0, float("inf"), float("nan")
    w, b = torch.ones(H, device="cuda"), torch.full((H,), 0.5, device="cuda")
    y, total, _, _ = qhead.add_norm(x, r, w, b, 1e-5)
    assert (y[[0, 1, 4]] == 0.5).all() and torch.isnan(y[2:4]).all() and torch.isinf(total[2]).all()
    codes, scale, _ = qhead.norm_8bit(x, w, None, 1e-5, residual=r)
    assert (codes[[0, 1, 4]].float() == 0).all() and torch.isnan(codes[2:4].float()).all()
    assert torch.isfinite(scale[[0, 1, 4]]).all()
    # 8-bit rows of zeros through the product: the bias alone
    one = torch.ones(16, H, device="cuda").to(E8)
    y = qhead.linear(codes, one, b[:16].contiguous(), x_scale=scale, w_scale=torch.ones(16, device="cuda"))
    assert (y[[0, 1, 4]] == 0.5).all() and torch.isnan(y[2:4]).all()
    assert qhead.add_norm(x[:0], r[:0], w)[0].shape == (0, H)
    assert qhead.norm_8bit(x[:0], w)[0].shape == (0, H)


def test_unaligned_views():
    g = gen(2)
    wide = torch.randn(33, 1026, device="cuda", generator=g).to(BF)
    w = torch.randn(1026, device="cuda", generator=g).to(BF)
    x, r, ww = wide[:, 1:1025], wide[:, 2:], w[1:1025]
    y, total, mean, rstd = qhead.add_norm(x, r, ww)
    z = qhead.add_norm(x.contiguous(), r.contiguous(), ww.contiguous())
    assert ((y.float() - z[0].float()).abs() <= 2.0 ** -7 * z[0].float().abs() + 1e-6).all()
    assert torch.equal(total, z[1])


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("M,H,tt,dt,wt,pad", [
    (1, 1, F, F, F, 0), (5, 2560, BF, BF, BF, 0), (300, 2563, F, F, F, 5), (64, 7, HF, HF, HF, 1),
    (700, 1536, F, BF, BF, 0), (3000, 256, BF, F, F, 8), (90, 4096, F, F, F, 0), (60, 6280, F, F, F, 0),
    (50, 8192, F, F, F, 0), (50, 8192, BF, F, BF, 0), (40, 5000, BF, BF, BF, 0), (1300, 1000, BF, BF, HF, 3),
    (2000, 2048, HF, F, F, 0), (33, 8191, F, BF, F, 0),
])
def test_gradient(center, M, H, tt, dt, wt, pad):
    t, _, w, _ = inputs(M, H, tt, F, wt, M + H, pad)
    g = gen(M)
    dy = (torch.randn(M, H + pad, device="cuda", generator=g) * 1e-2).to(dt)[:, :H]
    ds = (torch.randn(M, H + pad, device="cuda", generator=g) * 1e-2).to(tt)[:, :H]
    _, mean, rstd = qhead.layer_norm(t, w, None, 1e-5, center=center)
    dx, dw, db = qhead.add_norm_bwd(t, w, mean, rstd, dy, ds)
    bare = qhead.layer_norm_bwd(t, w, mean, rstd, dy)
    again = qhead.add_norm_bwd(t, w, mean, rstd, dy, ds)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))
    none = qhead.add_norm_bwd(t, w, mean, rstd, dy)
    assert all(torch.equal(p, q) for p, q in zip(none, bare))
    td, wd, dd = t.double(), w.double(), dy.double()
    rs = rstd.double()[:, None]
    m = mean.double()[:, None] if center else 0.0
    xh, gw = (td - m) * rs, dd * wd
    c1 = gw.mean(1, keepdim=True) if center else 0.0
    c2 = (gw * xh).mean(1, keepdim=True)
    own = rs * (gw - c1 - xh * c2)
    ref = own + ds.double()
    a1 = gw.abs().mean(1, keepdim=True) if center else 0.0
    # xh itself is off by the subtraction's and the product's rounding
    e_xh = 3 * U * rs * (td.abs() + (m.abs() if center else 0))
    e_c2 = D * U * (gw * xh).abs().mean(1, keepdim=True) + (gw.abs() * e_xh).mean(1, keepdim=True)
    tol = rs * (D * U * a1 + xh.abs() * e_c2 + e_xh * c2.abs() + 4 * U * (gw.abs() + a1 + (xh * c2).abs()))
    assert ((dx.double() - ref).abs() <= 1.01 * (tol + (half_step(tt) + U) * ref.abs() + U * own.abs()) + tiny(tt)).all()
    for got, terms, extra in ((dw, dd * xh, dd.abs() * e_xh), (db, dd, 0 * dd)):
        r = terms.sum(0)
        assert ((got.double() - r).abs() <= 1.01 * (M * U * terms.abs().sum(0) + extra.sum(0) + 2 * U * r.abs()) + 1e-40).all()
    # the parameter gradients are the norm's own (one row a step instead of two may
    # group the sums otherwise), and by differences the addition is 1 : 1
    assert ((dw - bare[1]).abs() <= 2 * M * U * (dd * xh).abs().sum(0) + 1e-30).all()


def test_gradient_against_differences():
    g = gen(3)
    M, H = 12, 96
    x, r, w, b = inputs(M, H, F, F, F, 3)
    dy, ds = torch.randn(M, H, device="cuda", generator=g), torch.randn(M, H, device="cuda", generator=g)
    _, total, mean, rstd = qhead.add_norm(x, r, w, b, 1e-5)
    dx, dw, db = (v.double() for v in qhead.add_norm_bwd(total, w, mean, rstd, dy, ds))

    def loss(xx, ww, bb):
        t = xx + r.double()
        c = t - t.mean(1, keepdim=True)
        y = c * (c.square().mean(1, keepdim=True) + 1e-5).rsqrt() * ww + bb
        return (y * dy.double()).sum() + (t * ds.double()).sum()

    at = [x.double(), w.double(), b.double()]
    for k, grad in enumerate((dx, dw, db)):
        v = torch.randn(grad.shape, device="cuda", generator=g, dtype=torch.float64)
        up, down = list(at), list(at)
        up[k], down[k] = at[k] + 1e-4 * v, at[k] - 1e-4 * v
        diff = (loss(*up) - loss(*down)) / 2e-4
        assert abs((grad * v).sum() - diff) <= 1e-5 * (grad * v).abs().sum() + 1e-5
