"""Tensors of more than 2^31 elements through the block between norm and head and the
clipping: the rows and columns at the start, at the 2^31st element and at the end, with the
tolerances of the shorter cases."""
import pytest
import torch

from ops_ref import U, half_step, tiny
from test_add_norm_gpu import norm_and_tol
from test_linear_gpu import ACTS, act_grad64, accumulated
from verify_vocab_blocked_gb300 import build as qbuild
from verify_vocab_blocked_gb300 import qhead

pytestmark = pytest.mark.gpu
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qhead.lib()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    yield
    torch.cuda.empty_cache()


def randn(g, *shape, dtype=BF):
    return torch.randn(*shape, device="cuda", generator=g, dtype=dtype)


def some_rows(M, N):
    at = 2 ** 31 // N
    return torch.tensor([0, 1, at - 1, at, at + 1, 2 * at - 1 if 2 * at - 1 < M else M - 3, M - 2, M - 1], device="cuda")


@pytest.mark.parametrize("M,N,out", [(230_001, 10240, BF), (230_001, 10240, F), (240_001, 9001, BF)])
def test_linear(M, N, out):
    """Rows that TMA writes, and others; a residual of a wider tensor."""
    K = 64
    g = torch.Generator(device="cuda").manual_seed(N)
    x, w, b = randn(g, M, K), randn(g, N, K) / 8, randn(g, N)
    r = randn(g, M, N + 8)[:, :N]
    y, pre = qhead.linear(x, w, b, "silu", r, out_dtype=out, want_pre=True)
    at = some_rows(M, N)
    z = x[at].double() @ w.double().t() + b.double()
    mag = x[at].double().abs() @ w.double().abs().t() + b.double().abs()
    ref = ACTS["silu"](z) + r[at].double()
    tol = 1.13 * accumulated(K, mag) + 2.0 ** -20 * (1 + z.abs()) + (half_step(out) + 2.0 ** -23) * ref.abs() + tiny(out)
    assert ((y[at].double() - ref).abs() <= 1.01 * tol).all()
    assert ((pre[at].double() - z).abs() <= 1.01 * (accumulated(K, mag) + (2.0 ** -11 + 2.0 ** -23) * z.abs() + tiny(HF))).all()
    del y, r
    if out == F:
        return
    dy = randn(g, M, N)
    dx, dw, db = qhead.linear_bwd(x, w, dy, pre, "silu", F)
    dz = dy[at].double() * act_grad64(pre[at].double(), "silu")
    e = dy[at].double().abs() * 2.0 ** -20 * (1 + pre[at].double().abs()) + half_step(BF) * dz.abs() + tiny(BF)
    ref = dz @ w.double()
    tol = e @ w.double().abs() + accumulated(N, 1.01 * dz.abs() @ w.double().abs()) + half_step(BF) * ref.abs() + tiny(BF)
    assert ((dx[at].double() - ref).abs() <= 1.01 * tol).all()
    cols = torch.tensor([0, 7, N // 2, N - 1], device="cuda")
    d, p = dy[:, cols].double(), pre[:, cols].double()
    dz = d * act_grad64(p, "silu")
    e = d.abs() * 2.0 ** -20 * (1 + p.abs())
    assert ((db[cols].double() - dz.sum(0)).abs() <= 1.01 * (e.sum(0) + M * U * dz.abs().sum(0)) + tiny(F)).all()
    e = e + half_step(BF) * dz.abs() + tiny(BF)
    ref, xd = dz.t() @ x.double(), x.double().abs()
    tol = e.t() @ xd + accumulated(M, 1.01 * dz.abs().t() @ xd) + half_step(BF) * ref.abs() + tiny(BF)
    assert ((dw[cols].double() - ref).abs() <= 1.01 * tol).all()


@pytest.mark.parametrize("M,K", [(230_001, 10240), (240_001, 9001)])
def test_linear_of_many_inputs(M, K):
    """x beyond 2^31 elements, as it lies and through the copy to aligned rows."""
    g = torch.Generator(device="cuda").manual_seed(K)
    x, w = randn(g, M, K), randn(g, 72, K) / K ** 0.5
    y = qhead.linear(x, w)
    at = some_rows(M, K)
    ref = x[at].double() @ w.double().t()
    tol = accumulated(K, x[at].double().abs() @ w.double().abs().t()) + half_step(BF) * ref.abs() + tiny(BF)
    assert ((y[at].double() - ref).abs() <= 1.01 * tol).all()


@pytest.mark.parametrize("M,H", [(1_050_001, 2048), (840_001, 2563)])
def test_add_norm(M, H):
    g = torch.Generator(device="cuda").manual_seed(H)
    x, r, w = randn(g, M, H), randn(g, M, H), 1 + randn(g, H) / 8
    y, total, mean, rstd = qhead.add_norm(x, r, w)
    codes, scale, _ = qhead.norm_8bit(x, w, residual=r)
    at = some_rows(M, H)
    t, ref, tol, *_, rs = norm_and_tol(x[at], r[at], w, None, 1e-6, True)
    assert ((total[at].double() - t).abs() <= 1.01 * (half_step(BF) + U) * t.abs()).all()
    assert ((y[at].double() - ref).abs() <= 1.01 * (tol + half_step(BF) * ref.abs()) + tiny(BF)).all()
    top = ref.abs().amax(1, keepdim=True)
    e_top = tol.amax(1, keepdim=True) + half_step(F) * top
    got = codes[at].double() * scale[at].double()[:, None]
    assert ((got - ref).abs() <= 1.01 * (tol + e_top + 2.0 ** -4 * ref.abs() + 2.0 ** -10 * top / 448)).all()
    del x, r, y, codes
    dy, dt = randn(g, M, H), randn(g, M, H)
    dx, dw, db = qhead.add_norm_bwd(total, w, mean, rstd, dy, dt)
    m, rs = mean[at].double()[:, None], rstd[at].double()[:, None]
    td, gw = total[at].double(), dy[at].double() * w.double()
    xh = (td - m) * rs
    own = rs * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True))
    ref = own + dt[at].double()
    xm = (td.abs() + m.abs()) * rs
    mag = rs * (gw.abs() + gw.abs().mean(1, keepdim=True) + xm * (gw.abs() * xm).mean(1, keepdim=True))
    assert ((dx[at].double() - ref).abs() <= 1.01 * (2 * 128 * U * mag + (half_step(BF) + U) * ref.abs()) + tiny(BF)).all()
    cols = torch.tensor([0, 7, H // 2, H - 1], device="cuda")
    d = dy[:, cols].double()
    assert ((db[cols].double() - d.sum(0)).abs() <= 1.01 * M * U * d.abs().sum(0)).all()
    xh = (total[:, cols].double() - mean.double()[:, None]) * rstd.double()[:, None]
    xm = (total[:, cols].double().abs() + mean.double().abs()[:, None]) * rstd.double()[:, None]
    assert ((dw[cols].double() - (d * xh).sum(0)).abs() <= 1.01 * (M + 8) * U * (d.abs() * xm).sum(0)).all()


def test_clip():
    n = 2 ** 31 + 8191
    g = torch.Generator(device="cuda").manual_seed(1)
    ts = [randn(g, 5), randn(g, n), randn(g, 1000, dtype=F)]
    want = sum(t.float().square().sum(dtype=torch.float64) for t in ts).sqrt()
    out = [torch.empty_like(t) for t in ts]
    norm = qhead.clip_grads(ts, 1.0, out=out)
    assert abs(norm.double() - want) <= 40 * U * want
    coef = 1.0 / (float(want) + 1e-6)
    for a, b in ((out[0], ts[0]), (out[2], ts[2]), *((out[1][i:i + 20000], ts[1][i:i + 20000]) for i in (0, 2 ** 31 - 10000, n - 20000))):
        ref = b.double() * coef
        assert ((a.double() - ref).abs() <= 1.01 * (half_step(a.dtype) + 44 * U) * ref.abs() + tiny(a.dtype)).all()
