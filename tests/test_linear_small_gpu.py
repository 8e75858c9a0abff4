"""The gradient behind pre-activations too small for fp16 but not for bf16 operands: relu's
is that of the 64-bit z wherever its sign is beyond doubt.

dz is dy or 0 exactly, and in bf16 as it was given, so that only the products' sums and the
outputs' rounding are off."""
import pytest
import torch

from ops_ref import gen, half_step, tiny
from test_linear_gpu import accumulated
from verify_vocab_blocked_gb300 import build as qbuild
from verify_vocab_blocked_gb300 import qhead
from verify_vocab_blocked_gb300.autograd import linear

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qhead.lib()


# every form of the epilogue: few rows, pairs and shared tiles, of aligned rows and others
@pytest.mark.parametrize("M,K,N", [(5, 64, 128), (5, 64, 131), (1, 2560, 72), (300, 64, 264), (300, 64, 263), (600, 4096, 600),
                                   (600, 4096, 601), (1300, 128, 256)])
@pytest.mark.parametrize("size", [1e-5, 1e-9, 1e-18])
def test_relu(M, K, N, size):
    g = gen(M + N)
    x = (torch.randn(M, K, device="cuda", generator=g) * size).to(BF)
    w = (torch.randn(N, K, device="cuda", generator=g) * size).to(BF)
    dy = torch.randn(M, N, device="cuda", generator=g).to(BF)
    z = x.double() @ w.double().t()
    sure = z.abs() > accumulated(K, x.double().abs() @ w.double().abs().t())
    dy = torch.where(sure, dy, 0)
    _, pre = qhead.linear(x, w, None, "relu", want_pre=True)
    assert ((pre > 0) == (z > 0))[sure].all() and torch.isfinite(pre).all()
    dx, dw, db = qhead.linear_bwd(x, w, dy, pre, "relu")
    dz = dy.double() * (z > 0)
    for got, ref, mag, n in ((dx, dz @ w.double(), dz.abs() @ w.double().abs(), N),
                             (dw, dz.t() @ x.double(), dz.abs().t() @ x.double().abs(), M), (db, dz.sum(0), dz.abs().sum(0), M)):
        tol = accumulated(n, mag) + half_step(BF) * ref.abs() + tiny(BF)
        assert ((got.double() - ref).abs() <= 1.01 * tol).all()
    assert dw.any() and dx.any()


def test_relu_of_zeros_and_signs():
    """Exactly 0 passes nothing; the smallest values keep their sign."""
    x = torch.tensor([[0.0], [-0.0], [2.0 ** -30], [-2.0 ** -30], [2.0 ** -25], [2.0 ** -100], [1.0]], device="cuda").to(BF)
    one = torch.ones(1, 1, device="cuda", dtype=BF)
    y, pre = qhead.linear(x, one, None, "relu", want_pre=True, out_dtype=F)
    assert torch.equal(y[:, 0], x[:, 0].float().clamp_min(0))
    assert torch.equal(pre[:, 0].sign(), x[:, 0].sign().half())
    dx = qhead.linear_bwd(x, one, torch.ones(7, 1, device="cuda", dtype=BF), pre, "relu")[0]
    assert dx[:, 0].tolist() == [0, 0, 1, 0, 1, 1, 1]


def test_autograd_of_a_small_layer():
    g = gen(3)
    x = (1e-5 * torch.rand(70, 64, device="cuda", generator=g)).to(BF).requires_grad_(True)
    w = (1e-5 * torch.rand(32, 64, device="cuda", generator=g)).to(BF).requires_grad_(True)
    y = linear(x, w, None, "relu")
    assert (y > 0).all() and (y < 2.0 ** -25).all()
    y.sum().backward()
    ref = w.detach().double().sum(0).expand(70, 64)
    assert ((x.grad.double() - ref).abs() <= 1.01 * half_step(BF) * ref + accumulated(32, ref)).all()
