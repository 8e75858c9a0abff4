"""The bias gradient in a type of its own against 64 bits: the fp32 sum of the unrounded dz,
at most M half steps of the magnitudes off, and one rounding."""
import pytest
import torch

from ops_ref import U, gen, half_step, tiny
from test_linear_gpu import act_grad64, operands
from verify_vocab_blocked_gb300 import build as qbuild
from verify_vocab_blocked_gb300 import qhead
from verify_vocab_blocked_gb300.autograd import linear

pytestmark = pytest.mark.gpu
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qhead.lib()


@pytest.mark.parametrize("out", [F, HF, BF])
@pytest.mark.parametrize("M,K,N,t,act,dt", [(1, 8, 8, BF, "none", BF), (70, 64, 131, BF, "silu", BF), (600, 96, 264, HF, "gelu", HF),
                                            (2000, 64, 520, BF, "relu", F)])
def test_types(M, K, N, t, act, dt, out):
    x, w, _, _ = operands(M, K, N, t, M)
    _, pre = qhead.linear(x, w, None, act, want_pre=True)
    dy = torch.randn(M, N, device="cuda", generator=gen(N)).to(dt)
    dx, dw, db = qhead.linear_bwd(x, w, dy, pre, act, out)
    assert db.dtype == out and dx.dtype == dw.dtype == t
    z = pre.double()
    dz = dy.double() * act_grad64(z, act)
    e = (dy.double().abs() * 2.0 ** -20 * (1 + z.abs()) * (act not in ("none", "relu"))).sum(0)
    ref = dz.sum(0)
    assert ((db.double() - ref).abs() <= 1.01 * (e + M * U * dz.abs().sum(0) + half_step(out) * ref.abs()) + tiny(out)).all()
    plain = qhead.linear_bwd(x, w, dy, pre, act)
    assert torch.equal(plain[0], dx) and torch.equal(plain[1], dw) and plain[2].dtype == (F if dt == F else t)
    if out == F:
        assert torch.equal(plain[2], db.to(plain[2].dtype))


def test_a_sum_beyond_fp16():
    """70000 ones: exact in float32, infinite in fp16."""
    x, w = torch.ones(70000, 8, device="cuda", dtype=HF), torch.ones(16, 8, device="cuda", dtype=HF)
    dy = torch.ones(70000, 16, device="cuda", dtype=HF)
    assert (qhead.linear_bwd(x, w, dy, None, "none", F, want_dx=False, want_dw=False)[2] == 70000).all()
    assert torch.isinf(qhead.linear_bwd(x, w, dy, want_dx=False, want_dw=False)[2]).all()
    b = torch.zeros(16, device="cuda", requires_grad=True)
    linear(x, w, b).backward(dy)
    assert (b.grad == 70000).all()


def test_a_float32_bias_of_a_bf16_block():
    g = gen(5)
    x = torch.randn(5001, 64, device="cuda", generator=g).to(BF)
    w = torch.randn(264, 64, device="cuda", generator=g).to(BF)
    b = torch.randn(264, device="cuda", generator=g).requires_grad_(True)
    dy = torch.randn(5001, 264, device="cuda", generator=g).to(BF)
    linear(x, w, b).backward(dy)
    d = dy.double()
    assert ((b.grad.double() - d.sum(0)).abs() <= 5001 * U * d.abs().sum(0)).all()
    assert (b.grad.to(BF).float() != b.grad).any()


@pytest.mark.parametrize("out", [F, HF])
def test_no_rows(out):
    x, w, _, _ = operands(1, 8, 9, BF, 1)
    db = qhead.linear_bwd(x[:0], w, torch.zeros(0, 9, device="cuda", dtype=BF), None, "none", out)[2]
    assert db.dtype == out and db.shape == (9,) and not db.any()
