"""Products whose every partial sum fp32 holds are exact, whichever kernel, tile and split
they take: an identity, one-hot rows and small integers.  Such a sum is a whole number of
units below 2^24 of them, in any order and grouping, so that nothing is rounded before the
output's own type."""
import pytest
import torch

from ops_ref import gen
from verify_vocab_blocked_gb300 import build as qbuild
from verify_vocab_blocked_gb300 import qhead

pytestmark = pytest.mark.gpu
BF, HF, F, E8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qhead.lib()


# pairs in tiles of 256 and 128 columns, with tiles whose reduction is shared; few rows in
# tiles of 16, 32, 64 and 128, alone and in several parts; rows that are padded
SHAPES = [(4096, 1024, 4096), (2048, 2560, 2560), (600, 4096, 600), (700, 5003, 520), (300, 4100, 601), (130, 1024, 128),
          (5, 2560, 2560), (3, 10240, 300), (16, 4096, 20000), (30, 2560, 1000), (64, 2560, 2560), (100, 1541, 700),
          (128, 10240, 256), (301, 1536, 1536), (512, 2560, 300), (7, 1, 3)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("t", [BF, HF])
def test_integers(M, K, N, t):
    """Factors up to 15: sums below 10240 x 225 = 2.3e6."""
    g = gen(M + K + N)
    for lo in (-15, 0):
        x = torch.randint(lo, 16, (M, K), device="cuda", generator=g).to(t)
        w = torch.randint(lo, 16, (N, K), device="cuda", generator=g).to(t)
        b = torch.randint(-99, 99, (N,), device="cuda", generator=g).float()
        ref = x.double() @ w.double().t() + b.double()
        assert torch.equal(qhead.linear(x, w, b, out_dtype=F).double(), ref)
        assert torch.equal(qhead.linear(x, w, b, out_dtype=BF), ref.to(BF))


@pytest.mark.parametrize("M,K,N", SHAPES[:-1])
def test_one_hot_rows(M, K, N):
    """Each row picks one column of the weights."""
    g = gen(K)
    w = torch.randn(N, K, device="cuda", generator=g).to(BF)
    at = torch.randint(0, K, (M,), device="cuda", generator=g)
    x = torch.zeros(M, K, device="cuda", dtype=BF)
    x[torch.arange(M, device="cuda"), at] = 1
    assert torch.equal(qhead.linear(x, w, out_dtype=F), w.t()[at].float())


@pytest.mark.parametrize("M", [5, 64, 300, 3000])
@pytest.mark.parametrize("K", [1024, 2560])
def test_identity(M, K):
    x = torch.randn(M, K, device="cuda", generator=gen(M)).to(BF)
    assert torch.equal(qhead.linear(x, torch.eye(K, device="cuda", dtype=BF), out_dtype=F), x.float())


@pytest.mark.parametrize("M,K,N", [(5, 2560, 2560), (100, 10240, 256), (300, 4096, 600), (2048, 2560, 2560)])
def test_integers_of_8_bits(M, K, N):
    g = gen(M)
    x = torch.randint(-15, 16, (M, K), device="cuda", generator=g).float()
    w = torch.randint(-15, 16, (N, K), device="cuda", generator=g).float()
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    y = qhead.linear(x.to(E8), w.to(E8), x_scale=one(M), w_scale=one(N), out_dtype=F)
    assert torch.equal(y.double(), x.double() @ w.double().t())


@pytest.mark.parametrize("M,K,N", [(600, 4096, 600), (5, 2560, 2560), (5000, 256, 300)])
def test_integers_of_the_gradient(M, K, N):
    g = gen(N)
    r = lambda *s: torch.randint(-3, 4, s, device="cuda", generator=g).to(HF)  # noqa: E731
    x, w, dy = r(M, K), r(N, K), r(M, N)
    dx, dw, db = qhead.linear_bwd(x, w, dy)
    assert torch.equal(dx, (dy.double() @ w.double()).to(HF)) and torch.equal(dw, (dy.double().t() @ x.double()).to(HF))
    assert torch.equal(db.double(), dy.double().sum(0).to(db.dtype).double())
