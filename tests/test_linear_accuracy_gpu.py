"""float32 outputs: the error over the result's norm.

The tensor cores truncate a running sum at each of the 32 MMAs that are summed there: half
a step in the mean, at most 2^-24 of the running sum, which for positive operands grows
evenly, so that the whole sum loses 16.5 x 2^-24 of itself (9.8e-7; less by where it lies
between two powers of two, and for operands of both signs).  These sums are added with
fp32 roundings, which in the root of the mean square are below sqrt(their number) x 2^-24.

Before an MMA's 16 products are added to the sum, each is itself cut at 2^-25 of the
largest term's power of two (as 15 x 2^-25 beside 1 show, which arrive whole, and
15 x 2^-26, of which nothing does).  A product of two bf16 has 16 bits: one that is
2^-10 of the sum or more ends above that.  A product of two fp16 has 22, so that up to 16
products lose half of 2^-25 in the mean, 4 x 2^-24 together, beside the sum's own 2^-24: 5
times as much."""
import pytest
import torch

from ops_ref import U, gen
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


def off(y, ref):
    return ((y.double() - ref).norm() / ref.norm()).item()


@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("M,K,N", [
    # pairs, shared tiles
    (2048, 2560, 2560), (600, 4096, 600), (700, 10240, 520), (1024, 1024, 4096),
    # few rows: long reductions in few parts, in tiles of 16 to 128
    (5, 2560, 10240), (16, 10240, 10240), (5, 14336, 70000), (30, 14336, 1000), (40, 10240, 20000), (64, 10240, 2560),
    (128, 2560, 10240), (128, 10240, 2560), (200, 28672, 2000), (300, 14336, 5120), (512, 10240, 2560), (301, 1541, 2563),
])
def test_float32_output(M, K, N, positive, t):
    g = gen(M + K + N)
    x = torch.randn(M, K, device="cuda", generator=g).to(t)
    w = (torch.randn(N, K, device="cuda", generator=g) / K ** 0.5).to(x.dtype)
    if positive:
        x, w = x.abs(), w.abs()
    limit = (16.5 * (1 if t == BF else 5) + (K / 512 + 1) ** 0.5) * U
    assert off(qhead.linear(x, w, out_dtype=F), x.double() @ w.double().t()) <= limit


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("M,K,N", [(2048, 10240, 2560), (600, 8192, 600), (128, 40960, 256), (5, 2560, 10240), (300, 20480, 3000)])
def test_float32_output_of_8_bits(M, K, N, positive):
    """Products of 8 bits end above the cut; 128 MMAs a sum; the scales add three roundings."""
    g = gen(M + K + N)
    x, w = torch.randn(M, K, device="cuda", generator=g), torch.randn(N, K, device="cuda", generator=g)
    if positive:
        x, w = x.abs(), w.abs()
    xs, ws = x.abs().amax(1) / 448, w.abs().amax(1) / 448
    x, w = (x / xs[:, None]).to(torch.float8_e4m3fn), (w / ws[:, None]).to(torch.float8_e4m3fn)
    ref = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    limit = (64.5 + (K / 4096 + 1) ** 0.5 + 3) * U
    assert off(qhead.linear(x, w, x_scale=xs, w_scale=ws, out_dtype=F), ref) <= limit
