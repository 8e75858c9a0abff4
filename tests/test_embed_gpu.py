"""Embedding lookup from the packed table and its gradient against the plain
64-bit forms.

Tolerances.  Lookup: one FMA and one product in fp32 (half a step each), one
rounding to the output type.  Gradient: a sum of n fp32 terms in any grouping
is off by at most (n - 1) half steps of the sum of magnitudes, the scale and
the addition into dw by one each."""
import pytest
import torch

from ops_ref import U, gen, half_step, make_table, table64, tiny
from verify_vocab_blocked_gb300 import build as qbuild
from verify_vocab_blocked_gb300 import qhead

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qhead.lib()


def _head(V, H, bits, seed=0, sb=torch.float16):
    return qhead.Head(*make_table(V, H, bits, seed, sb), bits)


def _tokens(M, V, kind, seed):
    if kind == "same":
        return torch.full((M,), V - 1, dtype=torch.int32, device="cuda")
    u = torch.rand(M, device="cuda", generator=gen(seed), dtype=torch.float64)
    if kind == "skewed":
        return ((V + 1.0) ** u - 1).long().clamp(0, V - 1).int()
    return (u * V).long().clamp(0, V - 1).int()


@pytest.mark.parametrize("M,V,H,bits,sb,out", [
    (1, 1, 128, 4, torch.float16, torch.bfloat16),
    (5, 1000, 2560, 4, torch.float16, torch.bfloat16),
    (7, 333, 1536, 8, torch.float16, torch.float32),
    (1000, 777, 640, 4, torch.bfloat16, torch.float16),
    (4099, 513, 384, 8, torch.float32, torch.bfloat16),
    (33, 64, 8192, 4, torch.float32, torch.float32),
])
def test_lookup(M, V, H, bits, sb, out):
    head = _head(V, H, bits, M, sb)
    t = _tokens(M, V, "uniform", M)
    scale = 50.596
    y = qhead.embed(head, t, scale, out_dtype=out)
    ref = torch.tensor(scale, dtype=torch.float32).double().item() * \
        table64(head.wq, head.scales, head.biases, bits)[t.long()]
    assert y.dtype == out and y.shape == (M, H)
    # q s and its sum with b may cancel: the FMA's half step is of the result
    tol = (half_step(out) + 2.1 * U) * ref.abs() + 2 * tiny(out)
    assert ((y.double() - ref).abs() <= tol).all()


def test_lookup_mask_and_bad_tokens():
    V, H, M = 100, 256, 9
    head = _head(V, H, 4)
    t = torch.tensor([0, 99, 100, -1, 5, 2 ** 31 - 1, -2 ** 31, 7, 100], dtype=torch.int32,
                     device="cuda")
    mask = torch.tensor([1, 1, 1, 1, 0, 1, 0, 255, 0], dtype=torch.uint8, device="cuda")
    y = qhead.embed(head, t, 2.0, mask)
    good = [0, 1, 7]
    assert torch.equal(y[good], qhead.embed(head, t[good], 2.0))
    assert torch.isnan(y[[2, 3, 5]]).all()
    assert (y[[4, 6, 8]] == 0).all()
    assert torch.equal(y.nan_to_num(7.0), qhead.embed(head, t, 2.0, mask.bool()).nan_to_num(7.0))


def test_lookup_far_row():
    """Rows of the table past 2^31 bytes."""
    V, H = 1_300_000, 2560
    wq = torch.zeros(V, H // 4, dtype=torch.int32, device="cuda")
    s = torch.ones(V, H // 64, dtype=torch.float16, device="cuda")
    b = torch.zeros(V, H // 64, dtype=torch.float16, device="cuda")
    wq[V - 1] = 0x04030201
    y = qhead.embed(qhead.Head(wq, s, b, 8), torch.tensor([V - 1, 0], dtype=torch.int32,
                                                          device="cuda"))
    want = torch.tensor([1.0, 2.0, 3.0, 4.0], device="cuda").repeat(H // 4)
    assert torch.equal(y[0].float(), want) and (y[1] == 0).all()


def _check_grad(M, V, H, kind, dtype, add, masked, scale=0.75, seed=3):
    head = _head(V, H, 4, seed)
    t = _tokens(M, V, kind, seed)
    dy = torch.randn(M, H, device="cuda", generator=gen(seed + 1)).to(dtype)
    mask = torch.rand(M, device="cuda", generator=gen(seed + 2)) < 0.7 if masked else None
    dw0 = torch.randn(V, H, device="cuda", generator=gen(seed + 4)) if add else None
    got = qhead.embed_bwd(head, t, dy, scale, mask, dw=dw0.clone() if add else None)
    again = qhead.embed_bwd(head, t, dy, scale, mask, dw=dw0.clone() if add else None)
    assert torch.equal(got, again)
    keep = torch.ones(M, dtype=torch.bool, device="cuda") if mask is None else mask
    ref = torch.zeros(V, H, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    n = torch.zeros(V, dtype=torch.float64, device="cuda")
    ref.index_add_(0, t[keep].long(), scale * dy[keep].double())
    mag.index_add_(0, t[keep].long(), scale * dy[keep].double().abs())
    n.index_add_(0, t[keep].long(), torch.ones(int(keep.sum()), dtype=torch.float64, device="cuda"))
    tol = (n[:, None] + 1) * U * mag
    if add:
        ref += dw0.double()
        tol = tol + U * ref.abs()
        assert torch.equal(got[n == 0], dw0[n == 0])
    else:
        assert (got[n == 0] == 0).all()
    assert ((got.double() - ref).abs() <= 1.01 * tol + 1e-40).all()


@pytest.mark.parametrize("M,V,H,kind,dtype,add,masked", [
    (1, 1, 128, "uniform", torch.float32, False, False),
    (1, 5000, 2560, "uniform", torch.bfloat16, True, False),
    (31, 3, 256, "uniform", torch.float16, False, False),
    (32, 10, 128, "same", torch.float32, True, False),
    (33, 600, 128, "same", torch.float32, False, False),
    (1025, 512, 384, "skewed", torch.bfloat16, False, True),
    (2048, 513, 1536, "skewed", torch.float32, True, True),
    (2049, 40000, 256, "skewed", torch.float32, False, False),
    (5003, 262144, 128, "uniform", torch.bfloat16, False, True),
    (20011, 270000, 128, "skewed", torch.bfloat16, True, False),
    (9000, 2, 128, "uniform", torch.float32, False, False),
    (4097, 100, 8192, "skewed", torch.float16, False, False),
    (70001, 131072, 128, "skewed", torch.float32, True, True),
])
def test_gradient(M, V, H, kind, dtype, add, masked):
    _check_grad(M, V, H, kind, dtype, add, masked)


def test_gradient_all_masked_or_out_of_range():
    V, H, M = 50, 256, 100
    head = _head(V, H, 8)
    dy = torch.ones(M, H, device="cuda")
    t = torch.full((M,), 3, dtype=torch.int32, device="cuda")
    off = torch.zeros(M, dtype=torch.bool, device="cuda")
    assert (qhead.embed_bwd(head, t, dy, 1.0, off) == 0).all()
    t[:50], t[50:] = -1, V
    assert (qhead.embed_bwd(head, t, dy) == 0).all()
    dw = torch.ones(V, H, device="cuda")
    assert (qhead.embed_bwd(head, t, dy, dw=dw) == 1).all()
    # a NaN gradient of a masked row stays out
    t[:] = 3
    dy[7] = float("nan")
    on = torch.ones(M, dtype=torch.bool, device="cuda")
    on[7] = False
    got = qhead.embed_bwd(head, t, dy, 1.0, on)
    assert (got[3] == 99).all() and not torch.isnan(got).any()


def test_empty():
    head = _head(20, 128, 4)
    t = torch.empty(0, dtype=torch.int32, device="cuda")
    assert qhead.embed(head, t).shape == (0, 128)
    assert (qhead.embed_bwd(head, t, torch.empty(0, 128, device="cuda")) == 0).all()
    dw = torch.ones(20, 128, device="cuda")
    assert (qhead.embed_bwd(head, t, torch.empty(0, 128, device="cuda"), dw=dw) == 1).all()


def test_gradient_against_differences():
    """The lookup is linear in the scales: the gradient contracted with a
    direction in the table is the difference quotient of sum(y dy)."""
    V, H, M = 64, 256, 40
    wq, s, b = make_table(V, H, 4, 5, torch.float32)
    t = _tokens(M, V, "skewed", 6)
    dy = torch.randn(M, H, device="cuda", generator=gen(7))
    g = qhead.embed_bwd(qhead.Head(wq, s, b, 4), t, dy, 2.0).double()
    d = torch.randn(V, H // 64, device="cuda", generator=gen(8))

    def f(e):
        y = qhead.embed(qhead.Head(wq, s, b + e * d, 4), t, 2.0, out_dtype=torch.float32)
        return (y.double() * dy.double()).sum().item()

    e = 2.0 ** -6
    quot = (f(e) - f(-e)) / (2 * e)
    want = (g.view(V, H // 64, 64).sum(2) * d.double()).sum().item()
    # roundings of b + e d and of y, two half steps of values below 0.5 each
    slack = 4 * U * 0.5 * 2.0 * dy.double().abs().sum().item() / e
    assert abs(quot - want) <= slack


def test_other_stream_and_graph():
    V, H, M = 3000, 512, 700
    head = _head(V, H, 4)
    t = _tokens(M, V, "skewed", 1)
    dy = torch.randn(M, H, device="cuda", generator=gen(2))
    y0, g0 = qhead.embed(head, t, 3.0), qhead.embed_bwd(head, t, dy, 3.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y1, g1 = qhead.embed(head, t, 3.0), qhead.embed_bwd(head, t, dy, 3.0)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y0, y1) and torch.equal(g0, g1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, g2 = qhead.embed(head, t, 3.0), qhead.embed_bwd(head, t, dy, 3.0)
    t.copy_(t.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, y0.flip(0))
    assert torch.equal(g2, qhead.embed_bwd(head, t, dy, 3.0))


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("M,V,H,kind,dtype,masked", [
    (2, 7, 128, "same", torch.bfloat16, False),
    (127, 40, 256, "skewed", torch.float32, True),
    (96, 100, 2560, "same", torch.bfloat16, False),
    (97, 100, 2560, "skewed", torch.bfloat16, True),
    (32, 128, 8192, "same", torch.bfloat16, False),
    (33, 128, 8192, "skewed", torch.float32, False),
    (128, 3000, 384, "uniform", torch.float16, True),
    (129, 128, 640, "same", torch.float32, True),
])
def test_gradient_few_rows(M, V, H, kind, dtype, masked, add):
    """Up to 128 rows (fewer when wide) one launch sums them, above them sorted rows."""
    _check_grad(M, V, H, kind, dtype, add, masked)
