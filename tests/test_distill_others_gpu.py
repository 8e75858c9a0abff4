"""Distillation where the student's mass lies on a few tokens that the teacher does not
list, wherever they lie: next to one another, in one block of 32 or 256 vocab rows, in
the last rows.  Those of a thousandth of the sum or more, up to 16, enter with exact
logits, so lse and the loss are off by the exact logits' fp32 steps, the kernel's error
only on what is left.

Tolerances.  An exact logit: H / 256 units (rounded up) of 4 products a lane, the
weight's rounding, 5 shuffles and the sums around them, n = 4 ceil(H / 256) + 8 half
steps of sum |h w|.  One of the kernel: 2^-11 of it besides (see test_distill_gpu).
lse: their mean under q over T, and 16 half steps of values that large; the loss: lse's,
the listed logits' under p, and as many steps again."""
import pytest
import torch

from ops_ref import U, distill64, gen, make_table, table64
from verify_vocab_blocked_gb300 import build as qbuild
from verify_vocab_blocked_gb300 import qhead

pytestmark = pytest.mark.gpu

F, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qhead.lib()


def _columns(kind, M, V, g):
    """The tokens with the mass, [M, n]."""
    at = torch.randint(0, V // 256, (M, 1), device="cuda", generator=g) * 256
    if kind == "adjacent":
        return at + 32 * 3 + 7 + torch.arange(2, device="cuda")
    if kind == "slice":          # five of one block of 32
        return at + 32 * 2 + torch.tensor([0, 3, 4, 17, 31], device="cuda")
    if kind == "tile":           # seven of one block of 256, in four of 32
        return at + torch.tensor([1, 2, 40, 41, 100, 230, 255], device="cuda")
    if kind == "last":           # the vocabulary's last rows
        return (V - 1 - torch.arange(3, device="cuda")).expand(M, 3)
    return torch.randint(0, V, (M, 4), device="cuda", generator=g)   # anywhere


def _case(kind, M, V, H, bits, K, cap, seed, sb=torch.float16, beside=False):
    head = qhead.Head(*make_table(V, H, bits, seed, sb), bits, softcap=cap)
    W = table64(head.wq, head.scales, head.biases, bits)
    g = gen(seed + 1)
    far = _columns(kind, M, V, g)
    rows = W[far]
    peak = 26.0 if cap <= 0 else 34.0
    h = 0.02 * torch.randn(M, H, device="cuda", generator=g, dtype=torch.float64) \
        + torch.einsum("mk,mkh->mh", peak / rows.square().sum(2), rows)
    ids = torch.randint(0, V, (M, K), device="cuda", generator=g)
    if beside:                   # the teacher lists one of them, and a neighbour of each
        ids[:, 0] = far[:, 0]
        ids[:, 1] = (far[:, -1] + 1) % V
    else:                        # and nothing among them
        ids = torch.where((ids[:, :, None] == far[:, None]).any(2), (ids + 300) % V, ids)
    t = 2 * torch.randn(M, K, device="cuda", generator=g)
    return head, W, h.to(BF), ids.int(), t


def _check(head, W, h, ids, t, T, rows=None):
    """`rows`: which rows are compared (all: None)."""
    M, K = ids.shape
    H, cap = head.H, head.softcap
    dl = torch.rand(M, device="cuda", generator=gen(99)) + 0.5
    loss, lse, kept = qhead.distill_fwd(head, h, ids, t, T)
    dh = qhead.distill_bwd(head, h, ids, t, kept, lse, dl, T)
    again = qhead.distill_fwd(head, h, ids, t, T)
    assert torch.equal(loss, again[0]) and torch.equal(lse, again[1])
    if rows is not None:
        h, ids, t, loss, lse, dh, dl = (x[rows] for x in (h, ids, t, loss, lse, dh, dl))
    hd = h.double().requires_grad_(True)
    L, E, z, p = distill64(W, hd, ids, t, T, cap)
    ref, = torch.autograd.grad((L * dl.double()).sum(), hd)
    with torch.no_grad():
        L, E, z = L.detach(), E.detach(), z.detach()
        mag = h.double().abs() @ W.abs().t()
        q = (z / T - E[:, None]).exp()
        at = ids.long()
        exact = torch.zeros_like(q).scatter_(1, at, 1.0) > 0
        big = (q >= 1.1e-3) & ~exact
        assert big.any()
        # (a row with more than 16 of them, mass spread wide: only the clearly largest count)
        wide = big.sum(1) > 16
        first = torch.zeros_like(big).scatter_(1, (q * big).topk(12, dim=1).indices, True)
        big &= first | ~wide[:, None]
        n = 4 * ((H + 255) // 256) + 8
        d = torch.where(exact | big, n * U, 2.0 ** -11 + H * 2 * U) * mag
        top = 1 + z.abs().amax(1) / T
        e_lse = (q * d).sum(1) / T + 16 * U * top
        e_loss = e_lse + (p * (n * U * mag).gather(1, at)).sum(1) / T + 64 * U * top
        assert ((lse.double() - E).abs() <= e_lse).all(), ((lse.double() - E).abs() / e_lse).max().item()
        assert ((loss.double() - L).abs() <= e_loss).all(), ((loss.double() - L).abs() / e_loss).max().item()
        assert ((dh.double() - ref).norm(dim=1) <= 4e-3 * ref.norm(dim=1)).all()


KINDS = ["adjacent", "slice", "tile", "last", "anywhere"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,bits,cap,T", [(6, 4, 0.0, 1.0), (60, 4, 0.0, 1.0), (200, 8, 50.0, 1.0), (700, 4, 0.0, 2.0)])
def test_wherever_they_lie(kind, M, bits, cap, T):
    _check(*_case(kind, M, 4001, 256, bits, 8, cap, 300 + M), T)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [6, 13, 150])
def test_beside_listed_tokens(kind, M):
    _check(*_case(kind, M, 2050, 384, 8, 8, 0.0, 400 + M, beside=True), 1.0)


@pytest.mark.parametrize("sb", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [6, 14, 90])
def test_scales_that_fp16_rounds(M, sb):
    """The kernels' scales and biases are rounded to fp16, so few rows are no exception."""
    _check(*_case("tile", M, 4001, 256, 4, 8, 0.0, 500 + M, sb), 1.0)


@pytest.mark.parametrize("kind,bits", [("adjacent", 4), ("tile", 8), ("last", 4)])
def test_logits_not_kept(kind, bits):
    """Past 4 GiB of logits the slices' columns are formed again."""
    head, W, h, ids, t = _case(kind, 4500, 262144, 128, bits, 5, 0.0, 600, beside=bits == 8)
    rows = torch.arange(0, 4500, 45, device="cuda")
    _check(head, W, h, ids, t, 1.0, rows)


def test_more_than_sixteen():
    """Of 40 in two blocks of 32 the sixteen largest: the loss is no further off than
    the rest's share of the kernel's error."""
    M, V, H = 50, 3000, 512
    head = qhead.Head(*make_table(V, H, 4, 700), 4)
    W = table64(head.wq, head.scales, head.biases, 4)
    far = 512 + torch.arange(40, device="cuda")
    rows = W[far]
    peak = 20.0 + torch.linspace(0, 6, 40, device="cuda", dtype=torch.float64)
    sol = torch.linalg.solve(rows @ rows.t(), peak)
    h = (rows.t() @ sol).expand(M, H) + 0.01 * torch.randn(M, H, device="cuda", generator=gen(701), dtype=torch.float64)
    h = h.to(BF)
    ids = torch.randint(0, 400, (M, 6), device="cuda", generator=gen(702)).int()
    t = torch.randn(M, 6, device="cuda", generator=gen(703))
    loss, lse, kept = qhead.distill_fwd(head, h, ids, t)
    L, E, z, _ = distill64(W, h.double(), ids, t, 1.0, 0.0)
    q = (z - E[:, None]).exp()
    top = q.topk(16, dim=1)
    got = kept[:, 6 + 16:6 + 32].contiguous().view(torch.int32).long() - 1
    # those far enough above the seventeenth that the kernel's error cannot swap them
    clear = top.values[:, :14]
    assert (clear[:, -1] > 1.02 * q.topk(17, dim=1).values[:, 16]).any()
    assert all(set(a.tolist()) <= set(b.tolist()) for a, b in zip(top.indices[:, :8], got))
    mag = h.double().abs() @ W.abs().t()
    kernel = torch.ones_like(q, dtype=torch.bool).scatter_(1, got, False)
    d = torch.where(kernel, 2.0 ** -11 + H * 2 * U, (4 * 2 + 8) * U) * mag
    e = (q * d).sum(1) + 80 * U * (1 + z.abs().amax(1))
    assert ((lse.double() - E).abs() <= e).all()
    assert ((loss.double() - L).abs() <= e + 16 * U * mag.gather(1, ids.long()).amax(1)).all()
