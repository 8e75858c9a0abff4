"""The global gradient norm and clipping against 64 bits.

Tolerances: a thread sums 32 squares in fp32 (32 half steps), the rest is fp64; the
norm is rounded once.  A scaled value carries the coefficient's relative error, its
rounding and the product's, and the rounding to its type."""
import pytest
import torch

from ops_ref import U, gen, half_step, tiny
from verify_vocab_blocked_gb300 import build as qbuild
from verify_vocab_blocked_gb300 import qhead

pytestmark = pytest.mark.gpu
BF, HF, F = torch.bfloat16, torch.float16, torch.float32
REL = 40 * U


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qhead.lib()


def norm64(ts):
    return torch.cat([t.double().reshape(-1) for t in ts] + [torch.zeros(1, device="cuda", dtype=torch.float64)]).norm()


def tensors(sizes, types, seed, scale=1.0):
    g = gen(seed)
    return [(torch.randn(n, device="cuda", generator=g) * scale).to(types[i % len(types)]) for i, n in enumerate(sizes)]


def check_clip(ts, max_norm, out=None):
    keep = [t.clone() for t in ts]
    want = norm64(keep)
    norm = qhead.clip_grads(ts, max_norm, out=out)
    assert norm.dtype == F and norm.dim() == 0 and abs(norm.double() - want) <= REL * want
    coef = min(1.0, max_norm / (float(want) + 1e-6))
    got = ts if out is None else out
    if out is not None:
        assert all(torch.equal(a, b) for a, b in zip(ts, keep))
    if coef == 1.0 and out is None:
        assert all(torch.equal(a, b) for a, b in zip(got, keep))
    for a, b in zip(got, keep):
        ref = b.double() * coef
        assert ((a.double() - ref).abs() <= 1.01 * (half_step(a.dtype) + REL + 4 * U) * ref.abs() + tiny(a.dtype)).all()


LISTS = [
    [1], [0], [7, 0, 9], [8192], [8191, 8193, 1], [100000, 3, 0, 40000, 17], [5] * 48, [3] * 49, [11] * 480,
    [9] * 481, [70] * 1000, [3_000_001, 12],
]


@pytest.mark.parametrize("types", [(F,), (BF,), (HF, F), (F, BF, HF)])
@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{s[0]}")
def test_norm_and_clip(sizes, types):
    ts = tensors(sizes, types, len(sizes))
    want = norm64(ts)
    norm = qhead.grad_norm(ts)
    assert abs(norm.double() - want) <= REL * want
    assert torch.equal(norm, qhead.grad_norm(ts))
    check_clip(ts, 2.0 * float(want) + 1.0)
    for ot in (F, BF):
        check_clip(ts, 0.3 * float(want) + 1e-3, [torch.empty(t.shape, device="cuda", dtype=ot) for t in ts])
    check_clip(ts, 2.0 * float(want) + 1.0, [torch.empty_like(t) for t in ts])
    check_clip(ts, 0.3 * float(want) + 1e-3)


@pytest.mark.parametrize("t,ot", [(F, F), (BF, BF), (F, BF), (BF, F), (HF, HF)])
def test_views_of_one_buffer(t, ot):
    """Starts at every alignment, and outputs whose alignment differs."""
    sizes = [1, 2, 3, 5, 8, 13, 9001, 4, 20000, 1, 7]
    flat = torch.randn(sum(sizes), device="cuda", generator=gen(1)).to(t)
    check_clip(list(flat.clone().split(sizes)), 1.0)
    other = torch.empty(sum(sizes) + 1, device="cuda", dtype=ot)
    check_clip(list(flat.split(sizes)), 1.0, list(other[1:].split(sizes)))
    assert len(list(flat.split(sizes))) == len(sizes)


def test_many_blocks_and_a_large_tensor():
    check_clip(tensors([40_000_003, 1000, 9_000_000], (BF, F), 5, 1e-3), 0.5)


@pytest.mark.parametrize("scale", [1e-25, 1e-19, 3e18, 1e25])
def test_squares_beyond_fp32(scale):
    """Their sum is still a norm that fp32 holds."""
    ts = tensors([20000, 77], (F,), 9, 1.0)
    for t in ts:
        t.mul_(scale)
    ts.append(torch.zeros(50000, device="cuda"))
    want = norm64(ts)
    assert abs(qhead.grad_norm(ts).double() - want) <= REL * want
    if scale > 1:
        check_clip(ts, 1.0)


def test_values_that_are_not_finite():
    ts = tensors([100, 100], (F,), 2)
    ts[1][7] = float("inf")
    keep = [t.clone() for t in ts]
    assert torch.isinf(qhead.clip_grads(ts, 1.0))
    assert (ts[0] == 0).all() and torch.isnan(ts[1][7]) and (ts[1][:7] == 0).all()
    keep[0][3] = float("nan")
    assert torch.isnan(qhead.clip_grads(keep, 1.0)) and torch.isnan(keep[0]).all()
    zero = [torch.zeros(9, device="cuda")]
    assert qhead.clip_grads(zero, 1.0) == 0 and not zero[0].any()


def test_what_may_not_overlap_is_refused():
    t = torch.zeros(100, device="cuda")
    for call in (lambda: qhead.clip_grads([t, t], 1.0), lambda: qhead.clip_grads([t, t[50:]], 1.0),
                 lambda: qhead.clip_grads([t[:50], t[50:]], 1.0, out=[t[50:], t[:50]]),
                 lambda: qhead.clip_grads([t[:50]], 1.0, out=[t[25:75]]),
                 lambda: qhead.clip_grads([t[:50]], 1.0, out=[t.view(torch.bfloat16)[:50]])):
        with pytest.raises(qhead.QheadError):
            call()
    assert qhead.grad_norm([t, t]) == 0                 # read twice: counted twice
    one = torch.ones(50, device="cuda")
    assert abs(qhead.grad_norm([one, one]).item() - 10) < 1e-5
    check_clip([t[:50].add_(1), t[50:].add_(1)], 1.0)


def test_version_counters_and_another_stream():
    ts = tensors([300, 20000], (F, BF), 4)
    before = [t._version for t in ts]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    keep = [t.clone() for t in ts]
    s.wait_stream(torch.cuda.current_stream())
    norm = qhead.clip_grads(ts, 0.5, stream=s)
    s.synchronize()
    assert [t._version for t in ts] != before
    assert torch.equal(norm, qhead.clip_grads(keep, 0.5)) and all(torch.equal(a, b) for a, b in zip(ts, keep))


def test_captured_and_replayed():
    ts = tensors([5000, 13, 90000], (F, BF), 6)
    out = [torch.empty_like(t) for t in ts]
    qhead.clip_grads(ts, 0.5, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = qhead.clip_grads(ts, 0.5, out=out)
    for t in ts:
        t.mul_(3)
    graph.replay()
    torch.cuda.synchronize()
    ref = [torch.empty_like(t) for t in ts]
    assert torch.equal(norm, qhead.clip_grads(ts, 0.5, out=ref)) and all(torch.equal(a, b) for a, b in zip(out, ref))
