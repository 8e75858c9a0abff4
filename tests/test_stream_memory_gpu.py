"""Calls on a given stream beside work of the current one: neither side's blocks are
handed to the other while its kernels are still queued."""
import pytest
import torch

from ops_ref import gen, make_table
from verify_vocab_blocked_gb300 import build as qbuild
from verify_vocab_blocked_gb300 import qhead

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qhead.lib()


def _busy(x):
    """Some tens of milliseconds of products on the current stream."""
    for _ in range(40):
        x = (x @ x).clamp_(-1, 1)
    return x


def test_blocks_freed_on_either_stream():
    M, V, H, K = 300, 30000, 512, 9
    head = qhead.Head(*make_table(V, H, 4, 8), 4)
    g = gen(9)
    h = torch.randn(M, H, device="cuda", generator=g).to(torch.bfloat16)
    ids = torch.randint(0, V, (M, K), device="cuda", generator=g).int()
    t = torch.randn(M, K, device="cuda", generator=g)
    dl = torch.rand(M, device="cuda", generator=g)
    w = torch.ones(H, device="cuda")
    slow = torch.randn(4096, 4096, device="cuda", generator=g)
    loss0, lse0, kept = qhead.distill_fwd(head, h, ids, t)
    dh0 = qhead.distill_bwd(head, h, ids, t, kept, lse0, dl)
    y0 = qhead.layer_norm(h, w)[0]
    cols = kept.shape[1]
    del kept
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of the outputs' sizes, freed while the current stream has yet to read them
    old = [torch.full(shape, 3.0, device="cuda") for shape in ((M, cols), (M,), (M,), (M, H))]
    torch.cuda.synchronize()
    _busy(slow)
    seen = [x.clone() for x in old]
    del old
    loss, lse, kept = qhead.distill_fwd(head, h, ids, t, stream=s)
    y = qhead.layer_norm(h, w, stream=s)[0]       # (mean and rstd dropped at once)
    with torch.cuda.stream(s):
        _busy(slow)
    dh = qhead.distill_bwd(head, h, ids, t, kept, lse, dl, stream=s)
    del kept, lse
    junk = [torch.full((M, cols), float("nan"), device="cuda") for _ in range(4)]
    junk += [torch.full((n,), float("nan"), device="cuda") for n in (M, M, M * H, M * H) * 8]
    torch.cuda.synchronize()
    assert all((x == 3.0).all() for x in seen)
    assert torch.equal(loss, loss0) and torch.equal(dh, dh0) and torch.equal(y, y0)
    del junk
