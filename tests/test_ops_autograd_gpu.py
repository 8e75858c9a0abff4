"""The differentiable forms of the operators beside the head: each backward is
the library's own call on the incoming gradient, and the example that runs
them together has the gradients of the plain 64-bit composition."""
import os
import sys

import pytest
import torch

from ops_ref import distill64, gen, make_table, norm64, table64
from verify_vocab_blocked_gb300 import build as qbuild
from verify_vocab_blocked_gb300 import qhead
from verify_vocab_blocked_gb300.autograd import embed, head_distill, layer_norm

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qhead.lib()


def test_distill_is_the_library_call():
    head = qhead.Head(*make_table(500, 256, 4, 1), 4, softcap=30.0)
    g = gen(2)
    h = torch.randn(70, 256, device="cuda", generator=g).to(torch.bfloat16).requires_grad_(True)
    ids = torch.randint(0, 500, (70, 6), device="cuda", generator=g).int()
    t = torch.randn(70, 6, device="cuda", generator=g)
    w = torch.rand(70, device="cuda", generator=g)
    mask = torch.rand(70, device="cuda", generator=g) < 0.8
    loss = head_distill(h, head, ids, t, 2.0, mask)
    (loss * w).sum().backward()
    ref, lse, kept = qhead.distill_fwd(head, h.detach(), ids, t, 2.0, mask)
    assert torch.equal(loss.detach(), ref)
    assert torch.equal(h.grad, qhead.distill_bwd(head, h.detach(), ids, t, kept, lse, w, 2.0, mask))
    h.grad = None
    head_distill(h, head, ids, t, 2.0, mask).sum().backward()     # an expanded cotangent
    assert torch.equal(h.grad, qhead.distill_bwd(head, h.detach(), ids, t, kept, lse,
                                                 torch.ones_like(w), 2.0, mask))


@pytest.mark.parametrize("center,bias", [(True, True), (True, False), (False, False), (False, True)])
def test_layer_norm_is_the_library_call(center, bias):
    g = gen(3)
    x = torch.randn(33, 320, device="cuda", generator=g).requires_grad_(True)
    w = torch.randn(320, device="cuda", generator=g).requires_grad_(True)
    b = torch.randn(320, device="cuda", generator=g).requires_grad_(True) if bias else None
    y = layer_norm(x, w, b, 1e-5, center=center, out_dtype=torch.float32)
    dy = torch.randn(33, 320, device="cuda", generator=g)
    y.backward(dy)
    ref, mean, rstd = qhead.layer_norm(x.detach(), w.detach(), b.detach() if bias else None, 1e-5,
                                       center=center, out_dtype=torch.float32)
    dx, dw, db = qhead.layer_norm_bwd(x.detach(), w.detach(), mean, rstd, dy)
    assert torch.equal(y.detach(), ref) and torch.equal(x.grad, dx) and torch.equal(w.grad, dw)
    assert b is None or torch.equal(b.grad, db)
    x.grad = None
    layer_norm(x, w, b, 1e-5, center=center, out_dtype=torch.float32).sum().backward()
    assert torch.equal(x.grad, qhead.layer_norm_bwd(x.detach(), w.detach(), mean, rstd,
                                                    torch.ones_like(dy))[0])


def test_embed_adds_into_dw():
    head = qhead.Head(*make_table(90, 256, 8, 4), 8)
    t = torch.randint(0, 90, (50,), device="cuda", generator=gen(5)).int()
    dw = torch.ones(90, 256, device="cuda")
    y = embed(head, t, 3.0, dw=dw, out_dtype=torch.float32)
    assert torch.equal(y.detach(), qhead.embed(head, t, 3.0, out_dtype=torch.float32))
    dy = torch.randn(50, 256, device="cuda", generator=gen(6))
    (y * dy).sum().backward()
    want = qhead.embed_bwd(head, t, dy, 3.0, dw=torch.ones(90, 256, device="cuda"))
    assert torch.equal(dw, want)
    assert not embed(head, t, 3.0).requires_grad


def test_example_step_against_64_bits():
    """embed -> body -> layer_norm -> head_distill and back.  Each stage is
    rounded to bf16 once per direction (the forward's x, x + x B, h; the
    backward's dh, the norm's dx and the body's dx): a handful of roundings of
    2^-9 rms relative each way, so gradients agree to 3e-2 of their norms."""
    from tied_distill import Step
    s = Step(300, 1024, 256, 8, seed=7)
    loss = s()
    W = table64(s.head.wq, s.head.scales, s.head.biases, 4).requires_grad_(False)
    emb = W.clone().requires_grad_(True)
    body = s.body.detach().double().requires_grad_(True)
    gain = s.gain.detach().double().requires_grad_(True)
    shift = s.shift.detach().double().requires_grad_(True)
    x = emb[s.tokens.long()] * s.scale * s.mask[:, None]
    x2 = x + x @ body
    xc = x2 - x2.mean(1, keepdim=True)
    h = xc * (xc.square().mean(1, keepdim=True) + 1e-6).rsqrt() * gain + shift
    L, _, _, _ = distill64(W, h, s.ids, s.teacher, 1.0, 30.0, s.mask)
    ref = L.sum() / s.mask.sum()
    ref.backward()
    assert abs(loss.item() - ref.item()) <= 1e-2 * abs(ref.item())
    for got, want in ((s.dw, emb.grad), (s.body.grad, body.grad), (s.gain.grad, gain.grad),
                      (s.shift.grad, shift.grad)):
        assert ((got.double() - want).norm() / want.norm()).item() <= 3e-2


def test_stream_argument():
    """Every call on a stream given to it: the same results, and its workspaces
    stay its own while other work allocates on the current stream."""
    head = qhead.Head(*make_table(3000, 512, 4, 8), 4)
    g = gen(9)
    M = 300
    tok = torch.randint(0, 3000, (M,), device="cuda", generator=g).int()
    h = torch.randn(M, 512, device="cuda", generator=g).to(torch.bfloat16)
    w = torch.ones(512, device="cuda")
    ids = torch.randint(0, 3000, (M, 9), device="cuda", generator=g).int()
    t = torch.randn(M, 9, device="cuda", generator=g)
    dl = torch.rand(M, device="cuda", generator=g)

    def every(stream):
        y, mean, rstd = qhead.layer_norm(h, w, out_dtype=torch.float32, stream=stream)
        dx, dw, db = qhead.layer_norm_bwd(h, w, mean, rstd, y, stream=stream)
        e = qhead.embed(head, tok, 2.0, stream=stream)
        de = qhead.embed_bwd(head, tok, y, stream=stream)
        loss, lse, kept = qhead.distill_fwd(head, h, ids, t, stream=stream)
        dh = qhead.distill_bwd(head, h, ids, t, kept, lse, dl, stream=stream)
        return y, mean, rstd, dx, dw, db, e, de, loss, lse, dh

    ref = every(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = every(s)
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(30)]
    torch.cuda.synchronize()
    del junk
    assert all(torch.equal(p, q) for p, q in zip(ref, got))
