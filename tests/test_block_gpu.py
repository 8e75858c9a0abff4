"""The block between norm and head as it is used: its autograd forms, a training step
of examples/draft_block.py against 64 bits, its 8-bit form on verify windows, and
calls that share a GPU."""
import os
import sys
import threading

import pytest
import torch

from ops_ref import distill64, gen, table64
from verify_vocab_blocked_gb300 import build as qbuild
from verify_vocab_blocked_gb300 import qhead
from verify_vocab_blocked_gb300.autograd import add_norm, linear

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qbuild.build()
    qhead.lib()


@pytest.mark.parametrize("act", ["none", "silu"])
def test_linear_is_the_library_call(act):
    g = gen(1)
    x = torch.randn(70, 96, device="cuda", generator=g).to(BF).requires_grad_(True)
    w = torch.randn(64, 96, device="cuda", generator=g).to(BF).requires_grad_(True)
    b = torch.randn(64, device="cuda", generator=g).requires_grad_(True)
    r = torch.randn(70, 64, device="cuda", generator=g).requires_grad_(True)
    y = linear(x, w, b, act, r, out_dtype=F)
    dy = torch.randn(70, 64, device="cuda", generator=g)
    y.backward(dy)
    xd, wd, bd, rd = (v.detach() for v in (x, w, b, r))
    ref, pre = qhead.linear(xd, wd, bd, act, rd, out_dtype=F, want_pre=True)
    dx, dw, db = qhead.linear_bwd(xd, wd, dy, pre, act)
    assert torch.equal(y.detach(), ref) and torch.equal(x.grad, dx) and torch.equal(w.grad, dw)
    assert torch.equal(b.grad, db.float()) and torch.equal(r.grad, dy)
    x.grad = None
    linear(x, wd, bd, act, rd, out_dtype=F).sum().backward()      # an expanded gradient
    assert torch.equal(x.grad, qhead.linear_bwd(xd, wd, torch.ones_like(dy), pre, act)[0])


@pytest.mark.parametrize("center", [True, False])
def test_add_norm_is_the_library_call(center):
    g = gen(2)
    x = torch.randn(33, 320, device="cuda", generator=g).to(BF).requires_grad_(True)
    r = torch.randn(33, 320, device="cuda", generator=g).requires_grad_(True)
    w = torch.randn(320, device="cuda", generator=g).requires_grad_(True)
    b = torch.randn(320, device="cuda", generator=g).requires_grad_(True)
    y, total = add_norm(x, r, w, b, 1e-5, center=center)
    dy, dt = torch.randn(33, 320, device="cuda", generator=g).to(BF), torch.randn(33, 320, device="cuda", generator=g)
    torch.autograd.backward((y, total), (dy, dt))
    ref, t, mean, rstd = qhead.add_norm(x.detach(), r.detach(), w.detach(), b.detach(), 1e-5, center=center)
    dx, dw, db = qhead.add_norm_bwd(t, w.detach(), mean, rstd, dy, dt)
    assert torch.equal(y.detach(), ref) and torch.equal(total.detach(), t)
    assert torch.equal(r.grad, dx) and torch.equal(x.grad, dx.to(BF)) and torch.equal(w.grad, dw) and torch.equal(b.grad, db)


def reference_step(block, x, h, head, ids, teacher):
    W = table64(head.wq, head.scales, head.biases, head.bits)
    leaves = [p.detach().double().requires_grad_(True) for p in block.parameters()]
    up, up_bias, down, gain = leaves
    t = x.double() + h.double()
    y = t * (t.square().mean(1, keepdim=True) + 1e-6).rsqrt() * gain
    out = t + torch.nn.functional.silu(y @ up.t() + up_bias) @ down.t()
    loss = distill64(W, out, ids, teacher, 1.0, head.softcap)[0].mean()
    loss.backward()
    return out.detach(), loss.detach(), [p.grad for p in leaves]


@pytest.mark.parametrize("rows,hidden", [(300, 256), (9, 512)])
def test_a_training_step(rows, hidden):
    """add_norm -> linear(silu) -> linear(residual) -> distillation and back, clipped.  Each
    stage rounds to bf16 once in each direction (forward: norm, inner product, its
    output; backward: dh, dz of both products, two dx and the norm's), a dozen roundings
    of 2^-9 relative in the worst case along a path: the gradients agree to 3e-2 of
    their norms."""
    from draft_block import Block, make_data, train_step
    block = Block(hidden, 4 * hidden + 8, seed=3)
    head, x, h, ids, teacher = make_data(rows, 2048, hidden, 8, seed=4)
    out, ref_loss, grads = reference_step(block, x, h, head, ids, teacher)
    got = block(x, h)
    assert ((got.double() - out).norm() / out.norm()).item() <= 1e-2
    loss, norm = train_step(block, head, x, h, ids, teacher, max_norm=1e9)
    assert abs(loss.item() - ref_loss.item()) <= 2e-2 * abs(ref_loss.item())
    for p, want in zip(block.parameters(), grads):
        assert ((p.grad.double() - want).norm() / want.norm()).item() <= 3e-2
    whole = torch.cat([p.grad.double().flatten() for p in block.parameters()]).norm()
    assert abs(norm.double() - whole) <= 1e-5 * whole
    # clipped to half of it
    keep = [p.grad.clone() for p in block.parameters()]
    again = qhead.clip_grads([p.grad for p in block.parameters()], 0.5 * whole.item())
    assert torch.equal(again, norm)
    for p, k in zip(block.parameters(), keep):
        assert ((p.grad.float() - 0.5 * k.float()).abs() <= 2.0 ** -7 * k.float().abs() + 1e-30).all()


def test_the_8_bit_block_on_verify_windows():
    """Three roundings to e4m3 on the way (2^-4 relative at most, 2^-5.8 rms each, of
    operands and weights): the block's own part of the hidden state, off by a tenth at
    most; the call alone and among the 5 rows of each window gives the same rows."""
    from draft_block import Block, make_data
    block = Block(512, 2048, seed=5)
    head, x, h, _, _ = make_data(20, 4096, 512, 8, seed=6)
    with torch.no_grad():
        block.quantize()
        exact, served = block(x, h), block.serve(x, h)
        total = (x.float() + h.float())
        part = (exact.float() - total).norm()
        assert ((served - exact).float().norm() / part).item() <= 0.1
        assert torch.equal(block.serve(x[5:10], h[5:10]), served[5:10])
        draft = qhead.fwd(head, served, want_lse=False)[2].view(4, 5)[:, :4].contiguous()
        n, _, am, _ = qhead.verify(head, served, 5, draft)
        assert (n == 4).all() and torch.equal(am.view(4, 5)[:, :4], draft)


def _work(seed, stream):
    g = gen(seed)
    x = torch.randn(300, 200, device="cuda", generator=g).to(BF)
    w = torch.randn(264, 200, device="cuda", generator=g).to(BF)
    r = torch.randn(300, 264, device="cuda", generator=g)
    gain = torch.ones(264, device="cuda")
    stream.wait_stream(torch.cuda.current_stream())
    kw = dict(stream=stream)
    y, pre = qhead.linear(x, w, None, "gelu", r, want_pre=True, **kw)
    few = qhead.linear(x[:6], w, None, "gelu", r[:6], **kw)
    n, total, mean, rstd = qhead.add_norm(y, r, gain, **kw)
    dx, dw, _ = qhead.add_norm_bwd(total, gain, mean, rstd, n, total, **kw)
    codes, scale, _ = qhead.norm_8bit(y, gain, residual=r, **kw)
    grads = qhead.linear_bwd(x, w, dx, pre, "gelu", **kw)
    out = [torch.empty_like(t) for t in grads]
    stream.wait_stream(torch.cuda.current_stream())
    norm = qhead.clip_grads(list(grads), 1e-3, out=out, **kw)
    return [y, few, n, total, dx, dw, codes.view(torch.uint8), scale, *grads, *out, norm]


def test_two_threads_on_two_streams():
    alone = [_work(k, torch.cuda.Stream()) for k in range(2)]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def run(k):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                got[k] = _work(k, s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not errors
    for a, b in zip(alone, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_a_step_captured_and_replayed():
    """The whole block's calls in one graph, on changed inputs."""
    g = gen(9)
    x = torch.randn(140, 256, device="cuda", generator=g).to(BF)
    r = torch.randn(140, 256, device="cuda", generator=g).to(BF)
    w = (torch.randn(256, 256, device="cuda", generator=g) / 16).to(BF)
    gain = torch.ones(256, device="cuda").to(BF)

    def step():
        y, total, mean, rstd = qhead.add_norm(x, r, gain, center=False)
        z, pre = qhead.linear(y, w, None, "silu", total, want_pre=True)
        dx, dw, db = qhead.linear_bwd(y, w, z, pre, "silu")
        dh, dg, _ = qhead.add_norm_bwd(total, gain, mean, rstd, dx, z, want_dbias=False)
        norm = qhead.clip_grads([dw, dg, db], 0.1)
        return [y, z, dh, dw, dg, db, norm]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for k in range(3):
        x.copy_(torch.randn(140, 256, device="cuda", generator=g))
        graph.replay()
        ref = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, ref))


def test_the_examples_run(capsys):
    import draft_block
    import tied_distill
    for module, argv in ((draft_block, ["--rows", "100", "--vocab", "4096", "--hidden", "256", "--steps", "2"]),
                         (tied_distill, ["--rows", "100", "--vocab", "4096", "--hidden", "256", "--steps", "2"])):
        old, sys.argv = sys.argv, ["example", *argv]
        try:
            module.main()
        finally:
            sys.argv = old
    said = capsys.readouterr().out
    assert "nan" not in said and said.count("gradient norm") == 4
