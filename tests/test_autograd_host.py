"""The autograd forms' own rules, with the library's calls replaced by constants:
a backward is not differentiated silently, a mask changed in place between the
directions is noticed, and nothing reaches a GPU."""
import pytest
import torch

from verify_vocab_blocked_gb300 import autograd, qhead

M, H, K = 4, 8, 3


@pytest.fixture(autouse=True)
def constants(monkeypatch):
    """Calls of the library's shapes whose results, like the library's, carry no graph."""
    def const(*shape, dtype=torch.float32):
        return torch.full(shape, 0.5, dtype=dtype)

    monkeypatch.setattr(qhead, "fwd", lambda *a, **k: (const(M), const(M), None))
    monkeypatch.setattr(qhead, "bwd", lambda *a, **k: const(M, H))
    monkeypatch.setattr(qhead, "distill_fwd", lambda *a, **k: (const(M), const(M), const(M, K)))
    monkeypatch.setattr(qhead, "distill_bwd", lambda *a, **k: const(M, H, dtype=torch.bfloat16))
    monkeypatch.setattr(qhead, "layer_norm", lambda *a, **k: (const(M, H), const(M), const(M)))
    monkeypatch.setattr(qhead, "layer_norm_bwd", lambda *a, **k: (const(M, H), const(H), const(H)))
    monkeypatch.setattr(qhead, "embed", lambda *a, **k: const(M, H))
    monkeypatch.setattr(qhead, "embed_bwd", lambda head, t, dout, *a, dw=None, **k: dw.add_(1.0))


def _bf(*shape):
    return torch.ones(*shape, dtype=torch.bfloat16, requires_grad=True)


def _logp():
    h = _bf(M, H)
    return autograd.head_logp(h, None, torch.zeros(M, dtype=torch.int32)), (h,)


def _distill():
    h = _bf(M, H)
    return autograd.head_distill(h, None, torch.zeros(M, K, dtype=torch.int32), torch.zeros(M, K)), (h,)


def _norm():
    x, w, b = (torch.ones(s, requires_grad=True) for s in ((M, H), (H,), (H,)))
    return autograd.layer_norm(x, w, b), (x, w, b)


@pytest.mark.parametrize("form", [_logp, _distill, _norm])
def test_a_gradient_penalty_is_refused(form):
    out, leaves = form()
    grads = torch.autograd.grad(out.float().square().sum(), leaves, create_graph=True)
    penalty = sum(g.float().square().sum() for g in grads)
    with pytest.raises(RuntimeError):
        (out.float().sum() + penalty).backward()


@pytest.mark.parametrize("form", [_logp, _distill, _norm])
def test_first_derivatives(form):
    out, leaves = form()
    out.float().sum().backward()
    assert all((x.grad == 0.5).all() for x in leaves)


def test_embed_gradient_goes_into_dw():
    dw = torch.zeros(5, H)
    y = autograd.embed(None, torch.zeros(M, dtype=torch.int32), dw=dw)
    y.sum().backward()
    assert (dw == 1.0).all()


def _masked(name, mask):
    t = torch.zeros(M, dtype=torch.int32)
    if name == "embed":
        return autograd.embed(None, t, 1.0, mask, dw=torch.zeros(5, H))
    if name == "logp":
        return autograd.head_logp(_bf(M, H), None, t, mask)
    return autograd.head_distill(_bf(M, H), None, torch.zeros(M, K, dtype=torch.int32), torch.zeros(M, K), 1.0,
                                 mask)


@pytest.mark.parametrize("name", ["logp", "distill", "embed"])
@pytest.mark.parametrize("dtype", [torch.bool, torch.uint8])
def test_a_mask_changed_between_the_directions(name, dtype):
    mask = torch.ones(M, dtype=dtype)
    _masked(name, mask).sum().backward()
    out = _masked(name, mask)
    mask[1] = 0
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
