"""The product's autograd form keeps its pre-activation only for a backward that can come.
Nothing here reaches a GPU."""
import contextlib

import pytest
import torch

from verify_vocab_blocked_gb300 import autograd, qhead

M, K, N = 6, 64, 32


@pytest.fixture
def kept(monkeypatch):
    asked = []

    def linear(x, w, *a, want_pre=False, **k):
        asked.append(want_pre)
        y = torch.zeros(M, N, dtype=torch.bfloat16)
        return (y, y.half()) if want_pre else y

    monkeypatch.setattr(qhead, "linear", linear)
    return asked


@pytest.mark.parametrize("mode,want", [(contextlib.nullcontext, True), (torch.enable_grad, True), (torch.no_grad, False),
                                       (torch.inference_mode, False)])
@pytest.mark.parametrize("act", ["silu", "none"])
def test_modes(kept, mode, want, act):
    x, w = torch.ones(M, K, dtype=torch.bfloat16), torch.ones(N, K, dtype=torch.bfloat16, requires_grad=True)
    with mode():
        y = autograd.linear(x, w, None, act)
    assert kept == [want and act != "none"] and y.requires_grad == want


def test_without_parameters(kept):
    x, w = torch.ones(M, K, dtype=torch.bfloat16), torch.ones(N, K, dtype=torch.bfloat16)
    r = torch.ones(M, N, requires_grad=True)
    assert autograd.linear(x, w, None, "silu", r).requires_grad and not autograd.linear(x, w, None, "silu").requires_grad
    assert kept == [False, False]


def test_recomputed_under_a_checkpoint(kept, monkeypatch):
    """The pass that the backward of a checkpointed block runs again keeps it."""
    from torch.utils.checkpoint import checkpoint
    monkeypatch.setattr(qhead, "linear_bwd", lambda x, w, *a, **k: (None, torch.ones_like(w), None))
    x, w = torch.ones(M, K, dtype=torch.bfloat16), torch.ones(N, K, dtype=torch.bfloat16, requires_grad=True)
    checkpoint(lambda: autograd.linear(x, w, None, "silu"), use_reentrant=False).float().sum().backward()
    assert kept[-1] and (w.grad == 1).all()


def test_applied_without_a_mode(kept, monkeypatch):
    monkeypatch.setattr(qhead, "linear_bwd", lambda x, w, *a, **k: (None, torch.ones_like(w), None))
    x, w = torch.ones(M, K, dtype=torch.bfloat16), torch.ones(N, K, dtype=torch.bfloat16, requires_grad=True)
    autograd.Linear.apply(x, w, None, "silu", None, None).float().sum().backward()
    assert kept == [True] and (w.grad == 1).all()
