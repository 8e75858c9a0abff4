"""A workspace must hold the bytes that its elements count.  Nothing here reaches a GPU."""
import types

import pytest
import torch

from verify_vocab_blocked_gb300 import qhead


@pytest.mark.parametrize("workspace,good", [
    (torch.empty(64, dtype=torch.uint8), True), (torch.empty(8, 8, dtype=torch.uint8), True),
    (torch.empty(1, dtype=torch.uint8).expand(1 << 30), False), (torch.empty(4, 1, dtype=torch.uint8).expand(4, 99), False),
    (torch.empty(64, dtype=torch.uint8)[::2], False),
])
def test_contiguous(monkeypatch, workspace, good):
    dev = types.SimpleNamespace(type="cuda", index=0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    given = types.SimpleNamespace(device=dev, is_contiguous=workspace.is_contiguous)
    if good:
        qhead._usable(dev, None, given)
    else:
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            qhead._usable(dev, None, given)
