"""Tensors of another device than the one whose stream the kernels are launched on
are refused before any allocation or call: host tensors that are otherwise valid,
and (with the current device a stand-in) a second GPU's; so is a head whose parts are
on two devices or do not fit one another."""
import pytest
import torch

from test_stream_memory_host import CALLS, M, _inputs
from verify_vocab_blocked_gb300 import qhead


class Library:
    """Sizes as asked for on a machine without a GPU; any launch is a failure."""

    def __getattr__(self, name):
        def fn(*args):
            if name.endswith(("workspace", "kept")):
                return 0
            raise AssertionError(f"{name} was reached")
        return fn


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    monkeypatch.setattr(qhead, "lib", lambda: Library())
    monkeypatch.setattr(qhead, "_distill_sizes", {})


@pytest.mark.parametrize("name", CALLS)
def test_host_tensors(name):
    with pytest.raises(ValueError, match="must be on a GPU"):
        CALLS[name](_inputs())


class Stream:
    cuda_stream = 7

    def __init__(self, device):
        self.device = torch.device(device)


def test_another_gpu(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    one = torch.device("cuda:1")
    with pytest.raises(ValueError, match="current device is cuda:0"):
        qhead._usable(one, None)
    with pytest.raises(ValueError, match="stream is of cuda:1"):
        qhead._usable(torch.device("cuda:0"), Stream(one))
    with pytest.raises(ValueError, match="workspace is on cpu"):
        qhead._usable(torch.device("cuda:0"), None, torch.zeros(8, dtype=torch.uint8))
    qhead._usable(torch.device("cuda:0"), None)
    qhead._usable(torch.device("cuda:0"), Stream("cuda:0"))


def test_a_head_of_two_devices():
    hd = _inputs()["head"]
    split = qhead.Head(hd.wq, hd.scales.to("meta"), hd.biases, 4)
    with pytest.raises(ValueError, match="one device"):
        split.c()
    with pytest.raises(ValueError, match="one device"):
        qhead.embed(split, torch.zeros(M, dtype=torch.int32))


@pytest.mark.parametrize("rows,groups", [(1000, 3), (999, 4), (1000, 8)])
def test_scales_that_do_not_cover_the_rows(rows, groups):
    """Too few would be read past their end, another grouping in the wrong places."""
    hd = _inputs()["head"]
    part = torch.zeros(rows, groups).half()
    for head in (qhead.Head(hd.wq, part, hd.biases, 4), qhead.Head(hd.wq, hd.scales, part, 4)):
        with pytest.raises(ValueError, match=r"shape \[1000, 4\]"):
            head.c()


def test_stream_handles(monkeypatch):
    """With and without torch's accessor of the bare handle."""
    dev = torch.device("cuda:0")
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: Stream(d))
    monkeypatch.setattr(qhead, "_raw_stream", lambda i: 40 + i)
    assert qhead._stream(None, dev) == 40
    monkeypatch.setattr(qhead, "_raw_stream", None)
    assert qhead._stream(None, dev) == 7
    assert qhead._stream(Stream(dev), dev) == 7
