"""Whose memory a call on a given stream uses: its workspace and outputs come from
that stream's pool, the outputs are recorded on the current stream and the inputs
on the given one, in every entry point of the binding.  The library and the
streams are stand-ins, so nothing reaches a GPU."""
import contextlib

import pytest
import torch

from verify_vocab_blocked_gb300 import qhead

M, H, V, K = 6, 256, 1000, 5


class Given:
    cuda_stream = 7


class Library:
    """Every size is 0 and every call succeeds; what the calls were given is kept."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            if not name.endswith(("workspace", "kept")):
                self.calls.append((name, args))
            return 0
        return fn


@pytest.fixture
def world(monkeypatch):
    """(stream given, current stream, library, stream -> its recorded tensors, tensors
    allocated with the stream that was current)."""
    given, current, lib = Given(), object(), Library()
    entered, recorded, made = [], {}, []
    plain_empty = torch.empty

    @contextlib.contextmanager
    def use(stream):
        entered.append(stream)
        yield
        entered.pop()

    def empty(*a, **kw):
        t = plain_empty(*a, **kw)
        made.append((t.data_ptr(), t, entered[-1] if entered else None))
        return t

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: recorded.setdefault(id(s), []).append(t), raising=False)
    monkeypatch.setattr(qhead, "lib", lambda: lib)
    monkeypatch.setattr(qhead, "_distill_sizes", {})
    monkeypatch.setattr(qhead, "_usable", lambda *a: None, raising=False)
    return given, current, lib, recorded, made


def _inputs():
    head = qhead.Head(torch.zeros(V, H // 8, dtype=torch.int32), torch.zeros(V, H // 64).half(),
                      torch.zeros(V, H // 64).half(), 4)
    f = lambda *s: torch.zeros(*s)                                    # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)                 # noqa: E731
    return dict(head=head, h=f(M, H).bfloat16(), t=i(M), lse=f(M), g=f(M), mask=torch.ones(M, dtype=torch.bool),
                bm=f(M, 4), draft=i(1, M - 1), dout=f(M, H), w=f(H), ids=i(M, K), tl=f(M, K),
                kept=f(M, 0), dw=f(V, H))


CALLS = {
    "fwd": lambda a, **s: qhead.fwd(a["head"], a["h"], a["t"], a["mask"], **s),
    "bwd": lambda a, **s: qhead.bwd(a["head"], a["h"], a["t"], a["lse"], a["g"], a["mask"], **s),
    "bwd_dw": lambda a, **s: qhead.bwd_dw(a["head"], a["h"], a["t"], a["lse"], a["g"], a["mask"],
                                          want_dh=True, **s),
    "fwd_blockmax": lambda a, **s: qhead.fwd_blockmax(a["head"], a["h"], a["t"], a["mask"], **s),
    "bwd_blockskip": lambda a, **s: qhead.bwd_blockskip(a["head"], a["h"], a["t"], a["lse"], a["g"],
                                                        a["bm"], 1e-5, a["mask"], **s),
    "bwd_filter": lambda a, **s: qhead.bwd_filter(a["head"], a["h"], a["t"], a["lse"], a["g"], 1e-5,
                                                  a["mask"], want_cold=True, **s),
    "verify": lambda a, **s: qhead.verify(a["head"], a["h"], M, a["draft"], a["mask"], want_lse=True, **s),
    "embed": lambda a, **s: qhead.embed(a["head"], a["t"], 2.0, a["mask"], **s),
    "embed_bwd": lambda a, **s: qhead.embed_bwd(a["head"], a["t"], a["dout"], 2.0, a["mask"], **s),
    "embed_bwd_added": lambda a, **s: qhead.embed_bwd(a["head"], a["t"], a["dout"], dw=a["dw"], **s),
    "layer_norm": lambda a, **s: qhead.layer_norm(a["h"], a["w"], a["w"], **s),
    "layer_norm_bwd": lambda a, **s: qhead.layer_norm_bwd(a["h"], a["w"], a["lse"], a["g"], a["dout"], **s),
    "distill_fwd": lambda a, **s: qhead.distill_fwd(a["head"], a["h"], a["ids"], a["tl"], 1.0, a["mask"], **s),
    "distill_bwd": lambda a, **s: qhead.distill_bwd(a["head"], a["h"], a["ids"], a["tl"], a["kept"], a["lse"],
                                                    a["g"], 1.0, a["mask"], **s),
}


def _same(t, tensors):
    return any(t.data_ptr() == x.data_ptr() and t.numel() == x.numel() for x in tensors)


@pytest.mark.parametrize("name", CALLS)
def test_call_on_a_given_stream(world, name):
    given, current, lib, recorded, made = world
    a = _inputs()
    made.clear()
    got = CALLS[name](a, stream=given)
    assert len(lib.calls) == 1 and lib.calls[0][1][-1] == given.cuda_stream
    assert made and all(s is given for _, _, s in made)
    outs = [t for t in (got if isinstance(got, tuple) else (got,)) if t is not None]
    mine = {p for p, _, _ in made}
    on_current, on_given = recorded.get(id(current), []), recorded.get(id(given), [])
    for t in outs:
        if t is a["dw"]:
            assert _same(t, on_given)
        else:
            assert t.data_ptr() in mine and _same(t, on_current)
    # every input that the call was given a pointer of
    pointers = {x for x in lib.calls[0][1] if isinstance(x, int)}
    for k, t in a.items():
        if k != "head" and t.numel() and t.data_ptr() in pointers:
            assert _same(t, on_given), k
    if name.startswith(("layer_norm", "embed_bwd")):
        return
    assert all(_same(t, on_given) for t in (a["head"].wq, a["head"].scales, a["head"].biases))


@pytest.mark.parametrize("name", CALLS)
def test_call_on_the_current_stream(world, monkeypatch, name):
    _, _, lib, recorded, made = world
    monkeypatch.setattr(qhead, "_stream", lambda stream, *a: 3)
    a = _inputs()
    made.clear()
    CALLS[name](a)
    assert not recorded and all(s is None for _, _, s in made)
    assert lib.calls[0][1][-1] == 3


def test_a_workspace_given_to_the_call_is_recorded(world):
    given, _, _, recorded, _ = world
    a = _inputs()
    ws = torch.zeros(512, dtype=torch.uint8)
    qhead.distill_fwd(a["head"], a["h"], a["ids"], a["tl"], workspace=ws, stream=given)
    qhead.fwd(a["head"], a["h"], a["t"], workspace=ws, stream=given)
    assert sum(x.data_ptr() == ws.data_ptr() for x in recorded[id(given)]) == 2
