"""Refusals of the block between norm and head and of the gradient norm, the memory of
their calls on a given stream, and the rules of their autograd forms: nothing here
reaches a GPU."""
import ctypes

import pytest
import torch

from test_device_host import Library as NoLaunch
from test_stream_memory_host import _same, world  # noqa: F401  (a fixture)
from verify_vocab_blocked_gb300 import autograd, qhead
from verify_vocab_blocked_gb300 import build as qbuild

EINVAL, EUNSUP, OK = qhead.QHEAD_EINVAL, qhead.QHEAD_EUNSUPPORTED, qhead.QHEAD_OK
BAD_SIZE = ctypes.c_size_t(-1).value
NAN, INF = float("nan"), float("inf")
F16, BF16, F32, E4M3 = 0, 1, 2, 3
BF, F, E8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return qhead.lib()


def _call(fn, order, base, kw):
    a = {**base, **kw}
    return fn(*[a[k] for k in order])


# ------------------------------------------------------------------- the C ABI

PLACE = ("x", "t", "ldx", "M", "K", "w", "ldw", "N")
place = dict(x=0x1000, t=BF16, ldx=64, M=4, K=64, w=0x2000, ldw=64, N=32)
LIN = (PLACE + ("xs", "ws", "b", "bt", "act", "r", "rt", "ldr", "y", "yt", "pre", "wsp", "n", "stream"),
       dict(place, xs=None, ws=None, b=None, bt=F32, act=2, r=None, rt=F32, ldr=32, y=0x3000, yt=BF16, pre=None,
            wsp=0x8000, n=1 << 30, stream=None))
LBWD = (PLACE + ("dy", "dt", "ldy", "pre", "act", "dx", "dw", "db", "wsp", "n", "stream"),
        dict(place, dy=0x4000, dt=F32, ldy=32, pre=0x5000, act=2, dx=0x6000, dw=0x7000, db=None, wsp=0x8000, n=1 << 30,
             stream=None))
BAD_PLACE = [
    (dict(t=F32), EUNSUP), (dict(t=9), EUNSUP), (dict(t=-1), EUNSUP), (dict(M=-1), EINVAL), (dict(M=2 ** 31), EINVAL),
    (dict(K=0), EINVAL), (dict(N=0), EINVAL), (dict(K=2 ** 24 + 1, ldx=2 ** 25, ldw=2 ** 25), EINVAL),
    (dict(N=2 ** 24 + 1), EINVAL), (dict(ldx=63), EINVAL), (dict(ldw=63), EINVAL), (dict(x=None), EINVAL),
    (dict(w=None), EINVAL), (dict(x=0x1001), EINVAL), (dict(w=0x2001), EINVAL), (dict(ldx=2 ** 60), EINVAL),
    (dict(M=2 ** 30, N=2 ** 24, ldr=2 ** 24, ldy=2 ** 24), EINVAL),
]


@pytest.mark.parametrize("kw,code", BAD_PLACE + [
    (dict(act=-1), EUNSUP), (dict(act=5), EUNSUP), (dict(yt=E4M3), EUNSUP), (dict(b=0x9000, bt=E4M3), EUNSUP),
    (dict(r=0x9000, rt=7), EUNSUP), (dict(r=0x9000, ldr=31), EINVAL), (dict(y=None), EINVAL), (dict(y=0x3001), EINVAL),
    (dict(pre=0x3001), EINVAL), (dict(b=0x9002), EINVAL), (dict(r=0x9002), EINVAL), (dict(xs=0x9000), EINVAL),
    (dict(ws=0x9000), EINVAL), (dict(t=E4M3), EINVAL), (dict(t=E4M3, xs=0x9000), EINVAL),
    (dict(t=E4M3, xs=0x9002, ws=0x9000), EINVAL),
    (dict(x=0x1002, wsp=None), EINVAL), (dict(x=0x1002, wsp=0x8010), EINVAL), (dict(x=0x1002, n=100), EINVAL),
    (dict(ldw=65, n=100), EINVAL),
    (dict(M=0, x=None, y=None, wsp=None, n=0), OK), (dict(M=0, t=E4M3, xs=None, ws=0x9000, x=None), OK),
])
def test_linear(L, kw, code):
    assert _call(L.qhead_linear, *LIN, kw) == code
    assert (L.qhead_last_error().decode() == "") == (code == OK)


@pytest.mark.parametrize("kw,code", BAD_PLACE + [
    (dict(t=E4M3), EUNSUP), (dict(act=5), EUNSUP), (dict(dt=E4M3), EUNSUP), (dict(ldy=31), EINVAL), (dict(dy=None), EINVAL),
    (dict(pre=None), EINVAL), (dict(dy=0x4002), EINVAL), (dict(pre=0x5001), EINVAL), (dict(dx=0x6001), EINVAL),
    (dict(dw=0x7001), EINVAL), (dict(db=0x7001), EINVAL), (dict(wsp=None), EINVAL), (dict(wsp=0x8010), EINVAL),
    (dict(n=100), EINVAL), (dict(M=0, x=None, dy=None, pre=None, dw=None, wsp=None), OK),
])
def test_linear_bwd(L, kw, code):
    assert _call(L.qhead_linear_bwd, *LBWD, kw) == code
    assert (L.qhead_last_error().decode() == "") == (code == OK)


@pytest.mark.parametrize("name", ["qhead_linear_workspace", "qhead_linear_bwd_workspace"])
@pytest.mark.parametrize("kw,code", BAD_PLACE)
def test_linear_sizes(L, name, kw, code):
    fn = getattr(L, name)
    assert fn(*[{**place, **kw}[k] for k in PLACE]) == BAD_SIZE and L.qhead_last_error().decode()
    assert fn(*[{**place, "M": 0, "x": None}[k] for k in PLACE]) == 0
    # a copy of each operand whose rows TMA cannot read, and no more than that
    plain = fn(*[place[k] for k in PLACE])
    padded = fn(*[{**place, "x": 0x1002, "ldw": 65}[k] for k in PLACE])
    assert plain < BAD_SIZE and padded - plain == 2 * 4 * 64 + 2 * 32 * 64


ADDN = (("x", "xt", "ldx", "r", "rt", "ldr", "M", "H", "w", "b", "wt", "eps", "center", "total", "y", "yt", "mean", "rstd",
         "stream"),
        dict(x=0x1000, xt=BF16, ldx=64, r=0x2000, rt=F32, ldr=64, M=4, H=64, w=0x3000, b=None, wt=F32, eps=1e-6, center=1,
             total=0x4000, y=0x5000, yt=BF16, mean=0x6000, rstd=0x7000, stream=None))
N8 = (("x", "xt", "ldx", "r", "rt", "ldr", "M", "H", "w", "b", "wt", "eps", "center", "total", "codes", "scale", "stream"),
      dict(x=0x1000, xt=BF16, ldx=64, r=0x2000, rt=F32, ldr=64, M=4, H=64, w=0x3000, b=None, wt=F32, eps=1e-6, center=1,
           total=0x4000, codes=0x5000, scale=0x6000, stream=None))
ANB = (("t", "tt", "ldt", "M", "H", "w", "wt", "mean", "rstd", "dy", "dyt", "ldy", "dt", "ldd", "dx", "dw", "db", "ws", "n",
        "stream"),
       dict(t=0x1000, tt=F32, ldt=64, M=4, H=64, w=0x2000, wt=F32, mean=0x3000, rstd=0x4000, dy=0x5000, dyt=BF16, ldy=64,
            dt=0x6000, ldd=64, dx=0x7000, dw=0x8000, db=None, ws=0x9000, n=1 << 30, stream=None))
BAD_ADD = [
    (dict(xt=3), EUNSUP), (dict(rt=3), EUNSUP), (dict(wt=-1), EUNSUP), (dict(M=-1), EINVAL), (dict(M=2 ** 31), EINVAL),
    (dict(H=0), EUNSUP), (dict(H=8193, ldx=9000, ldr=9000), EUNSUP), (dict(ldx=63), EINVAL), (dict(ldr=63), EINVAL),
    (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(total=None), EINVAL), (dict(r=None), EINVAL),
    (dict(x=0x1001), EINVAL), (dict(r=0x2002), EINVAL), (dict(total=0x4002), EINVAL), (dict(b=0x8002), EINVAL),
    (dict(eps=-1.0), EINVAL), (dict(eps=NAN), EINVAL), (dict(eps=INF), EINVAL),
]


@pytest.mark.parametrize("kw,code", BAD_ADD + [
    (dict(yt=3), EUNSUP), (dict(center=0), EINVAL), (dict(mean=None), EINVAL), (dict(rstd=None), EINVAL),
    (dict(y=None), EINVAL), (dict(r=None, total=None), EINVAL), (dict(y=0x5001), EINVAL), (dict(mean=0x6002), EINVAL),
    (dict(M=0, x=None, r=None, total=None, y=None), OK),
])
def test_add_norm(L, kw, code):
    assert _call(L.qhead_add_norm, *ADDN, kw) == code
    assert (L.qhead_last_error().decode() == "") == (code == OK)


@pytest.mark.parametrize("kw,code", BAD_ADD + [
    (dict(codes=None), EINVAL), (dict(scale=None), EINVAL), (dict(scale=0x6002), EINVAL), (dict(M=0, x=None, codes=None), OK),
])
def test_norm_8bit(L, kw, code):
    assert _call(L.qhead_norm_8bit, *N8, kw) == code
    assert (L.qhead_last_error().decode() == "") == (code == OK)


@pytest.mark.parametrize("kw,code", [
    (dict(tt=3), EUNSUP), (dict(dyt=3), EUNSUP), (dict(M=-1), EINVAL), (dict(H=8193), EUNSUP), (dict(ldt=63), EINVAL),
    (dict(ldy=63), EINVAL), (dict(ldd=63), EINVAL), (dict(t=None), EINVAL), (dict(dy=None), EINVAL), (dict(dx=None), EINVAL),
    (dict(dw=None), EINVAL), (dict(rstd=None), EINVAL), (dict(dt=0x6002), EINVAL), (dict(ws=None), EINVAL),
    (dict(ws=0x9010), EINVAL), (dict(n=10), EINVAL), (dict(dt=None, dw=None), EINVAL), (dict(dt=None, n=10), EINVAL),
])
def test_add_norm_bwd(L, kw, code):
    assert _call(L.qhead_add_norm_bwd, *ANB, kw) == code
    assert L.qhead_last_error().decode()


def _clip(L, ps, ns, ts, max_norm=1.0, out=None, ots=None, norm=0x100, ws=0x200, n=1 << 30, fn="qhead_clip_grads"):
    P, N, T = ctypes.c_void_p * len(ps), ctypes.c_int64 * len(ps), ctypes.c_int * len(ps)
    args = [P(*ps), N(*ns), T(*ts), len(ps)]
    if fn == "qhead_clip_grads":
        args += [max_norm, None if out is None else P(*out), None if ots is None else T(*ots)]
    return getattr(L, fn)(*[ctypes.cast(a, ctypes.c_void_p) if isinstance(a, ctypes.Array) else a for a in args], norm, ws,
                          n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(ts=[F32, E4M3]), EUNSUP), (dict(ts=[F32, -1]), EUNSUP), (dict(ns=[4, -1]), EINVAL),
    (dict(ns=[2 ** 42, 2 ** 42]), EINVAL), (dict(ns=[2 ** 62, 2 ** 62]), EINVAL), (dict(ps=[0x1000, None]), EINVAL),
    (dict(ps=[0x1000, 0x2002]), EINVAL), (dict(norm=None), EINVAL), (dict(norm=0x102), EINVAL), (dict(ws=None), EINVAL),
    (dict(ws=0x210), EINVAL), (dict(n=10), EINVAL),
])
@pytest.mark.parametrize("fn", ["qhead_grad_norm", "qhead_clip_grads"])
def test_grad_norm_and_clip(L, fn, kw, code):
    base = dict(ps=[0x1000, 0x2000], ns=[4, 8], ts=[F32, F32])
    assert _clip(L, **{**base, **kw}, fn=fn) == code and L.qhead_last_error().decode()


@pytest.mark.parametrize("kw,code", [
    (dict(max_norm=0.0), EINVAL), (dict(max_norm=-1.0), EINVAL), (dict(max_norm=NAN), EINVAL), (dict(max_norm=INF), EINVAL),
    (dict(out=[0x5000, 0x6000]), EINVAL), (dict(ots=[F32, F32]), EINVAL), (dict(out=[0x5000, None], ots=[F32, F32]), EINVAL),
    (dict(out=[0x5000, 0x6002], ots=[F32, F32]), EINVAL), (dict(out=[0x5000, 0x6000], ots=[F32, E4M3]), EUNSUP),
    # overlaps: an output in another's place, in a tensor's, in its own with another type
    (dict(out=[0x5000, 0x500c], ots=[F32, F32]), EINVAL), (dict(out=[0x2010, 0x6000], ots=[F32, F32]), EINVAL),
    (dict(out=[0x1000, 0x6000], ots=[BF16, F32]), EINVAL), (dict(out=[0x1004, 0x6000], ots=[F32, F32]), EINVAL),
    (dict(ps=[0x1000, 0x100c]), EINVAL), (dict(ps=[0x1000, 0x1000], ns=[4, 4]), EINVAL),
    (dict(ps=[0x1000, 0x1000], ns=[4, 4], out=[0x1000, 0x6000], ots=[F32, F32]), EINVAL),
])
def test_clip_refusals(L, kw, code):
    base = dict(ps=[0x1000, 0x2000], ns=[4, 8], ts=[F32, F32])
    assert _clip(L, **{**base, **kw}) == code and L.qhead_last_error().decode()


def test_grad_norm_sizes(L):
    assert L.qhead_grad_norm_workspace(-1) == BAD_SIZE and L.qhead_grad_norm_workspace(2 ** 20 + 1) == BAD_SIZE
    assert 0 < L.qhead_grad_norm_workspace(1) == L.qhead_grad_norm_workspace(480) < L.qhead_grad_norm_workspace(481)
    assert _clip(L, [0] * 3, [1] * 3, [F32] * 3, norm=None) == EINVAL
    assert L.qhead_grad_norm(None, None, None, -1, 0x100, 0x200, 100, None) == EINVAL
    assert L.qhead_grad_norm(None, None, None, 2, 0x100, 0x200, 1 << 30, None) == EINVAL


# ------------------------------------------------------------------ the binding

M, K, N = 6, 64, 32


def _inputs():
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    return dict(x=f(M, K).to(BF), w=f(N, K).to(BF), b=f(N), r=f(M, N), x8=f(M, K).to(E8), w8=f(N, K).to(E8), xs=f(M), ws=f(N),
                dy=f(M, N), pre=f(M, N).half(), h=f(M, K), g=f(K), mean=f(M), rstd=f(M), t1=f(9), t2=f(4).to(BF), o1=f(9),
                o2=f(4))


CALLS = {
    "linear": lambda a, **s: qhead.linear(a["x"], a["w"], a["b"], "silu", a["r"], want_pre=True, **s),
    "linear_8bit": lambda a, **s: qhead.linear(a["x8"], a["w8"], a["b"], x_scale=a["xs"], w_scale=a["ws"], **s),
    "linear_bwd": lambda a, **s: qhead.linear_bwd(a["x"], a["w"], a["dy"], a["pre"], "silu", **s),
    "add_norm": lambda a, **s: qhead.add_norm(a["h"], a["h"].clone() if not s else a["h"], a["g"], a["g"], **s),
    "norm_8bit": lambda a, **s: qhead.norm_8bit(a["h"], a["g"], residual=a["x"], **s),
    "add_norm_bwd": lambda a, **s: qhead.add_norm_bwd(a["h"], a["g"], a["mean"], a["rstd"], a["x"], a["h"], **s),
    "grad_norm": lambda a, **s: qhead.grad_norm([a["t1"], a["t2"]], **s),
    "clip_grads": lambda a, **s: qhead.clip_grads([a["t1"], a["t2"]], 1.0, **s),
    "clip_grads_out": lambda a, **s: qhead.clip_grads([a["t1"], a["t2"]], 1.0, out=[a["o1"], a["o2"]], **s),
}


@pytest.mark.parametrize("name", CALLS)
def test_host_tensors(monkeypatch, name):
    monkeypatch.setattr(qhead, "lib", lambda: NoLaunch())
    monkeypatch.setattr(qhead, "_linear_sizes", {})
    with pytest.raises(ValueError, match="must be on a GPU"):
        CALLS[name](_inputs())


@pytest.mark.parametrize("name", CALLS)
def test_call_on_a_given_stream(world, monkeypatch, name):  # noqa: F811
    """Workspace and outputs from the given stream's pool, the outputs recorded on the
    current stream, the inputs on the given one."""
    monkeypatch.setattr(qhead, "_linear_sizes", {})
    given, current, lib, recorded, made = world
    a = _inputs()
    made.clear()
    got = CALLS[name](a, stream=given)
    assert len(lib.calls) == 1 and lib.calls[0][1][-1] == given.cuda_stream
    assert made and all(s is given for _, _, s in made)
    outs = [t for t in (got if isinstance(got, tuple) else (got,)) if t is not None]
    mine = {p for p, _, _ in made}
    on_current, on_given = recorded.get(id(current), []), recorded.get(id(given), [])
    assert all(t.data_ptr() in mine and _same(t, on_current) for t in outs)
    pointers = {x for x in lib.calls[0][1] if isinstance(x, int)}
    named = {"grad_norm": ("t1", "t2"), "clip_grads": ("t1", "t2"), "clip_grads_out": ("t1", "t2", "o1", "o2")}.get(name, ())
    for k, t in a.items():
        if t.data_ptr() in pointers or k in named:
            assert _same(t, on_given), k


X = torch.zeros(M, K, dtype=BF)
W = torch.zeros(N, K, dtype=BF)


@pytest.mark.parametrize("call", [
    lambda: qhead.linear(X, W.half()), lambda: qhead.linear(X.float(), W.float()), lambda: qhead.linear(X, W[:, 1:]),
    lambda: qhead.linear(X[0], W), lambda: qhead.linear(X, W.t()), lambda: qhead.linear(X.t(), torch.zeros(N, M, dtype=BF)),
    lambda: qhead.linear(X[:1].expand(M, K), W), lambda: qhead.linear(X, W, act="swish"), lambda: qhead.linear(X, W, act=None),
    lambda: qhead.linear(X, W, torch.zeros(N + 1)), lambda: qhead.linear(X, W, torch.zeros(N, 1)),
    lambda: qhead.linear(X, W, torch.zeros(2 * N)[::2]), lambda: qhead.linear(X, W, torch.zeros(N, dtype=torch.float64)),
    lambda: qhead.linear(X, W, residual=torch.zeros(M, N + 1)), lambda: qhead.linear(X, W, residual=torch.zeros(1, N)),
    lambda: qhead.linear(X, W, residual=torch.zeros(N, M).t()), lambda: qhead.linear(X, W, out_dtype=E8),
    lambda: qhead.linear(X, W, x_scale=torch.ones(M), w_scale=torch.ones(N)), lambda: qhead.linear(X.to(E8), W.to(E8)),
    lambda: qhead.linear(X.to(E8), W.to(E8), x_scale=torch.ones(M)),
    lambda: qhead.linear(X.to(E8), W.to(E8), x_scale=torch.ones(M, 1), w_scale=torch.ones(N)),
    lambda: qhead.linear(X.to(E8), W.to(E8), x_scale=torch.ones(M).half(), w_scale=torch.ones(N)),
    lambda: qhead.linear(None, W), lambda: qhead.linear(X, None), lambda: qhead.linear(X, W.to("meta")),
    lambda: qhead.linear_bwd(X.to(E8), W.to(E8), torch.zeros(M, N)), lambda: qhead.linear_bwd(X, W, torch.zeros(M, N + 1)),
    lambda: qhead.linear_bwd(X, W, torch.zeros(M, N), None, "silu"),
    lambda: qhead.linear_bwd(X, W, torch.zeros(M, N), torch.zeros(M, N), "silu"),
    lambda: qhead.linear_bwd(X, W, torch.zeros(1, N).expand(M, N)),
    lambda: qhead.add_norm(X, None, torch.ones(K)), lambda: qhead.add_norm(X, X[:1], torch.ones(K)),
    lambda: qhead.add_norm(X, X, None), lambda: qhead.add_norm(X, X, torch.ones(K + 1)),
    lambda: qhead.add_norm(X, X, torch.ones(K), torch.ones(K).half()), lambda: qhead.add_norm(X, X, torch.ones(K), out_dtype=E8),
    lambda: qhead.add_norm(X, X.t(), torch.ones(K)), lambda: qhead.add_norm(X.to(E8), X, torch.ones(K)),
    lambda: qhead.norm_8bit(X, torch.ones(K), residual=X[:, 1:]), lambda: qhead.norm_8bit(X[0], torch.ones(K)),
    lambda: qhead.add_norm_bwd(X, torch.ones(K), None, torch.ones(M), X, X.float()),
    lambda: qhead.add_norm_bwd(X, torch.ones(K), None, torch.ones(M), X, X[:, 1:]),
    lambda: qhead.add_norm_bwd(X, torch.ones(K), None, torch.ones(M + 1), X, X),
    lambda: qhead.grad_norm([]), lambda: qhead.grad_norm([X, None]), lambda: qhead.grad_norm([X.t()]),
    lambda: qhead.grad_norm([X.double()]), lambda: qhead.clip_grads([], 1.0),
    lambda: qhead.clip_grads([X], 1.0, out=[]), lambda: qhead.clip_grads([X], 1.0, out=[X[1:]]),
    lambda: qhead.clip_grads([X], 1.0, out=[X.to("meta")]), lambda: qhead.clip_grads([X], 1.0, out=[X.to(E8)]),
])
def test_bad_tensors(monkeypatch, call):
    monkeypatch.setattr(qhead, "lib", lambda: NoLaunch())
    with pytest.raises(ValueError) as e:
        call()
    assert "must be on a GPU" not in str(e.value)


# ---------------------------------------------------------- the autograd forms

@pytest.fixture
def constants(monkeypatch):
    def const(*shape, dtype=F):
        return torch.full(shape, 0.5, dtype=dtype)

    monkeypatch.setattr(qhead, "linear", lambda x, w, *a, want_pre=False, **k: (
        (const(M, N, dtype=BF), const(M, N)) if want_pre else const(M, N, dtype=BF)))
    monkeypatch.setattr(qhead, "linear_bwd", lambda *a, want_dx, want_dw, want_dbias: (
        const(M, K, dtype=BF) if want_dx else None, const(N, K, dtype=BF) if want_dw else None,
        const(N, dtype=BF) if want_dbias else None))
    monkeypatch.setattr(qhead, "add_norm", lambda *a, **k: (const(M, K), const(M, K, dtype=BF), const(M), const(M)))
    monkeypatch.setattr(qhead, "add_norm_bwd", lambda t, w, m, r, dy, dt, want_dbias: (
        const(M, K, dtype=BF) if dt is None else const(M, K, dtype=BF) + dt, const(K), const(K) if want_dbias else None))


def _leaf(*shape, dtype=F):
    return torch.ones(*shape, dtype=dtype, requires_grad=True)


def _linear():
    a = _leaf(M, K, dtype=BF), _leaf(N, K, dtype=BF), _leaf(N), _leaf(M, N)
    return autograd.linear(a[0], a[1], a[2], "silu", a[3]), a[:3]


def _add_norm():
    a = _leaf(M, K), _leaf(M, K, dtype=BF), _leaf(K), _leaf(K)
    return autograd.add_norm(*a)[0], a


@pytest.mark.parametrize("form", [_linear, _add_norm])
def test_first_derivatives_only(constants, form):
    out, leaves = form()
    out.float().sum().backward()
    assert all((v.grad == 0.5).all() for v in leaves)
    out, leaves = form()
    grads = torch.autograd.grad(out.float().square().sum(), leaves, create_graph=True)
    with pytest.raises(RuntimeError):
        (out.float().sum() + sum(g.float().square().sum() for g in grads)).backward()


def test_only_what_is_asked_for(constants):
    x, w, r = torch.ones(M, K, dtype=BF), _leaf(N, K, dtype=BF), _leaf(M, N)
    autograd.linear(x, w, None, "gelu", r).float().sum().backward()
    assert (w.grad == 0.5).all() and (r.grad == 1).all() and r.grad.dtype == F
    r.grad = None
    autograd.linear(x, w.detach(), None, "gelu", r).float().sum().backward()   # the residual alone
    assert (r.grad == 1).all()


def test_a_sum_that_is_used(constants):
    x, r, w = _leaf(M, K), _leaf(M, K, dtype=BF), _leaf(K)
    y, total = autograd.add_norm(x, r, w)
    (y.sum() + 2 * total.float().sum()).backward()
    assert (x.grad == 2.5).all() and x.grad.dtype == F and (r.grad == 2.5).all() and r.grad.dtype == BF
    for v in (x, r, w):
        v.grad = None
    autograd.add_norm(x, r, w)[1].float().sum().backward()                     # and only it
    assert (x.grad == 1).all() and (r.grad == 1).all() and w.grad is None


def test_an_operand_changed_in_place_is_noticed(constants):
    x, w = _leaf(M, K, dtype=BF), _leaf(N, K, dtype=BF)
    y = autograd.linear(x * 1, w, None, "silu")
    with torch.no_grad():
        w.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.float().sum().backward()
