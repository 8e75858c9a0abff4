"""Refusals of the operators beside the head: argument errors come back as
the documented codes before anything touches a GPU, and the binding checks
its tensors."""
import ctypes

import pytest
import torch

from verify_vocab_blocked_gb300 import build as qbuild
from verify_vocab_blocked_gb300 import qhead

EINVAL, EUNSUP, OK = qhead.QHEAD_EINVAL, qhead.QHEAD_EUNSUPPORTED, qhead.QHEAD_OK
BAD_SIZE = ctypes.c_size_t(-1).value
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return qhead.lib()


def _head(**kw):
    # never-dereferenced device addresses
    base = dict(wq=0x10000, scales=0x20000, biases=0x30000, V=1000, H=256, bits=4, group=64,
                sb_dtype=qhead.QHEAD_SB_F16, softcap=0.0)
    base.update(kw)
    return qhead.CHead(**base)


def _call(fn, order, base, kw):
    a = dict(base)
    a.update(kw)
    vals = [ctypes.byref(a[k]) if isinstance(a[k], qhead.CHead) else a[k] for k in order]
    return fn(*vals)


EMBED = (("head", "tokens", "M", "mask", "scale", "out", "dt", "stream"),
         dict(head=_head(), tokens=0x1000, M=4, mask=None, scale=1.0, out=0x2000, dt=1, stream=None))
EMBED_BWD = (("head", "tokens", "M", "mask", "scale", "dout", "dt", "dw", "acc", "ws", "n", "stream"),
             dict(head=_head(), tokens=0x1000, M=4, mask=None, scale=1.0, dout=0x2000, dt=1,
                  dw=0x4000, acc=0, ws=0x8000, n=1 << 30, stream=None))
NORM = (("x", "xt", "ldx", "M", "H", "w", "b", "wt", "eps", "center", "y", "yt", "mean", "rstd",
         "stream"),
        dict(x=0x1000, xt=1, ldx=64, M=4, H=64, w=0x2000, b=None, wt=2, eps=1e-6, center=1,
             y=0x3000, yt=1, mean=0x4000, rstd=0x5000, stream=None))
NORM_BWD = (("x", "xt", "ldx", "M", "H", "w", "wt", "mean", "rstd", "dy", "dt", "ldy", "dx", "dw",
             "db", "ws", "n", "stream"),
            dict(x=0x1000, xt=1, ldx=64, M=4, H=64, w=0x2000, wt=2, mean=0x4000, rstd=0x5000,
                 dy=0x6000, dt=2, ldy=64, dx=0x7000, dw=0x8000, db=None, ws=0x9000, n=1 << 30,
                 stream=None))
DFWD = (("head", "h", "M", "ids", "t", "tt", "K", "T", "mask", "loss", "lse", "kept", "ws", "n",
         "stream"),
        dict(head=_head(), h=0x1000, M=4, ids=0x2000, t=0x3000, tt=2, K=8, T=1.0, mask=None,
             loss=0x4000, lse=0x5000, kept=0x6000, ws=0x10000, n=1 << 40, stream=None))
DBWD = (("head", "h", "M", "ids", "t", "tt", "K", "T", "mask", "kept", "lse", "dloss", "dh", "ws",
         "n", "stream"),
        dict(head=_head(), h=0x1000, M=4, ids=0x2000, t=0x3000, tt=2, K=8, T=1.0, mask=None,
             kept=0x6000, lse=0x5000, dloss=0x4000, dh=0x7000, ws=0x10000, n=1 << 40, stream=None))


@pytest.mark.parametrize("kw,code", [
    (dict(head=None), EINVAL), (dict(head=_head(bits=3)), EUNSUP), (dict(head=_head(H=100)), EUNSUP),
    (dict(M=-1), EINVAL), (dict(M=2 ** 31), EINVAL), (dict(tokens=None), EINVAL),
    (dict(out=None), EINVAL), (dict(out=0x2008), EINVAL), (dict(dt=3), EUNSUP),
    (dict(dt=-1), EUNSUP), (dict(scale=NAN), EINVAL), (dict(scale=INF), EINVAL),
    (dict(M=0, tokens=None, out=None), OK),
])
def test_embed(L, kw, code):
    assert _call(L.qhead_embed, *EMBED, kw) == code
    assert (L.qhead_last_error().decode() == "") == (code == OK)


@pytest.mark.parametrize("kw,code", [
    (dict(head=None), EINVAL), (dict(M=-1), EINVAL), (dict(M=2 ** 31), EINVAL),
    (dict(tokens=None), EINVAL), (dict(dout=None), EINVAL), (dict(dout=0x2004), EINVAL),
    (dict(dw=None), EINVAL), (dict(dw=0x4008), EINVAL), (dict(dt=9), EUNSUP),
    (dict(scale=-INF), EINVAL), (dict(ws=None), EINVAL), (dict(ws=0x8010), EINVAL),
    (dict(n=100), EINVAL), (dict(M=0, acc=1, tokens=None, dout=None, ws=None), OK),
])
def test_embed_bwd(L, kw, code):
    assert _call(L.qhead_embed_bwd, *EMBED_BWD, kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(y=None), EINVAL), (dict(rstd=None), EINVAL),
    (dict(mean=None), EINVAL), (dict(center=0), EINVAL), (dict(H=0), EUNSUP), (dict(H=8193, ldx=8193), EUNSUP),
    (dict(ldx=63), EINVAL), (dict(M=-1), EINVAL), (dict(xt=5), EUNSUP), (dict(wt=-1), EUNSUP),
    (dict(yt=3), EUNSUP), (dict(eps=-1e-6), EINVAL), (dict(eps=NAN), EINVAL), (dict(eps=INF), EINVAL),
    (dict(x=0x1001), EINVAL), (dict(w=0x2002), EINVAL), (dict(b=0x2002), EINVAL),
    (dict(y=0x3001), EINVAL), (dict(mean=0x4002), EINVAL), (dict(rstd=0x5001), EINVAL),
    (dict(M=0, y=None, rstd=None), OK),
])
def test_layer_norm(L, kw, code):
    assert _call(L.qhead_layer_norm, *NORM, kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(rstd=None), EINVAL), (dict(dy=None), EINVAL),
    (dict(dx=None), EINVAL), (dict(dw=None), EINVAL), (dict(H=0), EUNSUP), (dict(ldx=1), EINVAL),
    (dict(ldy=63), EINVAL), (dict(dt=4), EUNSUP), (dict(dy=0x6002), EINVAL), (dict(dx=0x7001), EINVAL),
    (dict(db=0x7002), EINVAL), (dict(ws=None), EINVAL), (dict(ws=0x9080), EINVAL), (dict(n=8), EINVAL),
    (dict(M=-2), EINVAL),
])
def test_layer_norm_bwd(L, kw, code):
    assert _call(L.qhead_layer_norm_bwd, *NORM_BWD, kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(head=None), EINVAL), (dict(head=_head(group=32)), EUNSUP), (dict(M=-1), EINVAL),
    (dict(h=None), EINVAL), (dict(h=0x1008), EINVAL), (dict(ids=None), EINVAL), (dict(t=None), EINVAL),
    (dict(tt=7), EUNSUP), (dict(K=0), EINVAL), (dict(K=1025), EINVAL), (dict(T=0.0), EINVAL),
    (dict(T=-1.0), EINVAL), (dict(T=NAN), EINVAL), (dict(T=INF), EINVAL), (dict(ws=None), EINVAL),
    (dict(ws=0x10010), EINVAL), (dict(M=0, h=None), OK),
])
def test_distill(L, kw, code):
    if kw.get("ws", 1) is None or kw.get("ws") == 0x10010:
        if qhead.lib().qhead_fwd_workspace(ctypes.byref(_head()), 4) == BAD_SIZE:
            pytest.skip("the plan needs a device")
    assert _call(L.qhead_distill_fwd, *DFWD, kw) == code
    assert _call(L.qhead_distill_bwd, *DBWD, kw) == code


@pytest.mark.parametrize("drop", ["loss", "lse", "kept"])
def test_distill_outputs(L, drop):
    assert _call(L.qhead_distill_fwd, *DFWD, {drop: None}) == EINVAL


@pytest.mark.parametrize("kw", [dict(kept=None), dict(lse=None), dict(dloss=None), dict(dh=None),
                                dict(dh=0x7008)])
def test_distill_bwd_args(L, kw):
    assert _call(L.qhead_distill_bwd, *DBWD, kw) == EINVAL


def test_workspace_queries(L):
    hd = ctypes.byref(_head())
    assert L.qhead_embed_bwd_workspace(hd, 0) == 0
    assert 0 < L.qhead_embed_bwd_workspace(hd, 1000) < 1 << 22
    assert L.qhead_embed_bwd_workspace(hd, -1) == BAD_SIZE
    assert L.qhead_embed_bwd_workspace(None, 5) == BAD_SIZE
    assert L.qhead_layer_norm_bwd_workspace(5, 0) == BAD_SIZE
    assert L.qhead_layer_norm_bwd_workspace(-1, 64) == BAD_SIZE
    assert L.qhead_distill_fwd_workspace(hd, 0, 4) == 0
    assert L.qhead_distill_fwd_workspace(hd, 5, 0) == BAD_SIZE
    assert L.qhead_distill_bwd_workspace(hd, 5, 1025) == BAD_SIZE
    assert L.qhead_distill_bwd_workspace(hd, -1, 4) == BAD_SIZE
    assert L.qhead_distill_kept(hd, 129, 4) == 40 + 1024      # V = 1000 in blocks of 32
    big = ctypes.byref(_head(V=1 << 20))
    assert L.qhead_distill_kept(big, 1024, 4) == 40 + (1 << 20)   # 4 GiB of logits
    assert L.qhead_distill_kept(big, 1025, 4) == 4 + 32
    assert L.qhead_distill_kept(ctypes.byref(_head(V=1 << 30)), 16, 4) == 40 + (1 << 30)
    assert L.qhead_distill_kept(hd, 5, 0) == -1


# ---- the binding's own checks (CPU tensors: refused before any call)

def _cpu_head():
    return qhead.Head(torch.zeros(10, 32, dtype=torch.int32), torch.zeros(10, 4).half(),
                      torch.zeros(10, 4).half(), 4)


@pytest.mark.parametrize("tokens", [
    torch.zeros(3), torch.zeros(3, dtype=torch.int64), torch.zeros(3, 1, dtype=torch.int32),
    torch.zeros(6, dtype=torch.int32)[::2], [1, 2]])
def test_binding_tokens(tokens):
    with pytest.raises(ValueError):
        qhead.embed(_cpu_head(), tokens)
    with pytest.raises(ValueError):
        qhead.embed_bwd(_cpu_head(), tokens, torch.zeros(3, 256))


def test_binding_embed():
    t = torch.zeros(3, dtype=torch.int32)
    for kw in (dict(mask=torch.ones(4, dtype=torch.bool)), dict(mask=torch.ones(3)),
               dict(out_dtype=torch.float64)):
        with pytest.raises(ValueError):
            qhead.embed(_cpu_head(), t, **kw)
    for dout, dw in ((torch.zeros(3, 255), None), (torch.zeros(3, 256).double(), None),
                     (torch.zeros(256, 3).t(), None), (torch.zeros(3, 256), torch.zeros(9, 256)),
                     (torch.zeros(3, 256), torch.zeros(10, 256).half()),
                     (torch.zeros(3, 256), torch.zeros(256, 10).t())):
        with pytest.raises(ValueError):
            qhead.embed_bwd(_cpu_head(), t, dout, dw=dw)


def test_binding_layer_norm():
    x, w = torch.zeros(4, 8), torch.ones(8)
    bad = [(x.double(), w, None), (x[0], w, None), (torch.zeros(8, 4).t(), w, None),
           (x[:1].expand(4, 8), w, None), (x, None, None), (x, torch.ones(7), None),
           (x, torch.ones(16)[::2], None), (x, w, torch.zeros(8).half()), (x, w, torch.zeros(9)),
           (None, w, None)]
    for a in bad:
        with pytest.raises(ValueError):
            qhead.layer_norm(*a)
    r = torch.zeros(4)
    for a in ((x, w, r, r, torch.zeros(4, 7)), (x, w, torch.zeros(3), r, x),
              (x, w, None, r.double(), x), (x, w, None, r[:3], x), (x, w, None, None, x)):
        with pytest.raises(ValueError):
            qhead.layer_norm_bwd(*a)


def test_binding_distill(L):
    hd, h = _cpu_head(), torch.zeros(3, 256, dtype=torch.bfloat16)
    ids, t = torch.zeros(3, 5, dtype=torch.int32), torch.zeros(3, 5)
    for a in ((h.float(), ids, t), (h, ids.long(), t), (h, ids[:2], t), (h, ids, t[:, :4]),
              (h, ids, t.double()), (h, ids[0], t), (h, ids.t().contiguous().t(), t),
              (h[:, :128].contiguous(), ids, t)):
        with pytest.raises(ValueError):
            qhead.distill_fwd(hd, *a)
    cols = qhead.lib().qhead_distill_kept(ctypes.byref(hd.c()), 3, 5)
    z, v = torch.zeros(3, cols), torch.zeros(3)
    for kept, lse, dl in ((z.half(), v, v), (z[:, :5].contiguous(), v, v), (z, v[:2], v), (z, v, v.double())):
        with pytest.raises(ValueError):
            qhead.distill_bwd(hd, h, ids, t, kept, lse, dl)
