"""The bias gradient's own type: refusals, and what the autograd form asks for.  Nothing here
reaches a GPU."""
import pytest
import torch

from test_block_host import BF16, E4M3, EINVAL, EUNSUP, F16, F32, K, LBWD, M, N, OK, _call, _leaf
from test_block_host import L  # noqa: F401  (a fixture)
from test_device_host import Library as NoLaunch
from verify_vocab_blocked_gb300 import autograd, qhead

ORDER = tuple(n for k in LBWD[0] for n in ((k, "dbt") if k == "db" else (k,)))
BASE = dict(LBWD[1], db=0x9000, dbt=F32)


@pytest.mark.parametrize("kw,code", [
    (dict(dbt=E4M3), EUNSUP), (dict(dbt=-1), EUNSUP), (dict(db=0x9002), EINVAL), (dict(db=0x9001, dbt=F16), EINVAL),
    (dict(db=0x9001, dbt=BF16), EINVAL), (dict(db=0x9002, dbt=F16, wsp=None), EINVAL), (dict(t=F32), EUNSUP),
    (dict(db=None, dbt=9, M=0, x=None, dy=None, pre=None, dw=None, wsp=None), OK),
])
def test_refusals(L, kw, code):  # noqa: F811
    assert _call(L.qhead_linear_bwd_dbias, ORDER, BASE, kw) == code
    assert (L.qhead_last_error().decode() == "") == (code == OK)


def test_a_bad_type(monkeypatch):
    monkeypatch.setattr(qhead, "lib", lambda: NoLaunch())
    x, w = torch.zeros(M, K).bfloat16(), torch.zeros(N, K).bfloat16()
    with pytest.raises(ValueError, match="dbias_dtype must be"):
        qhead.linear_bwd(x, w, torch.zeros(M, N), None, "none", torch.float64)


@pytest.mark.parametrize("t", [torch.float32, torch.float16, torch.bfloat16, None])
def test_the_autograd_form_asks_for_the_bias_type(monkeypatch, t):
    asked = []

    def bwd(x, w, dy, pre, act, dbias_dtype, *, want_dx, want_dw, want_dbias):
        asked.append((dbias_dtype, want_dbias))
        return x, w, torch.ones(N, dtype=dbias_dtype) if want_dbias else None

    monkeypatch.setattr(qhead, "linear", lambda *a, want_pre=False, **k: torch.zeros(M, N, dtype=torch.bfloat16))
    monkeypatch.setattr(qhead, "linear_bwd", bwd)
    b = None if t is None else _leaf(N, dtype=t)
    autograd.linear(_leaf(M, K, dtype=torch.bfloat16), _leaf(N, K, dtype=torch.bfloat16), b).sum().backward()
    assert asked == [(t, t is not None)]
    assert b is None or b.grad.dtype == t
