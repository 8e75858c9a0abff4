"""Layer norm with many rows to a block: at least six steps of every row loop and an
odd rest, so that ring slots are refilled with live rows, the row fetched ahead is
used, and the alternating sums alternate.  Checked element by element with the
tolerances of the shorter cases."""
import pytest
import torch

from test_norm_gpu import BF, F, HF, _check_bwd, _check_fwd, _inputs, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


# rows a step over a GB300's 152 SMs: 16-byte backward 1216 at 1536 columns, 304 at
# 4096, 152 at 8192; single elements 2432 (backward, 67 columns) to 152
@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("M,H,xt,dt,pad", [
    (8001, 1536, BF, BF, 0),
    (8001, 1536, BF, F, 8),
    (3001, 4096, F, F, 0),
    (2501, 4096, HF, BF, 16),
    (1501, 8192, BF, BF, 0),
    (1501, 8192, F, HF, 8),
    (30001, 256, BF, F, 0),
    (20001, 67, F, F, 0),
    (20003, 301, BF, F, 3),
    (4003, 2563, F, F, 5),
    (4003, 2563, BF, BF, 2),
    (1001, 8191, F, BF, 0),
    (2501, 1025, HF, HF, 1),
])
def test_backward(center, M, H, xt, dt, pad):
    _check_bwd(M, H, xt, dt, F, center, pad)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("M,H,xt,out,pad", [
    (40001, 67, F, F, 0),
    (20003, 301, BF, BF, 3),
    (10001, 701, HF, F, 1),
    (8003, 1500, BF, F, 1),
    (4003, 2563, F, BF, 5),
    (4003, 3500, BF, BF, 1),
    (1501, 5001, F, F, 0),
    (1001, 8191, BF, F, 1),
    (20001, 1536, BF, BF, 8),
])
def test_forward(center, M, H, xt, out, pad):
    x, w, b = _inputs(M, H, xt, F, M + H, offset=0.5, pad=pad)
    _check_fwd(x, w, b, 1e-5, center, out)


def test_without_dbias():
    _check_bwd(4001, 1536, BF, BF, BF, False, want_dbias=False)
    _check_bwd(4001, 333, BF, F, BF, True, want_dbias=False)
