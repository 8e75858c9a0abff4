"""The norm behind an addition with many rows to a block: at least six steps of every row
loop and an odd rest, so that ring slots are refilled with live rows, the row fetched ahead
is used, and the alternating sums alternate.  Checked element by element with the
tolerances of the shorter cases.

Rows a step over a GB300's 152 SMs: gradient 608 to 1216 at 1536 columns, 152 to 304 at
4096; single elements 3648 (67 columns) to 152 (8191)."""
import pytest
import torch

import test_add_norm_gpu as one
from test_add_norm_gpu import BF, F, HF, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("M,H,tt,dt,pad", [
    (8001, 1536, F, BF, 0), (8001, 1536, BF, BF, 8), (8001, 1536, HF, F, 0), (1501, 4096, F, F, 8), (2501, 4096, BF, HF, 0),
    (1501, 6400, F, F, 0), (1501, 8192, BF, BF, 0), (1501, 8192, HF, F, 8), (30001, 256, F, HF, 0), (30001, 256, BF, F, 0),
    # single elements
    (20001, 67, F, F, 0), (20003, 301, BF, F, 3), (4003, 2563, F, BF, 5), (4003, 2563, BF, BF, 2), (1001, 8191, HF, F, 0),
])
def test_gradient(center, M, H, tt, dt, pad):
    one.test_gradient(center, M, H, tt, dt, F, pad)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("M,H", [(25001, 67), (12001, 301), (6003, 701), (4001, 1500), (2503, 2563), (2001, 3500), (1001, 5001),
                                 (1001, 8191)])
@pytest.mark.parametrize("xt,rt,pad,padr", [(BF, BF, 0, 3), (HF, F, 5, 0)])
def test_single_elements(center, M, H, xt, rt, pad, padr):
    one.test_forward(center, M, H, xt, rt, F, True, pad, padr)
    one.test_8_bits(center, M, H, xt, rt, BF, False, pad, padr)


@pytest.mark.parametrize("H", [2560, 8192])
def test_rows_of_16_byte_accesses(H):
    one.test_forward(True, 5001, H, BF, F, F, True, 8, 0)
    one.test_8_bits(False, 5001, H, BF, BF, BF, False, 0, 8)


@pytest.mark.parametrize("M,H,tt,dt", [(61, 6400, F, F), (61, 6408, F, F), (1001, 6408, F, F), (61, 7680, F, BF), (61, 7688, F, HF),
                                       (61, 7688, BF, F)])
def test_gradient_where_the_ring_ends(M, H, tt, dt):
    """The widest rows of three streams that a ring holds, and the next ones."""
    one.test_gradient(True, M, H, tt, dt, F, 0)
