"""The gradient of the product over many rows: at least six turns of the row loops that form
dz and its column sums, with an odd rest, so that every turn's rows and sums count.  Checked
element by element with the tolerances of the shorter cases.

A block takes 24 rows a turn (16 of float32 dy, 8 of single elements) of the share that 608
(456) blocks leave it: 60 blocks stand above each other at 2560 columns, 45 with float32 dy,
152 at 1024."""
import pytest
import torch

from test_linear_gpu import BF, F, HF, _lib, check_bwd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N,t,act,dt,pad", [
    (9001, 64, 2560, BF, "silu", BF, 0),
    (9001, 64, 2560, HF, "gelu", F, 8),
    (9013, 40, 2560, BF, "none", F, 0),
    (23011, 64, 1024, BF, "relu", HF, 16),
    (23011, 16, 1024, HF, "gelu_tanh", HF, 0),
    (40003, 64, 264, BF, "silu", BF, 8),
    (9001, 64, 2563, BF, "silu", BF, 0),
    (9001, 64, 2563, HF, "gelu", F, 1),
])
def test_gradient(M, K, N, t, act, dt, pad):
    check_bwd(M, K, N, t, act, dt, pad)


def test_sums_alone():
    """dy as it is: its column sums without a dz that is written."""
    check_bwd(9001, 64, 2560, BF, "none", BF)
