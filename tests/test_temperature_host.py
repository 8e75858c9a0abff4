"""Temperatures that the distillation refuses."""
import pytest

from test_ops_host import DBWD, DFWD, EINVAL, L, _call  # noqa: F401


@pytest.mark.parametrize("T", [1e-45, 1e-40, 2.9e-39, 1.17e-38])
def test_below_the_normal_range(L, T):  # noqa: F811
    """The reciprocal is infinite there, or its product with log2(e): every loss NaN."""
    assert _call(L.qhead_distill_fwd, *DFWD, dict(T=T)) == EINVAL
    assert "temperature" in L.qhead_last_error().decode()
    assert _call(L.qhead_distill_bwd, *DBWD, dict(T=T)) == EINVAL
    assert "temperature" in L.qhead_last_error().decode()


def test_the_smallest_normal(L):  # noqa: F811
    assert _call(L.qhead_distill_fwd, *DFWD, dict(T=2.0 ** -126, loss=None)) == EINVAL
    assert "loss" in L.qhead_last_error().decode()
