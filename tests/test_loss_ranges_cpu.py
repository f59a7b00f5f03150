"""CPU checks of the linear losses' ranges: a temperature whose square, or a cap
whose reciprocal or double, is not a normal f32 number is refused, not answered
with NaN or 0."""
import ctypes

import pytest

from tests.test_losses_cpu import _distill, _distill_grad, _xent, _xent_grad

LOW, HIGH = 2.0 ** -63, 2.0 ** 63


@pytest.fixture(scope="module")
def fcc():
    import __graft_entry__
    __graft_entry__.build()
    import gemm_collective_gb300 as m
    return m


def test_temperatures_out_of_range_are_refused(fcc):
    for call in (_distill, _distill_grad):
        for tau in (1e-44, 1e-39, 1e-20, LOW * 0.999, HIGH * 1.001, 1e30, 3e38):
            assert call(fcc, tau=tau) == fcc.FCC_ERR_INVALID, (call.__name__, tau)
        for tau in (LOW, 0.5, 1.0, 100.0, HIGH):  # (accepted: refused for the form asked for, later)
            o = ctypes.byref(fcc.make_opts(algo=fcc.FCC_ALGO_UNFUSED))
            assert call(fcc, tau=tau, o=o) == fcc.FCC_ERR_UNSUPPORTED, (call.__name__, tau)


def test_caps_out_of_range_are_refused(fcc):
    for call in (_xent, _xent_grad, _distill, _distill_grad):
        for cap in (1e-45, 1e-39, 2.0 ** -127, 2.0 ** 126 * 1.001, 3e38):
            assert call(fcc, cap=cap) == fcc.FCC_ERR_INVALID, (call.__name__, cap)
        for cap in (0.0, 2.0 ** -126, 1e-3, 30.0, 1e30, 2.0 ** 126):
            o = ctypes.byref(fcc.make_opts(algo=fcc.FCC_ALGO_UNFUSED))
            assert call(fcc, cap=cap, o=o) == fcc.FCC_ERR_UNSUPPORTED, (call.__name__, cap)
