"""The dense 16-bit layers' test entry points without a GPU: a stage to leave out, or none, and the checks of the calls that
they change."""
import ctypes

import pytest

from test_abi import libvnm  # noqa: F401  (fixture)
from test_dense16_abi import BACK, BACK_OK, GATED, GATED_OK, INVALID


def _changed(order, defaults, extra, **change):
    """The arguments of the call, with ``extra`` before the stream."""
    args = [{**defaults, **change}[k] for k in order]
    return args[:-1] + list(extra) + args[-1:]


@pytest.mark.parametrize("skip", [-1, -2, -(1 << 31)])
def test_gated_refuses_no_stage(libvnm, skip):  # noqa: F811
    assert libvnm.vnm_testing_gated_linear_skip_stage(*_changed(GATED, GATED_OK, (skip,))) == INVALID


@pytest.mark.parametrize("skips", [(-2, 0), (0, -2)])
def test_backward_refuses_bad_stages(libvnm, skips):  # noqa: F811
    assert libvnm.vnm_testing_gated_linear_backward_skip_stage(*_changed(BACK, BACK_OK, skips)) == INVALID


def test_the_calls_checks_hold(libvnm):  # noqa: F811
    assert libvnm.vnm_testing_gated_linear_skip_stage(*_changed(GATED, GATED_OK, (0,), y=None)) == INVALID
    assert libvnm.vnm_testing_gated_linear_skip_stage(*_changed(GATED, GATED_OK, (0,), T=0)) == 0
    assert libvnm.vnm_testing_gated_linear_backward_skip_stage(*_changed(BACK, BACK_OK, (0, 0), ws=None)) == INVALID
    assert libvnm.vnm_testing_gated_linear_backward_skip_stage(*_changed(BACK, BACK_OK, (-1, -1), dx=None, dwg=None, dwu=None, h=None)) == 0


def test_plan_takes_the_alignment(libvnm):  # noqa: F811
    tile, rows, splits = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    out = ctypes.byref(tile), ctypes.byref(rows), ctypes.byref(splits)
    assert libvnm.vnm_testing_dense_plan(0, 3756, 7687, 273, 0, 0, 0, 1, 152, *out) == 0 and tile.value == 0
    assert libvnm.vnm_testing_dense_plan(0, 3756, 7687, 273, 0, 0, 0, 0, 152, *out) == 0 and tile.value == 128
    assert libvnm.vnm_testing_dense_plan(0, 3756, 7687, 273, 0, 0, 0, 2, 152, *out) == INVALID
