"""The norm, quantiser and 8-bit Linear entry points without a GPU: sizes, and
argument checks that fail before any CUDA call."""
import ctypes

import pytest

from test_abi import libvnm  # noqa: F401  (fixture)

P = 256       # an aligned pointer that is never followed
INVALID = 1


def _call(lib, name, order, defaults, **change):
    return getattr(lib, name)(*[{**defaults, **change}[k] for k in order])


NORM = ("x ld_x res ld_r w eps T D type h ld_h y ld_y rstd q ld_q q_type s s_rs s_cs stream").split()
NORM_OK = dict(x=P, ld_x=64, res=P, ld_r=64, w=P, eps=1e-6, T=4, D=64, type=0, h=P, ld_h=64, y=P, ld_y=64, rstd=P, q=P,
               ld_q=64, q_type=0, s=P, s_rs=1, s_cs=1, stream=None)


@pytest.mark.parametrize("change", [
    dict(type=3), dict(type=-1), dict(T=-1), dict(D=-1), dict(T=(1 << 31) + 1), dict(eps=-1e-6), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(x=None), dict(x=P + 1), dict(ld_x=63), dict(ld_r=63), dict(ld_h=63), dict(ld_y=63),
    dict(ld_q=63), dict(res=None), dict(y=None, q=None, s=None), dict(s=None), dict(q=None), dict(q_type=2), dict(w=P + 1),
    dict(rstd=P + 2), dict(s=P + 2), dict(type=1, y=P + 2)])
def test_norm_refusals(libvnm, change):  # noqa: F811
    assert _call(libvnm, "vnm_rmsnorm", NORM, NORM_OK, **change) == INVALID


@pytest.mark.parametrize("change", [dict(T=0), dict(D=0), dict(T=0, x=None, y=None, q=None, s=None, h=None, res=None)])
def test_norm_without_work(libvnm, change):  # noqa: F811
    assert _call(libvnm, "vnm_rmsnorm", NORM, NORM_OK, **change) == 0


GRAD = "dy ld_dy h ld_h w rstd res ld_r T D type dh ld_dh dw ws ws_bytes stream".split()
GRAD_OK = dict(dy=P, ld_dy=64, h=P, ld_h=64, w=P, rstd=P, res=P, ld_r=64, T=4, D=64, type=0, dh=P, ld_dh=64, dw=P, ws=P,
               ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("change", [
    dict(type=7), dict(T=-1), dict(dy=None), dict(h=None), dict(rstd=None), dict(ld_dy=1), dict(ld_h=1), dict(ld_r=1),
    dict(ld_dh=1), dict(dh=None, dw=None), dict(ws=None), dict(ws=P + 8), dict(ws_bytes=4 * 64 * 4 - 1), dict(dw=P + 1),
    dict(w=P + 1), dict(dy=P + 1)])
def test_norm_backward_refusals(libvnm, change):  # noqa: F811
    assert _call(libvnm, "vnm_rmsnorm_backward", GRAD, GRAD_OK, **change) == INVALID


def test_norm_backward_workspace_size(libvnm):  # noqa: F811
    n = ctypes.c_size_t()
    for T, D in ((0, 5), (1, 4096), (8192, 4096), (100000, 33)):
        assert libvnm.vnm_rmsnorm_backward_workspace_size(T, D, ctypes.byref(n)) == 0
        assert n.value % (4 * D) == 0 and n.value <= 4 * D * T and (n.value > 0) == (T > 0)
    assert libvnm.vnm_rmsnorm_backward_workspace_size(-1, 4, ctypes.byref(n)) == INVALID
    assert libvnm.vnm_rmsnorm_backward_workspace_size(4, 4, None) == INVALID


QUANT = "x ld_x R C type rows q_type q ld_q s s_rs s_cs qt ld_qt st st_rs st_cs stream".split()
QUANT_OK = dict(x=P, ld_x=64, R=32, C=64, type=0, rows=1, q_type=0, q=P, ld_q=64, s=P, s_rs=1, s_cs=1, qt=P, ld_qt=32, st=P,
                st_rs=1, st_cs=1, stream=None)


@pytest.mark.parametrize("change", [
    dict(type=3), dict(rows=0), dict(rows=64), dict(q_type=2), dict(R=-1), dict(C=-1), dict(x=None), dict(x=P + 1),
    dict(ld_x=63), dict(ld_q=63), dict(ld_qt=31), dict(s=None), dict(q=None), dict(st=None), dict(qt=None),
    dict(q=None, s=None, qt=None, st=None), dict(s=P + 1), dict(st=P + 1)])
def test_quantize_refusals(libvnm, change):  # noqa: F811
    assert _call(libvnm, "vnm_fp8_quantize", QUANT, QUANT_OK, **change) == INVALID


LINEAR = ("x ld_x x_type xs xs_rs xs_cs w ld_w w_type ws ws_rs ws_cs rows T R K bias b_type act y ld_y y_type status "
          "stream").split()
LINEAR_OK = dict(x=P, ld_x=64, x_type=0, xs=P, xs_rs=1, xs_cs=1, w=P, ld_w=64, w_type=0, ws=P, ws_rs=1, ws_cs=1, rows=128,
                 T=4, R=32, K=64, bias=P, b_type=0, act=0, y=P, ld_y=32, y_type=0, status=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(x_type=2), dict(w_type=-1), dict(rows=2), dict(T=-1), dict(R=-1), dict(K=-1), dict(K=(1 << 31) + 1), dict(x=None),
    dict(x=P + 8), dict(w=None), dict(w=P + 1), dict(ld_x=63), dict(ld_x=72), dict(ld_w=72), dict(ld_w=48), dict(xs=None),
    dict(ws=None), dict(xs=P + 1), dict(ws=P + 2), dict(b_type=3), dict(bias=P + 1), dict(act=3), dict(y=None),
    dict(y=P + 1), dict(y_type=1, y=P + 2), dict(ld_y=31), dict(y_type=5), dict(status=P + 1)])
def test_linear_refusals(libvnm, change):  # noqa: F811
    assert _call(libvnm, "vnm_fp8_linear", LINEAR, LINEAR_OK, **change) == INVALID


def test_linear_without_work_and_the_testing_form(libvnm):  # noqa: F811
    assert _call(libvnm, "vnm_fp8_linear", LINEAR, LINEAR_OK, T=0) == 0
    assert _call(libvnm, "vnm_fp8_linear", LINEAR, LINEAR_OK, R=0) == 0
    order = LINEAR[:-1] + ["skip", "stream"]
    for change in (dict(skip=-1, status=P), dict(skip=1, status=None)):
        assert _call(libvnm, "vnm_testing_fp8_linear_skip_stage", order, {**LINEAR_OK, "skip": 0}, **change) == INVALID


def test_the_older_entry_points_still_refuse_bf16(libvnm):  # noqa: F811
    # VNM_BF16 (2) is no type of C there; found before the handle is used
    assert libvnm.vnm_bitmap_spmm(64, 8, P, P, P, P, P, 8, 8, P, 8, 2, None, 0, None) == INVALID
