"""Refusals of the serving operators at the edges of what their arguments allow, without a GPU."""
import ctypes

import pytest

import selective_state_space_27_b200 as ms
from selective_state_space_27_b200 import build as msbuild
from tests.test_serving_cpu import BASE, conv_args, conv_filter
from tests.test_serving_edges_gpu import SCHEDULES


@pytest.fixture(scope="module")
def lib():
    msbuild.build()
    return ms.load_library()


def test_failures_need_a_count(lib):
    assert lib.mamba_ssd_packed_failures(None, None) == 1


@pytest.mark.parametrize("change", [
    dict(y=BASE + 128), dict(y=BASE - 128), dict(y=BASE + 99 * 128 + 64),                     # later and earlier rows
    dict(y=BASE + 126), dict(y=BASE - 2), dict(y=BASE + 2),                                   # an element of a row
    dict(x_token_stride=200, y_token_stride=200, y=BASE + 126), dict(x_token_stride=200, y_token_stride=200, y=BASE + 274),
    dict(x_token_stride=200, y_token_stride=100, y=BASE + 128), dict(x_token_stride=0, y=BASE - 64 * 128),
    dict(tokens=1, y=BASE + 2), dict(tokens=1, y=BASE - 126),
])
def test_conv_packed_refuses_overlapping_outputs(lib, change):
    """y that shares elements with x: its rows are written while x's are read again for later rows."""
    assert lib.mamba_conv_packed_fwd(ctypes.byref(conv_args(**change)), ctypes.byref(conv_filter()), None) == 1
    assert b"overlap" in lib.mamba_last_error()


def test_schedules_of_these_sizes(lib):
    """ms::ssd_packed_plan, which chooses a call's schedule from its sizes, on 148 SMs."""
    plan = lib["_ZN2ms15ssd_packed_planEllllli"]
    plan.restype, plan.argtypes = ctypes.c_int64, [ctypes.c_int64] * 5 + [ctypes.c_int]   # (two int32 in one register)
    extra = 130 + 3                                          # rows of no sequence
    for lens, heads, groups, *_, longest, schedule in SCHEDULES:
        got = plan(sum(lens) + extra, len(lens), heads, groups, longest, 148)
        assert (got & 0xFFFFFFFF, got >> 32) == schedule, (len(lens), heads)
