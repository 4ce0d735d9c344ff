"""Refusals of the serving operators at the edges of what their arguments allow, without a GPU."""
import ctypes

import pytest

import selective_state_space_27_b200 as ms
from selective_state_space_27_b200 import build as msbuild


@pytest.fixture(scope="module")
def lib():
    msbuild.build()
    return ms.load_library()


def test_failures_need_a_count(lib):
    assert lib.mamba_ssd_packed_failures(None, None) == 1
