"""sm_scale of cross attention and shared-prefix decode: finite numbers only
(no device work)."""
import ctypes

import numpy as np
import pytest

from test_rows_args import desc, lib  # noqa: F401 (lib is a fixture)

FLT_MAX = float(np.finfo(np.float32).max)


def cross(lib, scale, Nq=3, H_q=4, n=0):
    return lib.kv2_attention_cross(ctypes.byref(desc()), None, 256, 0x100, None, Nq, H_q, scale, 0x200, 0, 0x300, n, None)


def shared(lib, scale, n=0):
    return lib.kv2_attention_shared(ctypes.byref(desc(B=1)), None, 256, ctypes.byref(desc(B=6)), None, 256, 0x100, 4, scale, 0x200, 0,
                                    0x300, n, None)


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf"), 1e39])
def test_scales_that_are_not_numbers_are_refused(lib, scale):  # noqa: F811
    for Nq in (1, 3):                                              # both kernels
        assert cross(lib, scale, Nq) == 1 and b"sm_scale" in lib.kv2_last_error()
    assert cross(lib, scale, 0) == 1                               # also where there is nothing to do
    assert shared(lib, scale) == 1 and b"sm_scale" in lib.kv2_last_error()


@pytest.mark.parametrize("scale", [FLT_MAX, -FLT_MAX, 0.0, 1e-45])
def test_every_finite_scale_is_taken(lib, scale):  # noqa: F811
    # (ws of no bytes: the call ends at the workspace's check)
    assert cross(lib, scale, 1) == 6 and cross(lib, scale) == 6 and shared(lib, scale) == 6
