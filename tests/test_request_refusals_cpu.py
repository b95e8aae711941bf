"""CPU: where the per-request operators' refusals end.  A call whose arguments are all allowed gets as far as the check
of its pointers, which host memory does not pass."""
from __future__ import annotations

import ctypes
import os
import shutil

import numpy as np
import pytest

P, I64, INT, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
INVALID, NOT_DEVICE = 1, 4
FLT_MAX = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from q8_block_quantized_02_b200 import build
    return ctypes.CDLL(build.build())


@pytest.mark.parametrize("scale,status", [(1.0, NOT_DEVICE), (0.0, NOT_DEVICE), (-2.5, NOT_DEVICE), (FLT_MAX, NOT_DEVICE),
                                          (-FLT_MAX, NOT_DEVICE), (3.2e38, NOT_DEVICE), (float("inf"), INVALID),
                                          (float("-inf"), INVALID), (float("nan"), INVALID)])
def test_every_finite_route_scale_is_allowed(lib, scale, status):
    f = lib.q8_moe_route_grouped
    f.restype, f.argtypes = INT, [P, P, I64, I64, I64, I64, I64, INT, INT, INT, F, P, P, P]
    host = np.zeros(64, np.float32)
    p = host.ctypes.data
    assert f(p, None, 1, 8, 2, 2, 1, 1, 1, 1, scale, p, p, None) == status
