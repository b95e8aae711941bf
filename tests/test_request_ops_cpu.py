"""CPU checks of the per-request decode operators: every argument is checked
on the host before anything touches CUDA (so the refusals need no GPU), the
binding's constants are the header's, and the double-precision references the
GPU tests use agree with hand-computed cases."""
from __future__ import annotations

import ctypes
import os
import re
import shutil

import numpy as np
import pytest

import request_refs as refs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, I64, INT, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
INVALID, SHAPE, UNSUPPORTED = 1, 2, 5


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from q8_block_quantized_02_b200 import build
    return ctypes.CDLL(build.build())


def fn(lib, name, *argtypes):
    f = getattr(lib, name)
    f.restype, f.argtypes = INT, list(argtypes)
    return f


@pytest.mark.parametrize("name,extra", [("q8_lora", 0), ("q8_gemv_lora", 1), ("q8_gemv_lora_split", 1)])
@pytest.mark.parametrize("M,K,N,n_adapters,R,dtype,status", [
    (8, 48, 1, 1, 8, 0, SHAPE), (0, 32, 1, 1, 8, 0, SHAPE), (8, 0, 1, 1, 8, 0, SHAPE), (8, 32, 0, 1, 8, 0, SHAPE),
    (8, 32, 1, 0, 8, 0, SHAPE), (8, 32, 1, 1, 0, 0, SHAPE), (8, 32, 1, 1, 12, 0, SHAPE), (8, 32, -1, 1, 8, 0, SHAPE),
    (8, 32, 17, 1, 8, 0, UNSUPPORTED), (8, 32, 2 ** 32 + 1, 1, 8, 0, UNSUPPORTED), (8, 32, 1, 1, 136, 0, UNSUPPORTED),
    (8, 32, 1, 1, 2 ** 32 + 8, 0, UNSUPPORTED), (2 ** 25 + 1, 32, 1, 1, 8, 0, UNSUPPORTED),
    (8, 2 ** 24 + 32, 1, 1, 8, 0, UNSUPPORTED), (8, 32, 1, 2 ** 32 + 1, 8, 0, UNSUPPORTED),
    (8, 32, 1, 1, 8, 3, INVALID), (8, 32, 1, 1, 8, -1, INVALID), (8, 32, 1, 1, 8, 2, INVALID)])  # last: null x
def test_lora_refusals(lib, name, extra, M, K, N, n_adapters, R, dtype, status):
    f = fn(lib, name, *([P] * (8 + extra)), I64, I64, I64, I64, I64, INT, P)
    assert f(*([None] * (8 + extra)), M, K, N, n_adapters, R, dtype, None) == status


@pytest.mark.parametrize("T,E,k,G,keep,top,score,renorm,scale,status", [
    (0, 8, 1, 1, 1, 1, 0, 0, 1.0, SHAPE), (1, 0, 1, 1, 1, 1, 0, 0, 1.0, SHAPE), (1, 8, 0, 1, 1, 1, 0, 0, 1.0, SHAPE),
    (1, 8, 9, 1, 1, 1, 0, 0, 1.0, SHAPE), (1, 9, 2, 2, 1, 1, 0, 0, 1.0, SHAPE), (1, 8, 2, 2, 3, 1, 0, 0, 1.0, SHAPE),
    (1, 8, 3, 4, 1, 1, 0, 0, 1.0, SHAPE), (1, 8, 2, 0, 1, 1, 0, 0, 1.0, SHAPE), (1, 8, 2, 2, 0, 1, 0, 0, 1.0, SHAPE),
    (1, 8, 2, 8, 2, 2, 0, 0, 1.0, SHAPE),  # group_top above the group's size
    (2 ** 20 + 1, 8, 2, 1, 1, 1, 0, 0, 1.0, UNSUPPORTED), (1, 257, 2, 1, 1, 1, 0, 0, 1.0, UNSUPPORTED),
    (1, 64, 9, 1, 1, 1, 0, 0, 1.0, UNSUPPORTED), (1, 128, 2, 64, 32, 1, 0, 0, 1.0, UNSUPPORTED),
    (2 ** 32 + 1, 8, 2, 1, 1, 1, 0, 0, 1.0, UNSUPPORTED),
    (1, 8, 2, 2, 1, 3, 0, 0, 1.0, INVALID), (1, 8, 2, 2, 1, 0, 0, 0, 1.0, INVALID), (1, 8, 2, 1, 1, 1, 2, 0, 1.0, INVALID),
    (1, 8, 2, 1, 1, 1, 0, 2, 1.0, INVALID), (1, 8, 2, 1, 1, 1, 0, 0, float("nan"), INVALID),
    (1, 8, 2, 1, 1, 1, 0, 0, float("inf"), INVALID), (1, 8, 2, 1, 1, 1, 1, 1, 2.5, INVALID)])  # last: null logits
def test_route_grouped_refusals(lib, T, E, k, G, keep, top, score, renorm, scale, status):
    f = fn(lib, "q8_moe_route_grouped", P, P, I64, I64, I64, I64, I64, INT, INT, INT, F, P, P, P)
    assert f(None, None, T, E, k, G, keep, top, score, renorm, scale, None, None, None) == status


@pytest.mark.parametrize("N,V,ld,status", [
    (0, 8, 8, SHAPE), (-1, 8, 8, SHAPE), (1, 0, 8, SHAPE), (1, 8, 7, SHAPE), (1, -8, 8, SHAPE),
    (65537, 8, 8, UNSUPPORTED), (1, 524289, 524289, UNSUPPORTED), (1, 8, 2 ** 31 + 1, UNSUPPORTED),
    (2 ** 32 + 1, 8, 8, UNSUPPORTED), (1, 8, 8, INVALID)])  # last: null logits
def test_sample_refusals(lib, N, V, ld, status):
    f = fn(lib, "q8_sample", *([P] * 8), I64, I64, I64, P)
    assert f(*([None] * 8), N, V, ld, None) == status


def test_constants_match_the_header():
    import q8_block_quantized_02_b200 as q8
    text = open(os.path.join(ROOT, "include", "q8.h")).read()
    for name in ("Q8_F32", "Q8_F16", "Q8_BF16", "Q8_SCORE_SOFTMAX", "Q8_SCORE_SIGMOID"):
        assert int(re.search(rf"\b{name} = (\d+)", text).group(1)) == getattr(q8, name)


def test_sample_reference_by_hand():
    l = np.log(np.array([0.1, 0.4, 0.2, 0.3], np.float32))
    for u, want in ((0.0, 0), (0.05, 0), (0.15, 1), (0.45, 1), (0.55, 2), (0.75, 3), (0.999, 3)):
        assert refs.sample_row(l, u=u)[0] == want
    assert refs.sample_row(l, top_k=2, u=0.5)[0] == 1       # {1: 4/7, 3: 3/7}
    assert refs.sample_row(l, top_k=2, u=0.6)[0] == 3
    assert list(refs.sample_row(l, top_p=0.65)[2]) == [False, True, False, True]   # 0.4, 0.7 >= 0.65
    assert list(refs.sample_row(l, min_p=0.6)[2]) == [False, True, False, True]    # 0.3 / 0.4 >= 0.6
    assert list(refs.sample_row(l, top_p=0.0)[2]) == [False, True, False, False]
    assert refs.sample_row(l, temperature=0.0, u=0.9) [:2] == (1, 1.0)
    t, p, kept = refs.sample_row([1.0, 1.0, 1.0, 1.0], top_p=0.5, u=0.6)
    assert (t, p) == (1, 0.5) and kept.sum() == 2            # ties: lowest indices
    assert refs.sample_row([-np.inf] * 3)[:2] == (-1, 0.0)
    assert refs.sample_row([np.nan, 0.0], u=0.0)[0] == 1
    assert refs.sample_row([np.inf, 0.0, np.inf], u=0.6)[:2] == (2, 0.5)


def test_route_reference_by_hand():
    z = np.log(np.array([1, 2, 3, 4], np.float32))
    idx, w = refs.route_token(z, None, 2, 1, 1, 1, False, False, 1.0)
    assert list(idx) == [3, 2] and np.allclose(w, [0.4, 0.3])
    idx, w = refs.route_token(z, None, 2, 1, 1, 1, False, True, 2.0)
    assert np.allclose(w, [8 / 7, 6 / 7])
    # groups {0, 1} and {2, 3}: a bias lifts expert 0, its group wins by the maximum, not by the sum of two
    b = np.array([0.31, -0.2, 0, 0], np.float32)
    assert list(refs.route_token(z, b, 2, 2, 1, 1, False, False, 1.0)[0]) == [0, 1]
    assert list(refs.route_token(z, b, 2, 2, 1, 2, False, False, 1.0)[0]) == [3, 2]
    assert list(refs.route_token(np.zeros(6), None, 3, 3, 2, 1, True, False, 1.0)[0]) == [0, 1, 2]


def test_lora_reference_by_hand():
    x = np.array([[1.0, 2.0]], np.float32)
    A = np.array([[[1.0, 1.0], [np.nan, np.nan]]], np.float32)
    B = np.array([[[2.0, np.inf], [-1.0, np.nan]]], np.float32)
    y, mag = refs.lora(x, A, B, [1], [0.5], [0], np.array([[10.0, 20.0]], np.float32))
    assert y.tolist() == [[13.0, 18.5]] and mag.tolist() == [[3.0, 1.5]]
    y, _ = refs.lora(x, A, B, [1], [0.5], [-1], None)
    assert y.tolist() == [[0.0, 0.0]]
