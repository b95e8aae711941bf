"""GPU: an infinite scale of an adapter reaches the outputs as an infinity, whatever the adapter's rank: what lies past
the rank takes no part."""
from __future__ import annotations

import numpy as np
import pytest

from test_gpu_lora import bank_of, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rank", [1, 5, 8, 13, 24, 27])
def test_infinite_scale(dtype, rank):
    M, K, R = 70, 96, 32
    A, B, _, _, _ = bank_of(rank, 2, R, M, K, dtype)
    A, B = A.abs() + 2.0 ** -6, B.abs() + 2.0 ** -6  # no product of both signs, none zero
    x = np.abs(np.random.default_rng(rank).standard_normal((2, K)).astype(np.float32)) + 0.5
    y = run(x, A.cuda(), B.cuda(), [rank, rank], np.array([np.inf, -np.inf], np.float32), [0, 1], None, M, K, dtype)
    assert np.all(y[0] == np.inf) and np.all(y[1] == -np.inf)
