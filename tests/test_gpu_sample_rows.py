"""GPU parity of q8_sample on rows and parameters whose threads settle a row together in few steps, against double
precision (tests/test_sample_threads_cpu.py runs the same ones under schedules of its own)."""
from __future__ import annotations

import numpy as np
import pytest

from test_gpu_sample import check, sample

pytestmark = pytest.mark.gpu

NEG = -np.inf


@pytest.mark.parametrize("N", [1, 16, 160])
@pytest.mark.parametrize("live", [1, 20, 49])
def test_fewer_live_tokens_than_top_k(N, live):
    g = np.random.default_rng(N + live)
    V = 32000
    l = np.full((N, V), NEG, np.float32)
    for n in range(N):
        l[n, g.choice(V, live, replace=False)] = g.standard_normal(live).astype(np.float32) * 2
    u = g.random(N).astype(np.float32)
    check(l, top_k=50, u=u)
    check(l, top_k=50, top_p=0.7, min_p=0.02, u=u)
    cold = (g.standard_normal((N, V)) * 2).astype(np.float32)
    check(cold, top_k=50, temperature=0.004, u=u)


@pytest.mark.parametrize("N", [1, 16, 160])
@pytest.mark.parametrize("top_k", [20, 40, 50, 100, 128])
def test_two_sorts_in_turn(N, top_k):
    g = np.random.default_rng(N + top_k)
    l = (g.standard_normal((N, 32000)) * 2).astype(np.float32)
    for kw in ({}, dict(min_p=0.05), dict(top_p=0.8)):
        check(l, top_k=top_k, u=g.random(N).astype(np.float32), **kw)


@pytest.mark.parametrize("N,V", [(1, 3001), (16, 32000), (160, 32000), (4, 151936)])
def test_rows_without_top_k_and_top_p(N, V):
    g = np.random.default_rng(N + V)
    l = (g.standard_normal((N, V)) * 2).astype(np.float32)
    for kw in ({}, dict(min_p=0.05, temperature=0.7), dict(temperature=1.7)):
        check(l, u=g.random(N).astype(np.float32), **kw)


@pytest.mark.parametrize("V", [6, 5000, 151936])
@pytest.mark.parametrize("kw", [{}, dict(top_k=3), dict(top_k=300), dict(min_p=1e-10), dict(top_p=0.5), dict(temperature=0.0)])
def test_one_and_above_take_the_last_kept_token(V, kw):
    """u >= 1 is the last kept token in index order, however small its share (e^-24 of the heavy one's here)."""
    l = np.full((4, V), -4.0, np.float32)
    l[:, 1], l[:, 4], l[:, V - 2] = 20.0, 0.5, 0.25
    order = np.lexsort((np.arange(V), -l[0]))
    k = kw.get("top_k", V)
    last = 1 if "top_p" in kw or "temperature" in kw else int(order[:k].max()) if k < V else V - 1
    if "min_p" in kw:  # w >= 1e-10 is l > -3.03
        last = V - 2
    token, _ = sample(l, u=[1.0, 1.5, np.inf, 3e38], **kw)
    assert token.tolist() == [last] * 4
