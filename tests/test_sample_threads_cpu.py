"""The sampler's threads, without a GPU: csrc/sample.cuh run by tests/cta_emulator.h under schedules that let one warp
or CTA run as far ahead of the others as the barriers allow.  Whatever the schedule, the tokens are the
double-precision reference's."""
from __future__ import annotations

import shutil

import numpy as np
import pytest

import request_refs as refs
import sample_emulator as emu

NEG = -np.inf
ORDERS = sorted(emu.orders(1))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    return emu.build(str(tmp_path_factory.mktemp("sample")))


def check(lib, l, order, cl=1, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, u=0.5, fill=0xa5):
    l = np.atleast_2d(np.asarray(l, np.float32))
    token, prob = emu.sample(lib, l, temperature, top_k, top_p, min_p, u, cl=cl, order=emu.orders(cl)[order], fill=fill)
    at = lambda v, n: np.float32(np.broadcast_to(np.asarray(v, np.float64), (l.shape[0],))[n])
    for n in range(l.shape[0]):
        k = int(np.broadcast_to(np.asarray(top_k), (l.shape[0],))[n])
        rt, rp, _ = refs.sample_row(l[n], at(temperature, n), k, at(top_p, n), at(min_p, n), at(u, n))
        assert token[n] == rt, (n, token[n], rt)
        # one rounding to fp32, and the fixed-point total's V roundings of 2^-44 of the largest weight
        assert abs(prob[n] - rp) <= (2.0 ** -24 * 1.0001 + l.shape[1] * 2.0 ** -44) * rp + 2.0 ** -149, (n, prob[n], rp)


@pytest.mark.parametrize("order", ORDERS)
def test_fewer_live_tokens_than_top_k(lib, order):
    """A row masked down to a few tokens, and a cold one: fewer of the threads' maxima count than top_k asks for."""
    g = np.random.default_rng(1)
    l = (g.standard_normal((2, 2000)) * 2).astype(np.float32)
    l[0, 20:] = NEG
    check(lib, l, order, top_k=50, u=[0.3, 0.8], temperature=[1.0, 0.004])
    check(lib, l[0], order, top_k=50, top_p=0.6, min_p=0.01, u=0.9)


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("top_k", [20, 40, 50, 100, 128])
def test_two_sorts_in_turn(lib, order, top_k):
    """Top-k without top-p sorts twice with nothing between; the exchange buffer's halves follow on."""
    g = np.random.default_rng(2)
    l = (g.standard_normal((3, 3000)) * 2).astype(np.float32)
    check(lib, l, order, top_k=top_k, u=[0.1, 0.5, 0.9])
    check(lib, l, order, top_k=top_k, min_p=0.05, u=[0.2, 0.6, 0.95])
    check(lib, l, order, top_k=top_k, top_p=0.8, u=[0.2, 0.6, 0.95])


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("fill", [0, 0xa5, 0xff])
def test_weight_table_is_ready(lib, order, fill):
    """Rows without top-k and top-p use the weight table right after the first cluster barrier's wait."""
    g = np.random.default_rng(3)
    l = (g.standard_normal((3, 3000)) * 2).astype(np.float32)
    check(lib, l, order, u=[0.1, 0.5, 0.9], fill=fill)
    check(lib, l, order, min_p=0.05, temperature=0.7, u=[0.2, 0.6, 0.95], fill=fill)
    l[:, ::31] = np.inf
    check(lib, l, order, u=[0.1, 0.5, 0.9], fill=fill)


@pytest.mark.parametrize("order", sorted(emu.orders(2)))
@pytest.mark.parametrize("cl,V", [(2, 3001), (3, 4100), (2, 6)])
def test_no_access_to_a_cta_that_may_not_have_started(lib, order, cl, V):
    """Shared memory of another CTA is touched only behind a cluster barrier, and never once that CTA has ended."""
    g = np.random.default_rng(4)
    l = (g.standard_normal((2, V)) * 2).astype(np.float32)
    for kw in ({}, dict(temperature=0.0), dict(top_k=40), dict(top_p=0.9)):
        check(lib, l, order, cl=cl, u=[0.2, 0.85], **kw)
    check(lib, np.full((1, V), NEG), order, cl=cl)


@pytest.mark.parametrize("kw,last", [({}, 5), (dict(top_k=3), 4), (dict(top_k=5), 4), (dict(min_p=1e-10), 5),
                                     (dict(top_k=5, top_p=0.99999994), 1), (dict(top_p=0.5), 1), (dict(temperature=0.0), 1)])
def test_one_and_above_take_the_last_kept_token(lib, kw, last):
    """u >= 1 is the last kept token in index order, however small its share (e^-20 of the row here)."""
    l = np.array([[0.0, 20.0, 0.0, 0.0, 0.5, 0.0]], np.float32)
    for u in (1.0, 1.5, np.inf):
        token, prob = emu.sample(lib, l, u=u, **kw)
        assert token[0] == last, (u, token)
    token, _ = emu.sample(lib, l, u=np.nextafter(np.float32(1), np.float32(0)), **kw)
    assert token[0] == 1  # the largest number below 1 still falls into the heavy token
