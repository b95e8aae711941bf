"""GPU parity of q8_moe_route_grouped (softmax or sigmoid scores, selection
bias, groups, renormalised and scaled weights) against double precision:
experts are equal, weights within their one rounding."""
from __future__ import annotations

import numpy as np
import pytest

import q8gen
import request_refs as refs
from q8_test_utils import dev, torch

pytestmark = pytest.mark.gpu


def q8():
    import q8_block_quantized_02_b200 as m
    return m


def route(l, bias, k, G, keep, top, sigmoid, renorm, scale):
    t = torch()
    T, E = l.shape
    idx = t.full((T, k), -7, dtype=t.int32, device="cuda")
    w = t.full((T, k), float("nan"), device="cuda")
    q8().q8_moe_route_grouped(dev(l.astype(np.float32)), None if bias is None else dev(bias.astype(np.float32)), T, E,
                              k, G, keep, top, int(sigmoid), int(renorm), scale, idx, w)
    return idx.cpu().numpy(), w.cpu().numpy()


def check(l, bias, k, G, keep, top, sigmoid, renorm, scale):
    idx, w = route(l, bias, k, G, keep, top, sigmoid, renorm, scale)
    for t in range(l.shape[0]):
        ri, rw = refs.route_token(l[t], bias, k, G, keep, top, sigmoid, renorm, scale)
        assert np.array_equal(idx[t], ri), (t, idx[t], ri)
        # one rounding to fp32 (half a step, 2^-24 relative; 2^-150 below the smallest normal) of a double
        assert np.all(np.abs(w[t] - rw) <= 2.0 ** -24 * 1.0001 * np.abs(rw) + 2.0 ** -149), (t, w[t], rw)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k,G,keep,top", [(1, 1, 1, 1, 1, 1), (1, 60, 4, 1, 1, 1), (16, 256, 8, 8, 4, 2), (5, 33, 3, 3, 2, 1),
                                              (3, 256, 8, 32, 1, 2), (7, 160, 6, 5, 3, 2), (2, 64, 8, 32, 4, 2),
                                              (4, 31, 2, 31, 2, 1), (17, 254, 7, 2, 2, 1), (1031, 128, 8, 4, 2, 2)])
def test_route_matches_reference(sigmoid, with_bias, T, E, k, G, keep, top):
    g = np.random.default_rng(T * 1000 + E + G)
    l = (g.standard_normal((T, E)) * 2).astype(np.float32)
    bias = (g.standard_normal(E) * 0.1).astype(np.float32) if with_bias else None
    for renorm, scale in ((False, 1.0), (True, 2.5)):
        check(l, bias, k, G, keep, top, sigmoid, renorm, scale)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("G,keep,top", [(1, 1, 1), (4, 2, 2), (8, 3, 1)])
def test_ties_infinities_and_nan(sigmoid, G, keep, top):
    E, k = 64, 6
    g = np.random.default_rng(3)
    inf, nan = np.inf, np.nan
    rows = [np.zeros(E), np.full(E, -inf), np.full(E, nan), np.full(E, inf),
            np.where(np.arange(E) % 3 == 0, inf, 1.0), np.where(np.arange(E) < 60, -inf, 2.0),
            np.where(np.arange(E) == 63, 5.0, nan), g.integers(-2, 3, E).astype(float),
            np.where(np.arange(E) % 2 == 0, 200.0, -200.0), np.full(E, np.finfo(np.float32).min),
            np.full(E, -0.0), np.where(np.arange(E) % 2 == 0, -0.0, 0.0)]
    l = np.stack(rows).astype(np.float32)
    biases = [None, np.zeros(E), np.where(np.arange(E) < 16, -inf, 0.0), np.where(np.arange(E) == 40, inf, 0.0),
              np.where(np.arange(E) % 5 == 0, nan, 0.0), np.where(np.arange(E) == 41, inf, -inf)]
    for bias in biases:
        for renorm in (False, True):
            check(l, bias, k, G, keep, top, sigmoid, renorm, 1.5)


def test_agrees_with_q8_moe_route():
    t = torch()
    T, E, k = 16, 60, 4
    l = q8gen.logits(9, T, E)
    for renorm in (0, 1):
        idx, w = t.empty((T, k), dtype=t.int32, device="cuda"), t.empty((T, k), device="cuda")
        q8().q8_moe_route(dev(l), T, E, k, renorm, idx, w)
        gi, gw = route(l, None, k, 1, 1, 1, False, renorm, 1.0)
        assert np.array_equal(idx.cpu().numpy(), gi)
        # q8_moe_route works in fp32: about E terms of the softmax sum and a division or two
        assert np.all(np.abs(w.cpu().numpy() - gw) <= 40 * 2.0 ** -24 * gw)


def test_a_bias_moves_the_pick_but_not_the_weight():
    l = np.zeros((1, 8), np.float32)
    bias = np.zeros(8, np.float32)
    bias[6] = 1e-9  # far below fp32's step at 0.5: scores are compared in double
    idx, w = route(l, bias, 2, 1, 1, 1, True, False, 1.0)
    assert idx.tolist() == [[6, 0]] and w.tolist() == [[0.5, 0.5]]


def test_rows_past_the_batch_are_left_alone():
    t = torch()
    T, E, k = 5, 16, 3
    l = dev(np.random.default_rng(0).standard_normal((T + 3, E)).astype(np.float32))
    idx, w = t.full((T + 3, k), -9, dtype=t.int32, device="cuda"), t.full((T + 3, k), 9.0, device="cuda")
    q8().q8_moe_route_grouped(l, None, T, E, k, 2, 1, 1, 0, 0, 1.0, idx, w)
    assert (idx[T:] == -9).all() and (w[T:] == 9.0).all() and (idx[:T] >= 0).all()


def test_host_and_misaligned_pointers_are_refused():
    t = torch()
    m = q8()
    l, b = t.zeros(1, 8, device="cuda"), t.zeros(8, device="cuda")
    idx, w = t.zeros(1, 2, dtype=t.int32, device="cuda"), t.zeros(1, 2, device="cuda")
    for args, status in (((l.cpu(), b, idx, w), 4), ((l, b.cpu(), idx, w), 4), ((l, b, idx.cpu(), w), 4), ((l, b, idx, w.cpu()), 4),
                         ((l.data_ptr() + 2, b, idx, w), 3), ((l, b.data_ptr() + 1, idx, w), 3), ((l, b, idx.data_ptr() + 2, w), 3),
                         ((l, b, idx, w.data_ptr() + 2), 3)):
        with pytest.raises(m.Q8Error) as e:
            m.q8_moe_route_grouped(args[0], args[1], 1, 8, 2, 2, 1, 1, 0, 0, 1.0, args[2], args[3])
        assert e.value.status == status
