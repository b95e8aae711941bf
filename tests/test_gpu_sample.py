"""GPU parity of q8_sample (temperature, top-k, top-p and min-p sampling from
given uniform numbers) against double precision: tokens are equal, the
probability is within its roundings."""
from __future__ import annotations

import numpy as np
import pytest

import request_refs as refs
from q8_test_utils import dev, torch

pytestmark = pytest.mark.gpu

NEG, NAN, INF = -np.inf, np.nan, np.inf


def q8():
    import q8_block_quantized_02_b200 as m
    return m


def sample(l, temperature=None, top_k=None, top_p=None, min_p=None, u=None, V=None, ld=None, logits_dev=None):
    """q8_sample on the rows l [N][ld]; scalars are given to every row."""
    t = torch()
    N = l.shape[0]
    ld = l.shape[1] if ld is None else ld
    V = ld if V is None else V

    def row(v, dt):
        return None if v is None else dev(np.broadcast_to(np.asarray(v, dt), (N,)))

    token = t.full((N,), -99, dtype=t.int32, device="cuda")
    prob = t.full((N,), float("nan"), device="cuda")
    q8().q8_sample(dev(l.astype(np.float32)) if logits_dev is None else logits_dev, row(temperature, np.float32),
                   row(top_k, np.int32), row(top_p, np.float32), row(min_p, np.float32),
                   row(0.0 if u is None else u, np.float32), token, prob, N, V, ld)
    return token.cpu().numpy(), prob.cpu().numpy()


def check(l, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, u=0.5, V=None):
    l = np.atleast_2d(np.asarray(l, np.float32))
    N = l.shape[0]
    V = l.shape[1] if V is None else V
    token, prob = sample(l, temperature, top_k, top_p, min_p, u, V=V)
    at = lambda v, n: np.float32(np.broadcast_to(np.asarray(v, np.float64), (N,))[n])
    for n in range(N):
        k = int(np.broadcast_to(np.asarray(top_k), (N,))[n])
        rt, rp, _ = refs.sample_row(l[n, :V], at(temperature, n), k, at(top_p, n), at(min_p, n), at(u, n))
        assert token[n] == rt, (n, token[n], rt)
        # one rounding to fp32, and the fixed-point total's V roundings of 2^-44 of the largest weight
        assert abs(prob[n] - rp) <= (2.0 ** -24 * 1.0001 + V * 2.0 ** -44) * rp + 2.0 ** -149, (n, prob[n], rp)


FILTERS = {
    "plain": {}, "cold": dict(temperature=0.3), "hot": dict(temperature=4.0), "top_k": dict(top_k=40), "top_1": dict(top_k=1),
    "top_p": dict(top_p=0.9), "nucleus_hot": dict(top_p=0.97, temperature=2.0), "min_p": dict(min_p=0.05),
    "all": dict(temperature=0.8, top_k=50, top_p=0.95, min_p=0.02), "k_and_p": dict(top_k=1000, top_p=0.5),
    "tiny_p": dict(top_p=1e-6), "near_1": dict(top_p=0.9999999), "wide_k": dict(top_k=20000, top_p=0.999),
}


@pytest.mark.parametrize("name", sorted(FILTERS))
@pytest.mark.parametrize("N,V,ld", [(1, 1, 1), (3, 2, 2), (2, 31, 37), (5, 1000, 1000), (1, 151936, 151936), (16, 32003, 32064),
                                    (4, 152064, 152064), (40, 5001, 5001)])
def test_sample_matches_reference(name, N, V, ld):
    g = np.random.default_rng(N * 7 + V)
    l = (g.standard_normal((N, ld)) * 2).astype(np.float32)
    likely = g.integers(0, V, (N, min(V, 12)))
    np.put_along_axis(l, likely, 5 + 6 * g.random(likely.shape).astype(np.float32), 1)
    l[:, V:] = 1000.0  # padding of the vocabulary is not looked at
    check(l, **FILTERS[name], u=g.random(N).astype(np.float32), V=V)


@pytest.mark.parametrize("V", [1, 3, 64, 4097, 200000])
@pytest.mark.parametrize("kw", [{}, dict(top_p=0.5), dict(top_k=7), dict(top_k=7, top_p=0.6), dict(min_p=1.0), dict(top_p=0.3, min_p=0.9)])
def test_equal_logits(V, kw):
    """Nothing but ties: the filters cut inside one value, lowest indices stay."""
    u = np.array([0.0, 0.25, 0.5, 0.75, 0.999], np.float32)
    for value in (0.0, -3.25, 1e30):
        check(np.full((5, V), value), u=u, **kw)


@pytest.mark.parametrize("kw", [dict(top_k=100), dict(top_p=0.7), dict(top_k=3000, top_p=0.9), dict(min_p=0.3), {}])
def test_few_distinct_values(kw):
    """Coarse logits: every threshold lies inside a run of equals spread over the row."""
    g = np.random.default_rng(4)
    l = g.integers(-6, 5, (8, 30011)).astype(np.float32) * 0.5
    check(l, u=g.random(8).astype(np.float32), **kw)


def test_logits_closer_than_the_first_bins():
    """Large magnitudes and differences of single steps of fp32: the rounds go down to the key."""
    g = np.random.default_rng(5)
    base = np.float32(1000.0)
    l = (base + g.integers(0, 4000, (4, 20000)).astype(np.float32) * np.spacing(base)).astype(np.float32)
    for kw in (dict(top_k=777), dict(top_p=0.37), dict(top_k=5000, top_p=0.5)):
        check(l, u=g.random(4).astype(np.float32), **kw)
    tiny = (g.random((4, 9000)).astype(np.float32) - np.float32(0.5)) * np.float32(1e-30)
    tiny[:, 17] = 0.0
    for kw in (dict(top_k=1234), dict(top_p=0.61)):
        check(tiny, u=g.random(4).astype(np.float32), **kw)


def test_threshold_around_zero_logits():
    g = np.random.default_rng(6)
    l = (g.standard_normal((6, 50000)) * 1.0).astype(np.float32)
    l[:, 9] = 4.0
    mid = [int((row > 0).sum()) for row in l]
    check(l, top_k=np.array([mid[0], mid[1] + 1, mid[2] - 1, mid[3] + 30, mid[4] - 30, 25000]), u=g.random(6).astype(np.float32))
    l[1::2, 100:140] = -0.0
    l[:, 200:240] = 0.0
    check(l, top_k=np.array(mid) + 20, u=g.random(6).astype(np.float32))


@pytest.mark.parametrize("kw", [dict(top_k=200), dict(top_k=256, top_p=0.6), dict(top_k=257), dict(top_k=200, min_p=0.5)])
def test_large_logits_crowded_in_one_place(kw):
    """The largest logits side by side (few threads hold them), or at a stride (one thread holds most of them)."""
    g = np.random.default_rng(13)
    V = 100000
    l = g.standard_normal((4, V)).astype(np.float32)
    l[0, 500:3500] = 8 + np.arange(3000, dtype=np.float32) * 1e-3
    l[1, 90000:90600] = 9 - np.arange(600, dtype=np.float32) * 1e-4
    l[2, ::2048] = 7 + g.random(l[2, ::2048].size).astype(np.float32)
    l[3, 3::512] = 7.0
    check(l, u=g.random(4).astype(np.float32), **kw)


@pytest.mark.parametrize("top_p", [0.2, 0.5, 0.8, 0.97, 0.9995])
def test_mass_in_few_tokens(top_p):
    """Peaked rows, where the estimate of top-p's bin is at its coarsest: one, two, ten and a hundred heavy tokens."""
    g = np.random.default_rng(14)
    l = g.standard_normal((8, 60000)).astype(np.float32)
    for n, heavy in enumerate((1, 2, 2, 10, 10, 100, 100, 1000)):
        l[n, g.choice(60000, heavy, replace=False)] = 14 + (n % 2) * g.random(heavy).astype(np.float32) * 3
    check(l, top_p=top_p, u=g.random(8).astype(np.float32))
    check(l, top_p=top_p, temperature=2.5, min_p=0.01, u=g.random(8).astype(np.float32))


@pytest.mark.parametrize("V", [1024, 1025, 20064, 20065, 32768, 32769])
@pytest.mark.parametrize("N", [1, 20, 75, 149, 161])
def test_cluster_sizes(V, N):
    """Around the sizes and batches at which a row takes another number of CTAs."""
    g = np.random.default_rng(V + N)
    l = np.repeat((g.standard_normal((1, V)) * 1.5).astype(np.float32), N, 0)
    u = g.random(N).astype(np.float32)
    token, prob = sample(l, top_p=0.9, u=u)
    for n in sorted({0, N // 2, N - 1}):
        rt, rp, _ = refs.sample_row(l[0], top_p=np.float32(0.9), u=u[n])
        assert token[n] == rt and abs(prob[n] - rp) <= (2.0 ** -24 * 1.0001 + V * 2.0 ** -44) * rp


def test_masks_infinities_and_nan():
    g = np.random.default_rng(7)
    V = 5003
    bulk = g.standard_normal(V)
    low = np.finfo(np.float32).min
    rows = [np.full(V, NEG), np.full(V, NAN), np.full(V, low), np.where(np.arange(V) == V - 1, 1.0, NEG),
            np.where(np.arange(V) % 2 == 0, NEG, bulk), np.where(np.arange(V) % 2 == 0, low, bulk),
            np.where(np.arange(V) % 97 == 5, INF, bulk), np.where(np.arange(V) % 3 == 0, NAN, bulk),
            np.where(np.arange(V) == 0, np.finfo(np.float32).max, low), np.full(V, INF), np.where(np.arange(V) < 4000, NEG, 0.0)]
    l = np.stack(rows).astype(np.float32)
    u = np.linspace(0, 0.99, len(rows)).astype(np.float32)
    for kw in ({}, dict(top_k=5), dict(top_p=0.4), dict(min_p=0.2), dict(top_k=2000, top_p=0.8, min_p=1e-3), dict(temperature=0.0),
               dict(temperature=1e30, top_p=0.5), dict(temperature=1e-30), dict(top_k=V), dict(top_k=-4, top_p=2.0, min_p=-1.0)):
        check(l, u=u, **kw)


def test_parameters_at_their_ends():
    g = np.random.default_rng(8)
    V = 3001
    l = (g.standard_normal((1, V)) * 2).astype(np.float32)
    for u in (0.0, -1.0, NAN, 0.99999994, 1.0, 7.0, INF, NEG, 1e-45):
        check(l, u=u)
        check(l, u=u, top_k=20, top_p=0.8)
    for temperature in (0.0, -1.0, NAN, NEG):
        token, prob = sample(l, temperature=temperature, u=0.9)
        assert token[0] == int(np.argmax(l[0])) and prob[0] == 1.0
    for temperature in (1e-45, 1e-38, 1e-3, 1e3, 3e38, INF):
        check(l, temperature=temperature, u=0.63)
        check(l, temperature=temperature, u=0.63, top_k=500)
    for kw in (dict(top_p=0.0), dict(top_p=-1.0), dict(min_p=1.0), dict(min_p=50.0), dict(top_k=1), dict(top_p=1e-45)):
        token, prob = sample(l, u=0.9, **kw)
        assert token[0] == int(np.argmax(l[0])) and prob[0] == 1.0, kw
    for kw in (dict(top_p=NAN), dict(top_p=1.0), dict(min_p=NAN), dict(min_p=0.0), dict(top_k=0), dict(top_k=V), dict(top_k=2 ** 31 - 1),
               dict(top_k=-2 ** 31)):
        want, _ = sample(l, u=0.9)
        assert sample(l, u=0.9, **kw)[0][0] == want[0], kw


def test_greedy_takes_the_lowest_of_equal_maxima():
    l = np.zeros((3, 70000), np.float32)
    l[0, [69999, 40000, 123]] = 2.0
    l[1, [5, 6]] = -0.0
    token, prob = sample(l, temperature=[0.0, 0.0, 0.0])
    assert token.tolist() == [123, 0, 0] and prob.tolist() == [1.0, 1.0, 1.0]


def test_largest_vocabulary_and_offsets():
    """V at its limit, a row stride beyond V, rows that start off any 16-byte boundary."""
    t = torch()
    g = np.random.default_rng(9)
    V, ld, N = 524288, 524291, 3
    l = (g.standard_normal((N, ld)) * 1.5).astype(np.float32)
    u = g.random(N).astype(np.float32)
    check(l, u=u, V=V, top_p=0.9)
    check(l, u=u, V=V, top_k=9000)
    flat = t.zeros(N * ld + 1, device="cuda")
    flat[1:] = t.from_numpy(l.reshape(-1))
    a, _ = sample(l, top_p=0.9, u=u, V=V)
    b, _ = sample(l, top_p=0.9, u=u, V=V, logits_dev=flat[1:])
    assert np.array_equal(a, b)


def test_many_rows_with_their_own_parameters():
    g = np.random.default_rng(10)
    N, V = 300, 2500
    l = (g.standard_normal((N, V)) * 2).astype(np.float32)
    l[g.random((N, V)) < 0.3] = NEG
    check(l, temperature=g.choice([0.0, 0.5, 1.0, 1.7], N).astype(np.float32), top_k=g.choice([0, 1, 20, 700], N),
          top_p=g.choice([0.3, 0.9, 1.0], N).astype(np.float32), min_p=g.choice([0.0, 0.01, 0.5], N).astype(np.float32),
          u=g.random(N).astype(np.float32))


def test_a_row_does_not_depend_on_its_batch():
    """The cluster size follows the batch; the fixed-point sums do not."""
    g = np.random.default_rng(11)
    l = (g.standard_normal((1, 100003)) * 1.2).astype(np.float32)
    want = sample(l, top_p=0.95, u=0.77)
    for N in (2, 9, 33, 150):
        token, prob = sample(np.repeat(l, N, 0), top_p=0.95, u=0.77)
        assert np.all(token == want[0][0]) and np.all(prob == want[1][0])


def test_draws_follow_the_distribution():
    """Every u of an even grid: token i comes out as often as its probability says, to one grid step."""
    l = np.log(np.array([[0.5, 0.125, 0.25, 0.125]], np.float32))
    n = 1024
    token, prob = sample(np.repeat(l, n, 0), u=(np.arange(n) + 0.5).astype(np.float32) / n)
    counts = np.bincount(token, minlength=4)
    assert np.all(np.abs(counts - np.array([512, 128, 256, 128])) <= 1)
    assert np.allclose(prob, np.exp(l[0])[token], rtol=2.0 ** -22)


def test_outputs_past_the_rows_are_left_alone_and_prob_is_optional():
    t = torch()
    l = dev(np.random.default_rng(1).standard_normal((4, 333)).astype(np.float32))
    token, prob = t.full((6,), -5, dtype=t.int32, device="cuda"), t.full((6,), -5.0, device="cuda")
    u = t.full((4,), 0.3, device="cuda")
    q8().q8_sample(l, None, None, None, None, u, token, prob, 4, 333, 333)
    assert (token[4:] == -5).all() and (prob[4:] == -5.0).all() and (token[:4] >= 0).all()
    again = t.full((6,), -5, dtype=t.int32, device="cuda")
    q8().q8_sample(l, None, None, None, None, u, again, None, 4, 333, 333)
    assert t.equal(token, again)


def test_captured_replays_and_another_stream():
    t = torch()
    N, V = 5, 40000
    g = np.random.default_rng(12)
    l, u = dev((g.standard_normal((N, V)) * 2).astype(np.float32)), dev(g.random(N).astype(np.float32))
    top_p = t.full((N,), 0.9, device="cuda")
    token, prob = t.empty(N, dtype=t.int32, device="cuda"), t.empty(N, device="cuda")
    args = (l, None, None, top_p, None, u, token, prob, N, V, V)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        q8().q8_sample(*args)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=side):
        q8().q8_sample(*args)
    for k in range(3):
        u.copy_(t.from_numpy(g.random(N).astype(np.float32)))
        l.copy_(l.roll(17 + k, 1))
        graph.replay()
        t.cuda.synchronize()
        got = (token.clone(), prob.clone())
        q8().q8_sample(*args)
        assert t.equal(got[0], token) and t.equal(got[1], prob)


def test_host_and_misaligned_pointers_are_refused():
    t = torch()
    m = q8()
    N, V = 2, 100
    l, u, p = t.zeros(N, V, device="cuda"), t.zeros(N, device="cuda"), t.zeros(N, device="cuda")
    tok = t.zeros(N, dtype=t.int32, device="cuda")
    good = [l, p, tok, p, p, u, tok, p]
    for i in range(8):
        for wrong, status in ((good[i].cpu(), 4), (good[i].data_ptr() + 2, 3)):
            with pytest.raises(m.Q8Error) as e:
                m.q8_sample(*(good[:i] + [wrong] + good[i + 1:]), N, V, V)
            assert e.value.status == status, (i, e.value.status)
