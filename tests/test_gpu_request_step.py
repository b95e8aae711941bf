"""One decode step of a batch of requests on the library's entry points as they
are used together: adapters beside a projection with the residual added,
grouped routing, the expert block, the head, the sampler.  Every stage is
checked against double precision on the values the stage before it gave, and
the step captured in a CUDA graph gives the same bits for new inputs."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
import q8gen
import request_refs as refs
from q8_test_utils import TOL_REL, assert_within, dev, pack, torch

pytestmark = pytest.mark.gpu

N, H, I, IS, E, K, G, V, LD, R = 6, 256, 96, 160, 16, 4, 4, 4099, 4104, 16


def q8():
    import q8_block_quantized_02_b200 as m
    return m


class Step:
    """Weights and buffers of the step; run() enqueues it."""

    def __init__(self):
        t = torch()
        m = q8()
        g = np.random.default_rng(1)
        self.g_o, self.g_r, self.g_v = (q8gen.q8_matrix(s, M, H)[0] for s, M in ((1, H), (2, E), (3, LD)))
        self.p_o, self.p_r, self.p_v = pack(self.g_o, H, H), pack(self.g_r, E, H), pack(self.g_v, LD, H)
        self.gu = np.concatenate([q8gen.q8_matrix(100 + e, 2 * I, H)[0] for e in range(E)])
        self.dn = np.concatenate([q8gen.q8_matrix(200 + e, H, I)[0] for e in range(E)])
        self.sgu, self.sdn = q8gen.q8_matrix(300, 2 * IS, H)[0], q8gen.q8_matrix(301, H, IS)[0]

        def stack(all_, n, M, Kk):
            one, b = m.q8_packed_bytes(M, Kk), M * (Kk // 32) * 34
            out = t.empty(n * one, dtype=t.uint8, device="cuda")
            for e in range(n):
                m.q8_pack_weights(dev(all_[e * b:(e + 1) * b]), M, Kk, out[e * one:(e + 1) * one])
            return out

        self.p_gu, self.p_dn = stack(self.gu, E, 2 * I, H), stack(self.dn, E, H, I)
        self.p_sgu, self.p_sdn = pack(self.sgu, 2 * IS, H), pack(self.sdn, H, IS)
        self.A = t.from_numpy((g.standard_normal((3, R, H)) * 0.05).astype(np.float32)).to(t.bfloat16).cuda()
        self.B = t.from_numpy((g.standard_normal((3, H, R)) * 0.2).astype(np.float32)).to(t.bfloat16).cuda()
        self.rank, self.scale = dev(np.array([16, 5, 9], np.int32)), dev(np.array([1.0, 0.5, 2.0], np.float32))
        self.bias = dev((g.standard_normal(E) * 0.05).astype(np.float32))
        f = lambda *s: t.empty(s, device="cuda")
        self.x, self.y, self.rl, self.w, self.z, self.h = f(N, H), f(N, H), f(N, E), f(N, K), f(N, H), f(N, H)
        self.logits, self.prob, self.u, self.temp, self.top_p = f(N, LD), f(N), f(N), f(N), f(N)
        i = lambda *s: t.empty(s, dtype=t.int32, device="cuda")
        self.adapter, self.idx, self.token, self.top_k = i(N), i(N, K), i(N), i(N)
        self.ws_bytes = m.q8_moe_workspace_bytes(N, E, K, H, I, IS)
        self.ws = t.empty(self.ws_bytes, dtype=t.uint8, device="cuda")
        m.q8_moe_workspace_init(self.ws, self.ws_bytes)

    def inputs(self, seed):
        t = torch()
        g = np.random.default_rng(seed)
        put = lambda d, v: d.copy_(t.from_numpy(np.asarray(v)))
        put(self.x, g.standard_normal((N, H)).astype(np.float32) * 0.2)
        put(self.adapter, g.integers(-1, 3, N).astype(np.int32))
        put(self.u, g.random(N).astype(np.float32))
        put(self.temp, g.choice([0.0, 0.7, 1.2], N).astype(np.float32))
        put(self.top_p, g.choice([0.8, 1.0], N).astype(np.float32))
        put(self.top_k, g.choice([0, 40], N).astype(np.int32))

    def run(self):
        t = torch()
        m = q8()
        m.q8_gemv_lora_split(self.p_o, self.x, self.A, self.B, self.rank, self.scale, self.adapter, self.x, self.y, H, H, N,
                             3, R, m.Q8_BF16)
        m.q8_gemv(self.p_r, self.y, self.rl, E, H, N)
        m.q8_moe_route_grouped(self.rl, self.bias, N, E, K, G, 2, 2, m.Q8_SCORE_SIGMOID, 1, 1.5, self.idx, self.w)
        m.q8_moe_gemv(self.p_gu, self.p_dn, self.p_sgu, self.p_sdn, self.idx, self.w, self.y, self.z, N, E, K, H, I, IS,
                      self.ws, self.ws_bytes)
        t.mul(self.z, 1e-3, out=self.h)
        m.q8_gemv(self.p_v, self.h, self.logits, LD, H, N)
        m.q8_sample(self.logits, self.temp, self.top_k, self.top_p, None, self.u, self.token, self.prob, N, V, LD)


def test_every_stage_of_the_step():
    s = Step()
    for seed in (5, 6):
        s.inputs(seed)
        s.run()
        c = {k: getattr(s, k).float().cpu().numpy() if getattr(s, k).dtype.is_floating_point else getattr(s, k).cpu().numpy()
             for k in ("x", "y", "rl", "w", "z", "h", "logits", "prob", "u", "temp", "top_p", "adapter", "idx", "token",
                       "top_k", "A", "B", "rank", "scale", "bias")}
        part, mag = refs.lora(c["x"], c["A"], c["B"], c["rank"], c["scale"], c["adapter"], c["x"])
        wx, wabs = oracle.gemv(s.g_o, c["x"], H, H)
        tol = (H / 128 + 64) * 2.0 ** -24 * mag + TOL_REL * wabs + 2.0 ** -23 * (np.abs(part) + np.abs(part + wx))
        assert_within(c["y"], part + wx, tol, "adapters beside the projection")
        for n in range(N):
            idx, w = refs.route_token(c["rl"][n], c["bias"], K, G, 2, 2, True, True, 1.5)
            assert np.array_equal(c["idx"][n], idx)
            assert np.all(np.abs(c["w"][n] - w) <= 2.0 ** -24 * 1.0001 * np.abs(w))
        y_ref, bound, _ = oracle.moe(s.gu, s.dn, s.sgu, s.sdn, c["idx"], c["w"].astype(np.float64), c["y"], H, I, IS)
        assert np.all(np.abs(c["z"] - y_ref) <= bound)
        l_ref, l_abs = oracle.gemv(s.g_v, c["h"], LD, H)
        assert_within(c["logits"], l_ref, TOL_REL * l_abs, "head")
        for n in range(N):
            token, p, _ = refs.sample_row(c["logits"][n, :V], c["temp"][n], int(c["top_k"][n]), c["top_p"][n], 0.0, c["u"][n])
            assert c["token"][n] == token and abs(c["prob"][n] - p) <= (2.0 ** -24 * 1.0001 + V * 2.0 ** -44) * p
    assert q8().q8_read_device_error() == (0, 0)


def test_the_captured_step_follows_new_inputs():
    t = torch()
    s = Step()
    s.inputs(7)
    s.run()
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    side = t.cuda.Stream()
    with t.cuda.graph(graph, stream=side):
        s.run()
    outs = ("y", "rl", "idx", "w", "z", "logits", "token", "prob")
    for seed in (8, 9, 10):
        s.inputs(seed)
        graph.replay()
        t.cuda.synchronize()
        got = {k: getattr(s, k).clone() for k in outs}
        s.run()
        t.cuda.synchronize()
        for k in outs:
            assert t.equal(got[k], getattr(s, k)), k


def test_two_streams_at_once():
    """The operators keep nothing between calls, so calls on two streams do not touch each other's results."""
    t = torch()
    m = q8()
    g = np.random.default_rng(3)
    A, B = (t.from_numpy(g.standard_normal(sh).astype(np.float32)).cuda() for sh in ((4, 32, 2048), (4, 1000, 32)))
    adapter = [dev(g.integers(-1, 4, 8).astype(np.int32)) for _ in range(2)]
    x = [t.from_numpy(g.standard_normal((8, 2048)).astype(np.float32)).cuda() for _ in range(2)]
    l = [t.from_numpy((g.standard_normal((8, 30000)) * 2).astype(np.float32)).cuda() for _ in range(2)]
    u = [t.from_numpy(g.random(8).astype(np.float32)).cuda() for _ in range(2)]
    p = t.full((8,), 0.9, device="cuda")

    def go(i, y, tok, idx, w, stream):
        for _ in range(20):
            m.q8_lora(x[i], A, B, None, None, adapter[i], None, y, 1000, 2048, 8, 4, 32, m.Q8_F32, stream=stream)
            m.q8_sample(l[i], None, None, p, None, u[i], tok, None, 8, 30000, 30000, stream=stream)
            m.q8_moe_route_grouped(l[i], None, 8, 256, 8, 8, 4, 2, 1, 1, 1.0, idx, w, stream=stream)

    def buffers():
        return (t.empty(8, 1000, device="cuda"), t.empty(8, dtype=t.int32, device="cuda"),
                t.empty(8, 8, dtype=t.int32, device="cuda"), t.empty(8, 8, device="cuda"))

    want = []
    for i in range(2):
        want.append(buffers())
        go(i, *want[i], None)
    t.cuda.synchronize()
    streams, got = [t.cuda.Stream() for _ in range(2)], [buffers() for _ in range(2)]
    for i in range(2):
        go(i, *got[i], streams[i])
    t.cuda.synchronize()
    for i in range(2):
        assert all(t.equal(a, b) for a, b in zip(want[i], got[i]))
