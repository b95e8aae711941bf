"""GPU: calls of the per-request operators at the edges of what they allow: rows and adapters past 2^31 elements, and a
process whose first call is a captured one."""
from __future__ import annotations

import subprocess
import sys
import os

import numpy as np
import pytest

import request_refs as refs
from q8_test_utils import assert_within, dev, torch
from test_gpu_lora import bound

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def q8():
    import q8_block_quantized_02_b200 as m
    return m


def test_rows_of_logits_past_32_bits():
    t = torch()
    N, V, ld = 3, 5003, 2 ** 30 + 5  # the last row starts at element 2^31 + 10
    g = np.random.default_rng(1)
    l = (g.standard_normal((N, V)) * 2).astype(np.float32)
    big = t.empty(2 * ld + V, device="cuda")
    for n in range(N):
        big[n * ld:n * ld + V] = dev(l[n])
    u = np.array([0.2, 0.5, 0.8], np.float32)
    token, prob = t.full((N,), -9, dtype=t.int32, device="cuda"), t.zeros(N, device="cuda")
    for top_k, top_p in ((0, 1.0), (40, 1.0), (0, 0.9), (300, 0.8)):
        k, p = t.full((N,), top_k, dtype=t.int32, device="cuda"), t.full((N,), top_p, device="cuda")
        q8().q8_sample(big, None, k, p, None, dev(u), token, prob, N, V, ld)
        want = [refs.sample_row(l[n], 1.0, top_k, np.float32(top_p), 0.0, u[n])[0] for n in range(N)]
        assert token.tolist() == want, (top_k, top_p)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_adapters_past_32_bits(dtype):
    t = torch()
    m = q8()
    M, K, R, n = 300, 16384, 128, 1030  # A: 1030 x 2^21 elements, the last adapter's from 2^31 + 2^23 on
    td = t.float32 if dtype == "f32" else t.bfloat16
    A = t.empty(n, R, K, dtype=td, device="cuda")
    B = t.empty(n, M, R, dtype=td, device="cuda")
    g = np.random.default_rng(2)
    used = [0, 1024, n - 1]
    for a in used:
        A[a] = t.from_numpy((g.standard_normal((R, K)) / np.sqrt(K)).astype(np.float32)).to(td)
        B[a] = t.from_numpy((g.standard_normal((M, R)) * 0.2).astype(np.float32)).to(td)
    x = g.standard_normal((4, K)).astype(np.float32)
    rows = [n - 1, 0, 1024, n - 1]
    y = t.empty(4, M, device="cuda")
    m.q8_lora(dev(x), A, B, None, None, dev(np.array(rows, np.int32)), None, y, M, K, 4, n, R,
              m.Q8_F32 if dtype == "f32" else m.Q8_BF16)
    An, Bn = A[used].float().cpu().numpy(), B[used].float().cpu().numpy()
    want, mag = refs.lora(x, An, Bn, None, None, [used.index(a) for a in rows], None)
    assert_within(y.cpu().numpy(), want, bound(mag, want, K), dtype)


FIRST_CALL = """
import sys
import torch
sys.path.insert(0, {root!r})
import q8_block_quantized_02_b200 as q8
g = torch.Generator(device="cuda").manual_seed(1)
N, K, M, R, V = 5, 256, 300, 16, 9001
x, l = torch.randn(N, K, generator=g, device="cuda"), torch.randn(N, V, generator=g, device="cuda")
A, B = torch.randn(2, R, K, generator=g, device="cuda"), torch.randn(2, M, R, generator=g, device="cuda")
ad = torch.tensor([0, 1, -1, 1, 0], dtype=torch.int32, device="cuda")
u, p = torch.rand(N, generator=g, device="cuda"), torch.full((N,), 0.9, device="cuda")
y, tok, prob = torch.empty(N, M, device="cuda"), torch.empty(N, dtype=torch.int32, device="cuda"), torch.empty(N, device="cuda")
rl, idx, w = torch.randn(N, 32, generator=g, device="cuda"), torch.empty(N, 4, dtype=torch.int32, device="cuda"), torch.empty(N, 4, device="cuda")
torch.cuda.synchronize()
def step():
    q8.q8_lora(x, A, B, None, None, ad, None, y, M, K, N, 2, R, q8.Q8_F32)
    q8.q8_moe_route_grouped(rl, None, N, 32, 4, 4, 2, 2, q8.Q8_SCORE_SIGMOID, 1, 2.5, idx, w)
    q8.q8_sample(l, None, None, p, None, u, tok, prob, N, V, V)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
got = [v.clone() for v in (y, idx, w, tok, prob)]
step()
assert all(torch.equal(a, b) for a, b in zip(got, (y, idx, w, tok, prob)))
assert q8.q8_read_device_error() == (0, 0)
print("same")
"""


def test_the_first_call_of_a_process_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout + r.stderr
