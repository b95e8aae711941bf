"""GPU parity of q8_lora, q8_gemv_lora and q8_gemv_lora_split (low-rank adapters
of many requests, alone and beside a shared Q8_0 projection) against double
precision, through the C ABI."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
import request_refs as refs
from q8_test_utils import TOL_REL, assert_within, dev, matrix, pack, torch

pytestmark = pytest.mark.gpu

H24 = 2.0 ** -24  # half a step of fp32, relative


def q8():
    import q8_block_quantized_02_b200 as m
    return m


def tdtype(name):
    t = torch()
    return {"f32": t.float32, "f16": t.float16, "bf16": t.bfloat16}[name]


def code(name):
    return {"f32": q8().Q8_F32, "f16": q8().Q8_F16, "bf16": q8().Q8_BF16}[name]


def bank_of(seed, n, R, M, K, dtype):
    """Adapters in `dtype` on the device, and their values in numpy."""
    t = torch()
    g = np.random.default_rng(seed)
    A = t.from_numpy((g.standard_normal((n, R, K)) / np.sqrt(K)).astype(np.float32)).to(tdtype(dtype))
    B = t.from_numpy((g.standard_normal((n, M, R)) * 0.2).astype(np.float32)).to(tdtype(dtype))
    scale = (0.5 + g.random(n)).astype(np.float32)
    return A, B, scale, A.float().numpy(), B.float().numpy()


def bound(mag, y, K, roundings=1):
    """The header's fp32 bound on the adapters' part, plus a rounding of the stored value each time it is stored.
    K / 128: a lane's chain of fused multiply-adds, K split over 32 lanes and at least 4 CTAs; the rest: warp, warps' and
    CTAs' sums of u, the scale, 8 products and 4 steps of a row of B."""
    return (K / 128 + 64) * H24 * mag + roundings * 1.01 * H24 * np.abs(y)


def run(x, A, B, rank, scale, adapter, residual, M, K, dtype, R=None, base=None, packed=None, in_place=False, stream=None):
    t = torch()
    N = x.shape[0]
    res = None if residual is None else dev(residual)
    y = res if in_place else t.full((N, M), float("nan"), dtype=t.float32, device="cuda")
    i32 = lambda v: None if v is None else dev(np.asarray(v, np.int32))
    args = (dev(x), A, B, i32(rank), None if scale is None else dev(scale), i32(adapter), res, y, M, K, N, A.shape[0],
            A.shape[1] if R is None else R, code(dtype))
    if base is None:
        q8().q8_lora(*args, stream=stream)
    else:
        (q8().q8_gemv_lora_split if base == "split" else q8().q8_gemv_lora)(packed, *args, stream=stream)
    return y.cpu().numpy()


# (M, K, N, R, adapters of the rows): one token to sixteen, bare rows, one adapter for all, more than four tokens of one
LAYOUTS = {
    "one": [2], "bare": [-1], "pair": [0, 0], "mixed": [1, -1, 0, 1, -5, 2],
    "five_of_one": [1, 1, 1, 1, 1], "nine": [0, 1, 0, 0, 2, 0, 0, -1, 0],
    "shared": [2] * 16, "distinct": list(range(16)), "half": [0, 3] * 8, "all_bare": [-1] * 16,
}


@pytest.mark.parametrize("layout", sorted(LAYOUTS))
@pytest.mark.parametrize("M,K,R,dtype", [(1, 32, 8, "f32"), (203, 1408, 16, "f16"), (896, 896, 24, "bf16"),
                                         (1153, 4864, 40, "bf16"), (8, 18944, 128, "f16"), (3584, 64, 64, "f32")])
def test_lora_matches_reference(layout, M, K, R, dtype):
    adapter = LAYOUTS[layout]
    N, n = len(adapter), max(3, max(adapter) + 1)
    g = np.random.default_rng(M + 7 * K + N)
    A, B, scale, An, Bn = bank_of(M + K, n, R, M, K, dtype)
    x = g.standard_normal((N, K)).astype(np.float32)
    residual = g.standard_normal((N, M)).astype(np.float32) if N % 2 else None
    rank = g.integers(0, R + 1, n) if N % 3 else None
    y_ref, mag = refs.lora(x, An, Bn, rank, scale, adapter, residual)
    y = run(x, A.cuda(), B.cuda(), rank, scale, adapter, residual, M, K, dtype)
    assert_within(y, y_ref, bound(mag, y_ref, K), f"{layout} {M}x{K} R={R} {dtype}")
    for i, a in enumerate(adapter):  # rows without an adapter are the residual's bits
        if a < 0:
            assert np.array_equal(y[i], np.zeros(M, np.float32) if residual is None else residual[i])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_values_past_the_rank_are_not_used(dtype):
    M, K, R, n = 300, 352, 32, 4
    A, B, scale, An, Bn = bank_of(5, n, R, M, K, dtype)
    rank = [0, 1, 13, 32]
    for a, r in enumerate(rank):
        A[a, r:], B[a, :, r:] = float("nan"), float("inf")
    x = np.random.default_rng(6).standard_normal((4, K)).astype(np.float32)
    y_ref, mag = refs.lora(x, An, Bn, rank, scale, [3, 2, 1, 0], None)
    y = run(x, A.cuda(), B.cuda(), rank, scale, [3, 2, 1, 0], None, M, K, dtype)
    assert_within(y, y_ref, bound(mag, y_ref, K), dtype)
    assert np.array_equal(y[3], np.zeros(M, np.float32))  # rank 0


def test_outside_ranks_are_clamped_and_null_means_full():
    M, K, R = 64, 96, 16
    A, B, scale, An, Bn = bank_of(8, 2, R, M, K, "bf16")
    x = np.random.default_rng(9).standard_normal((2, K)).astype(np.float32)
    full = run(x, A.cuda(), B.cuda(), None, None, [0, 1], None, M, K, "bf16")
    y_ref, mag = refs.lora(x, An, Bn, None, None, [0, 1], None)
    assert_within(full, y_ref, bound(mag, y_ref, K), "null rank and scale")
    y = run(x, A.cuda(), B.cuda(), [10 ** 6, -3], None, [0, 1], None, M, K, "bf16")
    assert np.array_equal(y[0], full[0]) and np.array_equal(y[1], np.zeros(M, np.float32))


def test_adapter_past_the_bank_is_reported_and_left_out():
    M, K, R = 70, 64, 8
    A, B, scale, An, Bn = bank_of(10, 2, R, M, K, "f16")
    x = np.random.default_rng(11).standard_normal((3, K)).astype(np.float32)
    res = np.random.default_rng(12).standard_normal((3, M)).astype(np.float32)
    q8().q8_read_device_error()
    y = run(x, A.cuda(), B.cuda(), None, scale, [0, 2, 2 ** 31 - 1], res, M, K, "f16")
    st, word = q8().q8_read_device_error()
    assert st != 0 and word == 16
    y_ref, mag = refs.lora(x, An, Bn, None, scale, [0, -1, -1], res)
    assert_within(y, y_ref, bound(mag, y_ref, K), "rows with a bad index")
    assert np.array_equal(y[1:], res[1:])


@pytest.mark.parametrize("base", ["exact", "split"])
@pytest.mark.parametrize("M,K,N,R,dtype", [(896, 4864, 1, 16, "bf16"), (1152, 896, 8, 8, "f16"), (203, 1408, 5, 24, "f32"),
                                           (3584, 18944, 4, 64, "bf16"), (3584, 3584, 16, 32, "bf16"), (13, 32, 3, 8, "f16"),
                                           (4736, 896, 2, 8, "bf16")])
@pytest.mark.parametrize("in_place", [False, True])
def test_gemv_lora_matches_reference(base, M, K, N, R, dtype, in_place):
    gguf, x = matrix(31 * M + K + N, M, K, N)
    A, B, scale, An, Bn = bank_of(M + N, 3, R, M, K, dtype)
    g = np.random.default_rng(K + N)
    adapter = g.integers(-1, 3, N)
    rank = g.integers(1, R + 1, 3)
    residual = g.standard_normal((N, M)).astype(np.float32) if in_place or N % 2 else None
    part, mag = refs.lora(x, An, Bn, rank, scale, adapter, residual)
    wx, wabs = oracle.gemv(gguf, x, M, K, threads=oracle.max_threads())
    y = run(x, A.cuda(), B.cuda(), rank, scale, adapter, residual, M, K, dtype, base=base, packed=pack(gguf, M, K),
            in_place=in_place)
    y_ref = part + wx
    assert_within(y, y_ref, bound(mag, part, K) + TOL_REL * wabs + 1.01 * H24 * np.abs(y_ref), f"{base} {M}x{K} N={N}")


def test_rows_without_adapters_have_the_projections_bits():
    t = torch()
    M, K, N = 1152, 896, 4
    gguf, x = matrix(77, M, K, N)
    p = pack(gguf, M, K)
    res = np.random.default_rng(1).standard_normal((N, M)).astype(np.float32)
    A, B, scale, *_ = bank_of(3, 2, 8, M, K, "bf16")
    y = run(x, A.cuda(), B.cuda(), None, scale, [-1] * N, res, M, K, "bf16", base="exact", packed=p)
    want = t.empty((N, M), device="cuda")
    q8().q8_gemv_residual(p, dev(x), dev(res), want, M, K, N)
    assert np.array_equal(y, want.cpu().numpy())


def test_equal_rows_get_equal_bits_wherever_they_stand():
    """The same request at other places of other batches: its adapter part does not depend on its neighbours."""
    M, K, R = 500, 2048, 48
    A, B, scale, *_ = bank_of(15, 3, R, M, K, "bf16")
    A, B = A.cuda(), B.cuda()
    x = np.random.default_rng(16).standard_normal((1, K)).astype(np.float32)
    nine = np.repeat(x, 9, 0)
    y = run(nine, A, B, None, scale, [1] * 9, None, M, K, "bf16")
    assert all(np.array_equal(y[0], y[i]) for i in range(9))
    z = run(nine, A, B, None, scale, [0, 1, 2, 1, -1, 1, 1, 1, 1], None, M, K, "bf16")
    for i in (1, 3, 5, 6, 7, 8):
        assert np.array_equal(z[i], y[0])


def test_outputs_past_the_batch_are_left_alone():
    t = torch()
    M, K, R, N = 33, 64, 8, 3
    A, B, scale, An, Bn = bank_of(20, 2, R, M, K, "f32")
    x = np.random.default_rng(21).standard_normal((N, K)).astype(np.float32)
    y = t.full((N + 2, M), 7.0, device="cuda")
    q8().q8_lora(dev(x), A.cuda(), B.cuda(), None, None, dev(np.array([0, 1, -1], np.int32)), None, y, M, K, N, 2, R,
                 q8().Q8_F32)
    assert np.array_equal(y[N:].cpu().numpy(), np.full((2, M), 7.0, np.float32))


def test_captured_replays_follow_new_inputs_on_another_stream():
    """A captured call replayed with other activations and other adapters per row gives what a direct call gives."""
    t = torch()
    M, K, N, R = 896, 896, 6, 16
    gguf, x = matrix(5, M, K, N)
    p = pack(gguf, M, K)
    A, B, scale, *_ = bank_of(6, 4, R, M, K, "bf16")
    A, B, sc = A.cuda(), B.cuda(), dev(scale)
    xd, ad = dev(x), dev(np.array([0, 1, 2, 3, -1, 0], np.int32))
    y = t.empty((N, M), device="cuda")
    args = (p, xd, A, B, None, sc, ad, None, y, M, K, N, 4, R, q8().Q8_BF16)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        q8().q8_gemv_lora_split(*args)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=side):
        q8().q8_gemv_lora_split(*args)
    for k, rows in enumerate(([3, 3, 3, 3, 3, 3], [-1, 0, -1, 1, 2, 2])):
        xd.copy_(t.from_numpy(np.roll(x, k + 1, 1).copy()))
        ad.copy_(t.tensor(rows, dtype=t.int32))
        graph.replay()
        t.cuda.synchronize()
        got = y.clone()
        q8().q8_gemv_lora_split(*args)
        assert t.equal(got, y)
    assert q8().q8_read_device_error() == (0, 0)


def test_long_reductions_and_many_rows():
    """K beyond what a cluster stages of x at once, and M beyond what its warps gather at once."""
    for M, K, R, dtype in ((5, 70016, 16, "bf16"), (40007, 96, 8, "f16"), (20011, 128, 128, "f32")):
        A, B, scale, An, Bn = bank_of(M, 2, R, M, K, dtype)
        g = np.random.default_rng(K)
        x = g.standard_normal((5, K)).astype(np.float32)
        res = g.standard_normal((5, M)).astype(np.float32)
        adapter = [0, 1, 0, 0, -1]
        y_ref, mag = refs.lora(x, An, Bn, [R, R - 3], scale, adapter, res)
        y = run(x, A.cuda(), B.cuda(), [R, R - 3], scale, adapter, res, M, K, dtype, in_place=M > 1000)
        assert_within(y, y_ref, bound(mag, y_ref, K), f"{M}x{K} R={R}")


def test_nan_and_infinite_activations_stay_in_their_row():
    M, K, R = 100, 256, 16
    A, B, scale, An, Bn = bank_of(40, 2, R, M, K, "bf16")
    x = np.random.default_rng(41).standard_normal((5, K)).astype(np.float32)
    x[1, 7], x[3, 9] = np.nan, np.inf
    y = run(x, A.cuda(), B.cuda(), None, scale, [0, 0, 0, 0, 1], None, M, K, "bf16")
    assert np.all(np.isnan(y[1])) and not np.any(np.isfinite(y[3]))
    y_ref, mag = refs.lora(x[[0, 2, 4]], An, Bn, None, scale, [0, 0, 1], None)
    assert_within(y[[0, 2, 4]], y_ref, bound(mag, y_ref, K), "the other rows")


def test_misaligned_and_host_pointers_are_refused():
    t = torch()
    M, K, R = 16, 64, 8
    A, B, *_ = bank_of(1, 1, R, M, K, "f16")
    x, y, ad = t.zeros(1, K, device="cuda"), t.zeros(1, M, device="cuda"), t.zeros(1, dtype=t.int32, device="cuda")
    m = q8()
    for args, status in (((x.data_ptr() + 4, A.cuda(), B.cuda(), None, None, ad, None, y), 3),
                         ((x, A.cuda().data_ptr() + 8, B.cuda(), None, None, ad, None, y), 3),
                         ((x, A, B.cuda(), None, None, ad, None, y), 4), ((x, A.cuda(), B.cuda(), None, None, None, None, y), 1),
                         ((x, A.cuda(), B.cuda(), None, None, ad.data_ptr() + 2, None, y), 3),
                         ((x, A.cuda(), B.cuda(), None, None, ad, None, y.data_ptr() + 4), 3)):
        with pytest.raises(m.Q8Error) as e:
            m.q8_lora(*args, M, K, 1, 1, R, m.Q8_F16)
        assert e.value.status == status
