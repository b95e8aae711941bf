"""What each request of a batch brings to a decode step of its own, timed case by case: the low-rank adapters
beside a shared Q8_0 projection, the expert router with biased and grouped scores, and the sampler behind the head.

``run`` computes the operators in plain torch operations, or, with ``own`` set, calls the library's entry points on
the same inputs.  ``exact`` gives the same outputs from the definitions in double precision.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_CODES = {"f32": 0, "f16": 1, "bf16": 2}  # the library's Q8_F32, Q8_F16, Q8_BF16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _lora(name, M, K, N, R, bank, used, bare, dtype, base, residual, ragged):
    """base: "none" (the adapters alone), "exact" or "split" (beside the projection).  used: distinct adapters among
    the rows that have one; bare: rows without an adapter."""
    return {"name": name, "op": "lora", "M": M, "K": K, "N": N, "R": R, "bank": bank, "used": used, "bare": bare,
            "dtype": dtype, "base": base, "residual": residual, "ragged": ragged}


def _route(name, T, E, top_k, groups, keep, group_top, sigmoid, bias, renormalize, scale):
    return {"name": name, "op": "route", "T": T, "E": E, "top_k": top_k, "groups": groups, "keep": keep,
            "group_top": group_top, "sigmoid": sigmoid, "bias": bias, "renormalize": renormalize, "scale": scale}


def _sample(name, N, V, ld, mode, spread, masked):
    """mode: which filters the rows use.  spread: standard deviation of the logits' bulk.  masked: share of the
    vocabulary at -inf in every other row."""
    return {"name": name, "op": "sample", "N": N, "V": V, "ld": ld, "mode": mode, "spread": spread, "masked": masked}


def listed():
    return [
        # one request with an adapter on the 0.5B down projection: the smallest decode call
        _lora("lora_down_05b_n1", 896, 4864, 1, 16, 4, 1, 0, "bf16", "exact", True, False),
        # a mixed batch on the 0.5B qkv projection: some rows bare, ranks of several adapters differing
        _lora("lora_qkv_05b_n8", 1152, 896, 8, 8, 8, 3, 2, "f16", "split", False, True),
        # four requests with their own adapters on the 7B-class down projection
        _lora("lora_down_7b_n4", 3584, 18944, 4, 64, 8, 4, 0, "bf16", "exact", True, False),
        # the full batch, every row with another adapter, beside the tensor-core projection
        _lora("lora_down_7b_n16", 3584, 18944, 16, 128, 24, 16, 0, "bf16", "split", True, False),
        # the adapters alone, as they stand beside a K-quant or integer product; the whole batch on one adapter
        _lora("lora_alone_shared_n16", 3584, 3584, 16, 32, 4, 1, 0, "f32", "none", True, False),
        # the adapters alone, sixteen of them, their ranks differing up to the largest
        _lora("lora_alone_n16", 3584, 18944, 16, 128, 16, 16, 0, "bf16", "none", True, True),
        # the router of one token over 60 experts, renormalised
        _route("route_t1", 1, 60, 4, 1, 1, 1, False, True, True, 1.0),
        # a full decode batch over 256 experts in 8 groups, sigmoid scores and a balance bias
        _route("route_t16", 16, 256, 8, 8, 4, 2, True, True, True, 2.5),
        # a prompt routed at once
        _route("route_t4096", 4096, 256, 8, 8, 4, 2, True, True, True, 2.5),
        # one request's sampler on the 0.5B vocabulary, all filters on
        _sample("sample_n1", 1, 151936, 151936, "all", 2.5, 0.0),
        # a batch on the padded 7B vocabulary, nucleus only on a flat distribution: the filter's boundary lies deep
        _sample("sample_n16_nucleus", 16, 151936, 152064, "nucleus", 1.0, 0.0),
        # several samples a request from a large batch, rows with different filters, constrained tokens at -inf
        _sample("sample_n128_mixed", 128, 152064, 152064, "mixed", 2.0, 0.4),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lora", "lora", "route", "sample", "sample"])
    if op == "lora":
        N = rng.randint(1, 16)
        bare = rng.randint(0, N // 3)
        used = rng.randint(1, N - bare)
        dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
        return _lora("", _log_int(rng, 200, 3584), 32 * _log_int(rng, 28, 592), N,
                     8 * _log_int(rng, 1, 8 if dtype == "f32" else 16), used + rng.randint(0, 8), used, bare, dtype,
                     rng.choice(["exact", "split", "none"]), rng.random() < 0.6, rng.random() < 0.5)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        size = rng.randint(4, 256 // groups)
        E = groups * size
        keep = rng.randint(max(1, groups // 2), groups)
        return _route("", _log_int(rng, 1, 4096), E, rng.randint(1, min(8, keep * size)), groups, keep,
                      rng.choice([1, 2]), rng.random() < 0.6, rng.random() < 0.7, rng.random() < 0.6,
                      rng.choice([1.0, 2.5]))
    V = _log_int(rng, 1000, 152064)
    return _sample("", _log_int(rng, 1, 128), V, V + rng.choice([0, 0, rng.randint(1, 128)]),
                   rng.choice(["all", "nucleus", "top_k", "min_p", "plain", "mixed"]), rng.uniform(0.7, 3.0),
                   rng.choice([0.0, 0.0, 0.4, 0.95]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _rank_of(case, i):
    """Rank of the i-th adapter in use."""
    return case["R"] if not case["ragged"] else max(1, case["R"] - (i % 4) * case["R"] // 5)


def _prepare_lora(case, g):
    dev = "cuda"
    M, K, N, R, bank = case["M"], case["K"], case["N"], case["R"], case["bank"]
    dt = _DTYPES[case["dtype"]]
    place = torch.randperm(bank, generator=g, device=dev)  # where in the bank the i-th adapter in use lies
    rows = torch.randperm(N, generator=g, device=dev)
    adapter = torch.full((N,), -1, dtype=torch.int32, device=dev)
    lead = torch.arange(N - case["bare"], device=dev)
    adapter[rows[lead]] = place[lead % case["used"]].to(torch.int32)
    rank = torch.tensor([_rank_of(case, i) for i in range(bank)], dtype=torch.int32, device=dev)
    rank = torch.empty_like(rank).scatter_(0, place, rank)
    s = {"op": "lora", "M": M, "K": K, "N": N, "R": R, "bank": bank, "dtype": case["dtype"], "base": case["base"],
         "adapter": adapter, "rank": rank,
         "A": (torch.randn(bank, R, K, generator=g, device=dev) / math.sqrt(K)).to(dt),
         "B": (torch.randn(bank, M, R, generator=g, device=dev) * 0.1).to(dt),
         "scale": 0.5 + 1.5 * torch.rand(bank, generator=g, device=dev),
         "x": torch.randn(N, K, generator=g, device=dev),
         "residual": torch.randn(N, M, generator=g, device=dev) if case["residual"] else None,
         "y": torch.empty(N, M, device=dev), "W": None}
    if case["base"] != "none":
        # Q8_0 weights in the library's packed layout: groups of 8 rows; per group the 16-byte columns of the 8 rows
        # (q + 128), then a binary16 scale for each block of 32 and row; rows past M are zero
        B, G = K // 32, -(-M // 8)
        q = torch.randint(1, 256, (G, 2 * B, 8, 16), generator=g, device=dev, dtype=torch.uint8)
        d = ((0.5 + torch.rand(G, B, 8, generator=g, device=dev)) / (127.0 * math.sqrt(K))).to(torch.float16)
        pad = torch.arange(8 * G, device=dev).view(G, 8) >= M
        q.masked_fill_(pad[:, None, :, None], 128)
        d.masked_fill_(pad[:, None, :], 0.0)
        s["W"] = torch.cat([q.view(G, 256 * B), d.view(G, 8 * B).view(torch.uint8)], 1).contiguous()
    return s


def _prepare_route(case, g):
    dev = "cuda"
    T, E, k = case["T"], case["E"], case["top_k"]
    s = {key: case[key] for key in ("op", "T", "E", "top_k", "groups", "keep", "group_top", "sigmoid", "renormalize",
                                    "scale")}
    s["logits"] = torch.randn(T, E, generator=g, device=dev) * 1.5
    s["bias"] = torch.randn(E, generator=g, device=dev) * 0.05 if case["bias"] else None
    s["idx"] = torch.empty(T, k, dtype=torch.int32, device=dev)
    s["w"] = torch.empty(T, k, device=dev)
    return s


def _prepare_sample(case, g):
    dev = "cuda"
    N, V, ld, mode = case["N"], case["V"], case["ld"], case["mode"]
    logits = torch.randn(N, ld, generator=g, device=dev) * case["spread"]
    # a handful of likely tokens above the bulk, one in each 24th of the vocabulary (a token drawn twice would get
    # whichever of its two values is written last)
    likely = torch.arange(24, device=dev) * (V // 24) + torch.randint(0, V // 24, (N, 24), generator=g, device=dev)
    logits.scatter_(1, likely, 3.0 * case["spread"] + 3.0 * torch.rand(N, 24, generator=g, device=dev))
    if case["masked"]:
        out = torch.rand(N, ld, generator=g, device=dev) < case["masked"]
        out[::2] = False
        logits.masked_fill_(out, -math.inf)

    def pick(lo, hi):
        return lo + (hi - lo) * torch.rand(N, generator=g, device=dev)

    row = torch.arange(N, device=dev)
    s = {"op": "sample", "N": N, "V": V, "ld": ld, "logits": logits, "u": torch.rand(N, generator=g, device=dev),
         "temperature": pick(0.6, 1.3), "top_k": None, "top_p": None, "min_p": None,
         "token": torch.empty(N, dtype=torch.int32, device=dev), "prob": torch.empty(N, device=dev)}
    if mode in ("all", "top_k", "mixed"):
        s["top_k"] = pick(5, 200).to(torch.int32)
    if mode in ("all", "nucleus", "mixed"):
        s["top_p"] = pick(0.8, 0.99)
    if mode in ("all", "min_p", "mixed"):
        s["min_p"] = pick(0.01, 0.1)
    if mode == "mixed":  # some rows greedy, the others with one filter, two, three or none
        s["temperature"][row % 8 == 7] = 0.0
        s["top_k"][row % 2 == 1] = 0
        s["top_p"][row % 3 == 2] = 1.0
        s["min_p"][row % 4 != 0] = 0.0
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"lora": _prepare_lora, "route": _prepare_route, "sample": _prepare_sample}[case["op"]](case, g)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own_lora(q8, s):
    tail = (s["x"], s["A"], s["B"], s["rank"], s["scale"], s["adapter"], s["residual"], s["y"], s["M"], s["K"], s["N"],
            s["bank"], s["R"], _CODES[s["dtype"]])
    if s["base"] == "none":
        q8.q8_lora(*tail)
    elif s["base"] == "exact":
        q8.q8_gemv_lora(s["W"], *tail)
    else:
        q8.q8_gemv_lora_split(s["W"], *tail)
    return s["y"]


def _own_route(q8, s):
    q8.q8_moe_route_grouped(s["logits"], s["bias"], s["T"], s["E"], s["top_k"], s["groups"], s["keep"], s["group_top"],
                            int(s["sigmoid"]), int(s["renormalize"]), s["scale"], s["idx"], s["w"])
    return s["idx"], s["w"]


def _own_sample(q8, s):
    q8.q8_sample(s["logits"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"], s["token"], s["prob"],
                 s["N"], s["V"], s["ld"])
    return s["token"], s["prob"]


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _weights(W, M, K, dt):
    """Packed Q8_0 bytes -> [M][K] in `dt`."""
    B, G = K // 32, W.shape[0]
    q = W[:, :256 * B].reshape(G, 2 * B, 8, 16).to(dt) - 128.0
    d = W[:, 256 * B:].contiguous().view(torch.float16).reshape(G, B, 8).to(dt)
    w = q.view(G, B, 2, 8, 16) * d[:, :, None, :, None]
    return w.permute(0, 3, 1, 2, 4).reshape(8 * G, K)[:M]


def _plain_lora(s):
    a = s["adapter"].long().clamp(min=0)
    has = (s["adapter"] >= 0).float()
    A, B = s["A"][a].float(), s["B"][a].float()  # [N][R][K], [N][M][R]
    u = torch.matmul(A, s["x"][:, :, None])[:, :, 0]
    u = torch.where(torch.arange(s["R"], device=u.device) < s["rank"][a][:, None], u, torch.zeros_like(u))
    y = torch.matmul(B, u[:, :, None])[:, :, 0] * (s["scale"][a] * has)[:, None]
    if s["residual"] is not None:
        y = y + s["residual"]
    if s["W"] is not None:
        y = y + torch.matmul(s["x"], _weights(s["W"], s["M"], s["K"], torch.float32).t())
    return y


def _plain_route(s):
    # in double: picks are decided between scores that lie next to each other
    l = s["logits"].double()
    if s["sigmoid"]:
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        p = torch.exp(l - l.max(1, keepdim=True).values)
        score = p / p.sum(1, keepdim=True)
    c = score if s["bias"] is None else score + s["bias"].double()
    by_group = c.view(s["T"], s["groups"], -1)
    if s["groups"] > 1:
        best = by_group.sort(dim=2, descending=True).values[:, :, :s["group_top"]].sum(2)
        order = best.sort(dim=1, descending=True, stable=True).indices[:, :s["keep"]]
        stays = torch.zeros_like(best, dtype=torch.bool).scatter_(1, order, True)
        c = by_group.masked_fill(~stays[:, :, None], -math.inf).reshape(s["T"], -1)
    idx = c.sort(dim=1, descending=True, stable=True).indices[:, :s["top_k"]]
    w = score.gather(1, idx)
    if s["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return idx.to(torch.int32), (w * s["scale"]).float()


def _plain_sample(s):
    # in double: a token is decided by long sums next to a border
    N, V = s["N"], s["V"]
    l = s["logits"][:, :V]
    v, order = l.sort(dim=1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    w = torch.exp((v.double() - v[:, :1].double()) / torch.where(greedy, torch.ones_like(t), t))
    w = torch.where(w < 2.0 ** -44, torch.zeros_like(w), w)
    place = torch.arange(V, device=l.device)[None, :]
    keep = (place == 0) | ~greedy
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep = keep & ((k <= 0) | (place < k))
    w = torch.where(keep, w, torch.zeros_like(w))
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        before = torch.cumsum(w, 1) - w
        w = torch.where((p >= 1) | (place == 0) | (before < p * w.sum(1, keepdim=True)), w, torch.zeros_like(w))
    if s["min_p"] is not None:
        w = torch.where((place == 0) | (w >= s["min_p"].double()[:, None]), w, torch.zeros_like(w))
    w = torch.zeros_like(w).scatter_(1, order, w)  # back to the tokens' order
    c = torch.cumsum(w, 1)
    total = c[:, -1:]
    hit = (c > s["u"].double()[:, None] * total) & (w > 0)
    token = torch.where(hit, place, torch.full_like(place, V - 1)).min(1).values
    return token.to(torch.int32), (w.gather(1, token[:, None]) / total)[:, 0].float()


def run(state):
    op = state["op"]
    if own:
        import q8_block_quantized_02_b200 as q8
        return {"lora": _own_lora, "route": _own_route, "sample": _own_sample}[op](q8, state)
    return {"lora": _plain_lora, "route": _plain_route, "sample": _plain_sample}[op](state)


# ---------------------------------------------------------------------------
# the definitions in double precision
# ---------------------------------------------------------------------------
def _exact_lora(s):
    y = torch.zeros(s["N"], s["M"], dtype=torch.float64, device="cuda")
    if s["residual"] is not None:
        y += s["residual"]
    x = s["x"].double()
    for n in range(s["N"]):
        a = int(s["adapter"][n])
        if a >= 0:
            r = int(s["rank"][a])
            u = (s["A"][a, :r].double() * x[n]).sum(1)
            y[n] += float(s["scale"][a]) * (s["B"][a, :, :r].double() * u).sum(1)
    if s["W"] is not None:
        B = s["K"] // 32
        raw = s["W"][:, :256 * B].reshape(-1, B, 2, 8, 16)
        d = s["W"][:, 256 * B:].contiguous().view(torch.float16).reshape(-1, B, 8).double()
        for n in range(s["N"]):
            xb = x[n].view(B, 2, 16)
            for g0 in range(0, raw.shape[0], 64):
                dot = ((raw[g0:g0 + 64].double() - 128) * xb[None, :, :, None, :]).sum((2, 4))  # [groups][block][row]
                rows = (dot * d[g0:g0 + 64]).sum(1).reshape(-1)
                lo = 8 * g0
                hi = min(s["M"], lo + rows.numel())
                y[n, lo:hi] += rows[:hi - lo]
    return y


def _exact_route(s):
    import numpy as np
    l = s["logits"].double().cpu().numpy()
    T, E = l.shape
    score = 1 / (1 + np.exp(-l)) if s["sigmoid"] else np.exp(l - l.max(1, keepdims=True))
    if not s["sigmoid"]:
        score = score / score.sum(1, keepdims=True)
    c = score + (0 if s["bias"] is None else s["bias"].double().cpu().numpy())
    size = E // s["groups"]
    idx = np.empty((T, s["top_k"]), np.int32)
    w = np.empty((T, s["top_k"]))
    for t in range(T):
        value = [sum(sorted(c[t, g * size:(g + 1) * size])[::-1][:s["group_top"]]) for g in range(s["groups"])]
        stay = sorted(range(s["groups"]), key=lambda g: (-value[g], g))[:s["keep"]]
        open_ = [e for g in stay for e in range(g * size, (g + 1) * size)]
        idx[t] = sorted(open_, key=lambda e: (-c[t, e], e))[:s["top_k"]]
        w[t] = score[t, idx[t]]
    if s["renormalize"]:
        w = w / w.sum(1, keepdims=True)
    return torch.from_numpy(idx).cuda(), torch.from_numpy(w * s["scale"]).cuda()


def _exact_sample(s):
    import numpy as np
    token = np.empty(s["N"], np.int32)
    prob = np.empty(s["N"])
    host = {k: None if s[k] is None else s[k].cpu().numpy() for k in ("temperature", "top_k", "top_p", "min_p", "u")}
    for n in range(s["N"]):
        l = s["logits"][n, :s["V"]].cpu().numpy()
        order = np.lexsort((np.arange(l.size), -l))
        t = float(host["temperature"][n])
        if t <= 0:
            token[n], prob[n] = order[0], 1.0
            continue
        w = np.exp((l[order].astype(np.float64) - float(l[order[0]])) / t)
        w[w < 2.0 ** -44] = 0
        k = l.size if host["top_k"] is None or host["top_k"][n] <= 0 else min(l.size, int(host["top_k"][n]))
        m = k
        if host["top_p"] is not None and host["top_p"][n] < 1:
            c = np.cumsum(w[:k])
            m = 1 + int(np.searchsorted(c, float(host["top_p"][n]) * c[-1], side="left"))
        if host["min_p"] is not None:
            m = min(m, int(np.sum(w >= float(host["min_p"][n]))))
        m = max(1, min(m, k))
        kept = np.zeros(l.size)
        kept[order[:m]] = w[:m]
        c = np.cumsum(kept)
        token[n] = int(np.searchsorted(c, float(host["u"][n]) * c[-1], side="right"))
        prob[n] = kept[token[n]] / c[-1]
    return torch.from_numpy(token).cuda(), torch.from_numpy(prob).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    return {"lora": _exact_lora, "route": _exact_route, "sample": _exact_sample}[case["op"]](s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "lora":
        M, K, N = case["M"], case["K"], case["N"]
        size = 4 if case["dtype"] == "f32" else 2
        ranks = [_rank_of(case, i) for i in range(case["used"])]
        rows = sum(ranks[i % case["used"]] for i in range(N - case["bare"]))  # sum of the rows' ranks
        n_bytes = sum(ranks) * (K + M) * size + 4 * N * K + 4 * N * M * (2 if case["residual"] else 1)
        flops = 2 * rows * (K + M)
        if case["base"] != "none":
            n_bytes += -(-M // 8) * 8 * K // 32 * 34
            flops += 2 * N * M * K
        return {"bytes": n_bytes, "flops": flops}
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        return {"bytes": 4 * T * E + 4 * E * case["bias"] + 8 * T * case["top_k"], "flops": 4 * T * E}
    return {"bytes": 4 * case["N"] * case["V"] + 28 * case["N"], "flops": 4 * case["N"] * case["V"]}
