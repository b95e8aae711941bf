"""Double-precision references (numpy) of the per-request decode operators:
q8_sample, q8_moe_route_grouped and q8_lora, written from their statements in
include/q8.h."""
from __future__ import annotations

import numpy as np

NEG = -np.inf


def sample_row(logits, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, u=0.0):
    """(token, probability, kept set in the tokens' order) of one row."""
    l = np.asarray(logits, np.float32).astype(np.float64)
    l = np.where(np.isnan(l), NEG, l)
    V = l.size
    order = np.lexsort((np.arange(V), -l))
    m = l[order[0]]
    if m == NEG:
        return -1, 0.0, np.zeros(V, bool)
    kept = np.zeros(V, bool)
    if not temperature > 0:
        kept[order[0]] = True
        return int(order[0]), 1.0, kept
    s = l[order]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(s == m, 1.0, np.where(s == NEG, 0.0, np.exp((s - m) / float(temperature))))
    w = np.where(np.isnan(w), 1.0, w)
    w[w < 2.0 ** -44] = 0.0
    k = V if top_k <= 0 else min(V, int(top_k))
    n = k
    if top_p < 1:
        c = np.concatenate([[0.0], np.cumsum(w[:k])])
        n = max(1, int(np.sum(c[:-1] < float(top_p) * c[-1])))
    if min_p > 0:
        n = min(n, max(1, int(np.sum(w >= min(1.0, float(min_p))))))
    kept[order[:n]] = True
    full = np.zeros(V)
    full[order[:n]] = w[:n]
    kept &= full > 0
    c = np.cumsum(full)
    u = 0.0 if not u > 0 else min(float(u), 0.99999994)
    token = int(np.argmax(c > u * c[-1]))
    return token, full[token] / c[-1], kept


def route_token(logits, bias, top_k, n_group, topk_group, group_top, sigmoid, renormalize, scale):
    """(experts, weights) of one token."""
    l = np.asarray(logits, np.float32).astype(np.float64)
    l = np.where(np.isnan(l), NEG, l)
    E = l.size
    with np.errstate(invalid="ignore", over="ignore"):
        if sigmoid:
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            m = l.max()
            p = np.where(l == NEG, 0.0, np.where(l == m, 1.0, np.exp(l - m)))
            s = p / p.sum() if p.sum() > 0 else p
        c = s + (np.zeros(E) if bias is None else np.asarray(bias, np.float32).astype(np.float64))
        c = np.where(np.isnan(c), NEG, c)
        size = E // n_group
        value = []
        for g in range(n_group):
            best = np.sort(c[g * size:(g + 1) * size])[::-1][:group_top]
            v = best.sum()
            value.append(NEG if np.isnan(v) else v)
    stay = sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group] if n_group > 1 else [0]
    pool = sorted(e for g in stay for e in range(g * size, (g + 1) * size))
    idx = sorted(pool, key=lambda e: (-c[e], e))[:top_k]
    w = s[idx]
    if renormalize:
        w = w / w.sum() if w.sum() > 0 else np.zeros(top_k)
    return np.array(idx, np.int32), w * float(np.float32(scale))


def lora(x, A, B, rank, scale, adapter, residual):
    """(y, the sum of absolute products that the error bound scales with), both [N][M].  A [n][R][K], B [n][M][R]."""
    N, M = x.shape[0], B.shape[1]
    y = np.zeros((N, M)) if residual is None else residual.astype(np.float64)
    mag = np.zeros((N, M))
    for n in range(N):
        a = int(adapter[n])
        if not 0 <= a < A.shape[0]:
            continue
        r = A.shape[1] if rank is None else min(max(int(rank[a]), 0), A.shape[1])
        sc = 1.0 if scale is None else float(scale[a])
        Ar, Br, xn = A[a, :r].astype(np.float64), B[a, :, :r].astype(np.float64), x[n].astype(np.float64)
        y[n] += sc * (Br @ (Ar @ xn))
        mag[n] = abs(sc) * (np.abs(Br) @ (np.abs(Ar) @ np.abs(xn)))
    return y, mag
