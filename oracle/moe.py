"""The operators around the experts' products (oracle; test infrastructure only).

Everything in float64 from the definitions: routing and its gradient, the rows
of each expert, the quantiser with fp32 scales, dispatch and combine with its
gradients, and the products whose block scales are fp32 numbers.
"""

import numpy as np

from .fp8 import e4m3_to_f64
from .quant import e4m3_encode_rne, quantize_fp8_1x128

EPS = 1e-20
BLOCK = 128


def scores(logits, score):
    """Softmax or sigmoid of float64 logits [T, E]; a softmax row of -inf alone is 0."""
    x = np.asarray(logits, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        top = x.max(axis=1, keepdims=True)
        e = np.exp(x - np.where(np.isneginf(top), 0.0, top))
        s = e.sum(axis=1, keepdims=True)
        return np.where(s == 0, 0.0, e / np.where(s == 0, 1.0, s))


def _best(keys, n):
    """Indices of the n largest of a 1-D list, largest first, ties to the lowest index."""
    return sorted(range(len(keys)), key=lambda i: (-keys[i], i))[:n]


def _ranked(v):
    """Keys and group scores rank as themselves, a NaN as -inf."""
    return np.where(np.isnan(v), -np.inf, v)


def route(logits, k, bias=None, score="softmax", n_groups=1, top_groups=1, group_top=2, renormalize=True, scale=1.0):
    """(ids int32 [T, k], weights float64 [T, k]). Without a bias the experts are
    ranked by their logits, which rank like the scores without their rounding."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    s = scores(x, score)
    key = _ranked(s if bias is None else s + np.asarray(bias, np.float64))
    rank = _ranked(x) if bias is None else key
    size = E // n_groups
    top = min(group_top, size)
    by_logit = bias is None and top == 1
    ids = np.zeros((T, k), np.int32)
    for t in range(T):
        groups = range(n_groups)
        if top_groups < n_groups:
            per = []
            for g in groups:
                mine = (rank if by_logit else key)[t, g * size:(g + 1) * size]
                with np.errstate(invalid="ignore"):
                    per.append(float(_ranked(sum(sorted(mine, reverse=True)[:top]))))
            groups = _best(per, top_groups)
        pool = sorted(e for g in groups for e in range(g * size, (g + 1) * size))
        ids[t] = [pool[i] for i in _best([rank[t, e] for e in pool], k)]
    w = np.take_along_axis(s, ids.astype(np.int64), axis=1)
    if renormalize:
        w = w / (w.sum(axis=1, keepdims=True) + EPS)
    return ids, scale * w


def route_weights(logits, ids, score="softmax", renormalize=True, scale=1.0):
    """The weights of given ids."""
    w = np.take_along_axis(scores(logits, score), np.asarray(ids, np.int64), axis=1)
    if renormalize:
        w = w / (w.sum(axis=1, keepdims=True) + EPS)
    return scale * w


def route_backward(logits, ids, d_weights, score="softmax", renormalize=True, scale=1.0):
    """(d_logits float64 [T, E], magnitude [T, E]): the gradient, slot by slot, and
    the sum of the absolute values of the terms it is added up from."""
    s = scores(logits, score)
    g = np.asarray(d_weights, np.float64)
    T, E = s.shape
    k = g.shape[1]
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        live = [j for j in range(k) if 0 <= ids[t, j] < E]
        S = sum(s[t, ids[t, j]] for j in live) + EPS
        ds, ms = np.zeros(E), np.zeros(E)
        for j in live:
            e = ids[t, j]
            if renormalize:
                terms = [(g[t, j] - g[t, l]) * s[t, ids[t, l]] for l in live] + [g[t, j] * EPS]
                ds[e] += scale / S ** 2 * sum(terms)
                ms[e] += abs(scale) / S ** 2 * sum(map(abs, terms))
            else:
                ds[e] += scale * g[t, j]
                ms[e] += abs(scale * g[t, j])
        if score == "sigmoid":
            d[t] = ds * s[t] * (1 - s[t])
            mag[t] = ms * s[t] * (1 - s[t])
        else:
            d[t] = s[t] * (ds - (ds * s[t]).sum())
            mag[t] = s[t] * (ms + (ms * s[t]).sum())
    return d, mag


def rows_bound(T, k, G):
    """Rows of T*k choices when min(G, T*k) experts each waste at most 127 of a 128-row block."""
    n = T * k
    return -(-(n + min(G, n) * 127) // BLOCK) * BLOCK


def expert_rows(ids, G, max_m=0):
    """(row_of [T, k], counts [G], first row of every expert [G]) for the contiguous
    layout (max_m = 0) or the masked one."""
    ids = np.asarray(ids)
    counts = np.array([(ids == e).sum() for e in range(G)], np.int64)
    if max_m:
        first = np.arange(G) * max_m
    else:
        blocks = -(-counts // BLOCK) * BLOCK
        first = np.cumsum(blocks) - blocks
    seen = np.zeros(G, np.int64)
    row_of = np.full(ids.shape, -1, np.int32)
    for t in range(ids.shape[0]):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            if 0 <= e < G:
                if not max_m or seen[e] < max_m:
                    row_of[t, j] = first[e] + seen[e]
                seen[e] += 1
    return row_of, counts, first


def m_indices(counts, first, rows):
    idx = np.full(rows, -1, np.int32)
    for e, (c, f) in enumerate(zip(counts, first)):
        idx[f:f + c] = e
    return idx


def quantize_fp8_1x128_sf_f32(x):
    """(codes uint8 [R, K], sf float32 [R, K/128]): amax / 448 and E4M3(x * (448 / amax)),
    quotients and products rounded to fp32 as the definition says."""
    x = np.asarray(x, np.float32)
    R, K = x.shape
    xb = x.reshape(R, K // BLOCK, BLOCK)
    amax = np.maximum(np.abs(xb).max(axis=2), np.float32(1e-4))
    sf = amax / np.float32(448)
    prod = xb * (np.float32(448) / amax)[:, :, None]
    return e4m3_encode_rne(prod.astype(np.float64)).reshape(R, K), sf


def dispatch(x, row_of, rows, packed):
    """{row: (codes [H], scale row)} of every row that a slot names."""
    if packed:
        q, sf, _ = quantize_fp8_1x128(np.asarray(x, np.float64))
    else:
        q, sf = quantize_fp8_1x128_sf_f32(x)
    return {int(r): (q[t], sf[t]) for t in range(x.shape[0]) for r in row_of[t] if 0 <= r < rows}


def combine(y, row_of, weights=None):
    """(out float64 [T, H], sum of the terms' magnitudes)."""
    y = np.asarray(y, np.float64)
    T, k = row_of.shape
    out, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= row_of[t, j] < y.shape[0]:
                term = y[row_of[t, j]] * (1.0 if weights is None else float(weights[t, j]))
                out[t] += term
                mag[t] += abs(term)
    return out, mag


def combine_backward(y, row_of, weights, d_out):
    """({row: d_y row}, d_weights [T, k], sum of the magnitudes of its terms)."""
    y, d_out = np.asarray(y, np.float64), np.asarray(d_out, np.float64)
    T, k = row_of.shape
    d_y, d_w, mag = {}, np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = int(row_of[t, j])
            if 0 <= r < y.shape[0]:
                d_y[r] = d_out[t] * (1.0 if weights is None else float(weights[t, j]))
                d_w[t, j] = (y[r] * d_out[t]).sum()
                mag[t, j] = abs(y[r] * d_out[t]).sum()
    return d_y, d_w, mag


def dequant_sf_f32(q, sf, gran=1):
    """Values of codes uint8 [R, K] with fp32 scales [ceil(R/gran), K/128]."""
    v = e4m3_to_f64(q)
    s = np.repeat(np.repeat(np.asarray(sf, np.float64), gran, axis=0)[:q.shape[0]], BLOCK, axis=1)
    return v * s


def fp8_gemm_nt_sf_f32(a, sfa, b, sfb, gran=128, c=None):
    """(D float64 [M, N], sum of the terms' magnitudes)."""
    x, w = dequant_sf_f32(a, sfa), dequant_sf_f32(b, sfb, gran)
    d, mag = x @ w.T, abs(x) @ abs(w).T
    if c is not None:
        d, mag = d + np.asarray(c, np.float64), mag + abs(np.asarray(c, np.float64))
    return d, mag
