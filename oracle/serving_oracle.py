"""Plain 64-bit definitions of the serving operators, in numpy, written from
their formulas: rotary positions and the paged cache's append, attention over
the cache, and the rules on logits.  Loops over sequences, tokens and heads;
nothing is shared with the GPU path.

A cache is an array [page, head, slot, dim]; a batch is (q_start, kv_len,
pages) as lists or arrays of integers.  Token j of the n new tokens of a
sequence has the position kv_len - n + j.
"""
from __future__ import annotations

import math

import numpy as np

NORM, NEOX = 0, 1


def positions(q_start, kv_len):
    """(sequence, position) of every packed row, (-1, 0) for rows of no sequence."""
    T = int(q_start[-1])
    out = [(-1, 0)] * T
    for b in range(len(kv_len)):
        n = q_start[b + 1] - q_start[b]
        for j in range(n):
            out[q_start[b] + j] = (b, int(kv_len[b]) - int(n) + j)
    return out


def rotate(x, pos, freqs, rot, style, scale=1.0):
    """x [..., dim]: pair i of the first `rot` values turned by pos * freqs[i]."""
    y = np.array(x, np.float64)
    for i in range(rot // 2):
        a = math.fmod(float(pos) * float(freqs[i]), 2 * math.pi)
        c, s = math.cos(a), math.sin(a)
        u, v = (2 * i, 2 * i + 1) if style == NORM else (i, i + rot // 2)
        y[..., u] = scale * (x[..., u] * c - x[..., v] * s)
        y[..., v] = scale * (x[..., u] * s + x[..., v] * c)
    return y


def append(q, k, v, freqs, rot, style, scale, q_start, kv_len, pages, k_cache, v_cache, rope_positions=None):
    """(q_out, k_cache, v_cache) in 64 bits; tokens of negative position are not stored."""
    kc, vc = np.array(k_cache, np.float64), np.array(v_cache, np.float64)
    qo = None if q is None else np.full(q.shape, np.nan)
    page = kc.shape[2]
    for t, (b, p) in enumerate(positions(q_start, kv_len)):
        if b < 0:
            continue
        at = p if rope_positions is None else int(rope_positions[t])
        if qo is not None:
            qo[t] = rotate(q[t], at, freqs, rot, style, scale)
        if p >= 0:
            g = pages[b][p // page]
            kc[g, :, p % page] = rotate(k[t], at, freqs, rot, style, scale)
            vc[g, :, p % page] = v[t]
    return qo, kc, vc


def attention(q, k_cache, v_cache, q_start, kv_len, pages, scale, causal, window):
    """(out, lse, bound, smax): bound[t, h] = max |V| over the keys row (t, h) sees,
    smax[t, h] = max over them of scale * sum |q_i K_i| (both 0 for a row that sees none)."""
    T, H, D = q.shape
    KV, page = k_cache.shape[1], k_cache.shape[2]
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    vmax, smax = np.zeros((T, H)), np.zeros((T, H))
    for t, (b, p) in enumerate(positions(q_start, kv_len)):
        if b < 0:
            continue
        see = [j for j in range(int(kv_len[b])) if (not causal or j <= p) and (not window or j > p - window)]
        if not see:
            continue
        j = np.array(see)
        g = np.asarray(pages[b])[j // page]
        for h in range(H):
            K, V = k_cache[g, h * KV // H, j % page], v_cache[g, h * KV // H, j % page]
            s = scale * (K @ q[t, h])
            m = s.max()
            e = np.exp(s - m)
            out[t, h] = (e @ V) / e.sum()
            lse[t, h] = m + np.log(e.sum())
            vmax[t, h] = np.abs(V).max()
            smax[t, h] = scale * (np.abs(K) @ np.abs(q[t, h])).max()
    return out, lse, vmax, smax


def logits(x, hist, repeat, frequency, presence, biases, allow):
    """x [rows, vocab]; hist: a list of ids per row or None; biases: a list of (id, value) per row or
    None; allow: truth values [rows, vocab] or None."""
    y = np.array(x, np.float64)
    rows, vocab = y.shape
    for r in range(rows):
        count = {}
        for i in (hist[r] if hist is not None else ()):
            if 0 <= i < vocab:
                count[int(i)] = count.get(int(i), 0) + 1
        for i, c in count.items():
            rp = 1.0 if repeat is None else float(repeat[r])
            y[r, i] = y[r, i] / rp if y[r, i] > 0 else y[r, i] * rp
            y[r, i] -= c * (0.0 if frequency is None else float(frequency[r])) + \
                (0.0 if presence is None else float(presence[r]))
        for i, b in (biases[r] if biases is not None else ()):
            if 0 <= i < vocab:
                y[r, i] += float(b)
        if allow is not None:
            y[r, ~allow[r]] = -np.inf
    return y


def head_norm(x, weight, eps):
    """x [..., dim] divided by the root of its mean square and multiplied by weight [dim] (None: x itself)."""
    x = np.array(x, np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + float(eps)) * np.asarray(weight, np.float64)


def router(x, w, bias, top_k, sigmoid, renormalize, scale):
    """(ids, weights) of each token: the largest p + bias first, the lower index among equals."""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    T, E = z.shape
    ids, weights = np.zeros((T, top_k), np.int64), np.zeros((T, top_k))
    for t in range(T):
        if sigmoid:
            p = 1.0 / (1.0 + np.exp(-z[t]))
        else:
            p = np.exp(z[t] - z[t].max())
            p = p / p.sum()
        # without a bias the scores have the order of p, also where p is too small to tell
        rank = z[t] if bias is None else p + np.asarray(bias, np.float64)
        ids[t] = sorted(range(E), key=lambda e: (-rank[e], e))[:top_k]
        v = p[ids[t]]
        weights[t] = (v / v.sum() if renormalize else v) * float(scale)
    return ids, weights


def activate(a, gelu):
    a = np.asarray(a, np.float64)
    if gelu:
        return 0.5 * a * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a ** 3)))
    return a / (1.0 + np.exp(-a))


def moe_ffn(x, gate, up, down, ids, weights, gelu, residual):
    """x [T, K]; gate, up [E, F, K], down [E, K, F] as values; ids outside the experts add nothing."""
    y = np.zeros(x.shape) if residual is None else np.array(residual, np.float64)
    for t in range(x.shape[0]):
        for s, e in enumerate(ids[t]):
            if 0 <= e < gate.shape[0]:
                y[t] += weights[t, s] * (down[e] @ (activate(gate[e] @ x[t], gelu) * (up[e] @ x[t])))
    return y


def sample(x, temperature, top_k, top_p, min_p, u):
    """(token, logprob, number kept) of one row of logits."""
    x = np.array(x, np.float64) + 0.0
    t, u = float(temperature), float(u)
    u = u if u > 0 else 0.0
    top = x.max() if x.size else -np.inf
    if not t >= 0 or np.isnan(x).any() or not np.isfinite(top):
        return -1, np.nan, 0
    if t == 0:
        return int(np.argmax(x)), 0.0, 1
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf]
    if top_k > 0:
        order = order[:int(top_k)]
    with np.errstate(over="ignore"):
        w = np.exp((x[order] - top) / t)
    n = len(order)
    if top_p < 1:
        n = min(n, 1 + int((np.cumsum(w) < max(float(top_p), 0.0) * w.sum()).sum()))
    if min_p > 0:
        least = top + t * math.log(min(float(min_p), 1.0)) if math.isfinite(t) else -np.inf
        n = min(n, int((x[order] >= least).sum()))
    kept = np.sort(order[:n])
    with np.errstate(over="ignore"):
        w = np.exp((x[kept] - top) / t)
    upto = np.cumsum(w)
    past = np.flatnonzero(upto > u * upto[-1]) if u < 1 else []
    at = int(past[0]) if len(past) else int(np.flatnonzero(w > 0)[-1])
    return int(kept[at]), float(np.log(w[at] / upto[-1])), len(kept)
