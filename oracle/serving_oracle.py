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
