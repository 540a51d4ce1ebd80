"""CPU oracles, in float64, of the operators before and after the TopK.
TEST INFRASTRUCTURE, NOT PRODUCT: only ``tests/`` may import this module.

Plain loops over rows, written from the formulas in ``include/dsel.h``; inputs are
numpy arrays that already hold the values of the device tensors (float64 holds every
float32, bfloat16, float16 and e4m3 value exactly).
"""
from __future__ import annotations

import numpy as np


def oracle_logits(x, stride, *, tokens=None, prompt_len=None, total_len=None, repetition=None, frequency=None,
                  presence=None, biases=None, mask=None, mask_rows=None):
    """Rows of ``process_logits`` and, beside them, the sum of the magnitudes that each value was
    computed from and the number of roundings in float32 (for a bound on the device's error).

    ``biases``: a list of (id, value) pairs per row.  Returns (y, magnitude, roundings), each
    [rows, stride] float64."""
    rows, vocab = x.shape
    y = np.full((rows, stride), -np.inf)
    mag = np.zeros((rows, stride))
    rnd = np.zeros((rows, stride))
    with np.errstate(invalid="ignore", over="ignore"):
        for r in range(rows):
            z = x[r].astype(np.float64).copy()
            m, n = np.abs(z), np.zeros(vocab)
            if tokens is not None:
                total = tokens.shape[1] if total_len is None else min(max(int(total_len[r]), 0), tokens.shape[1])
                prompt = 0 if prompt_len is None else int(prompt_len[r])
                rep = 1.0 if repetition is None else float(repetition[r])
                freq = 0.0 if frequency is None else float(frequency[r])
                pres = 0.0 if presence is None else float(presence[r])
                seen, count = set(), {}
                for i in range(total):
                    v = int(tokens[r, i])
                    if 0 <= v < vocab:
                        seen.add(v)
                        if i >= prompt:
                            count[v] = count.get(v, 0) + 1
                for v in seen:
                    z[v] = z[v] / rep if z[v] > 0 else z[v] * rep
                    m[v] = max(m[v], abs(z[v]))
                    n[v] += 2.001     # the reciprocal and the product: (1 + e)^2 - 1 < 2.001 e for e = 2^-24
                for v, c in count.items():
                    z[v] -= freq * c + pres
                    m[v] += abs(freq * c) + abs(pres)
                    n[v] += 3
            for v, b in (biases[r] if biases is not None else []):
                if 0 <= v < vocab:
                    z[v] += float(b)
                    m[v] += abs(float(b))
                    n[v] += 2
            if mask is not None:
                at = r if mask_rows is None else int(mask_rows[r])
                if 0 <= at < mask.shape[0]:
                    for v in range(vocab):
                        if not (int(mask[at, v // 32]) >> (v % 32)) & 1:
                            z[v], m[v], n[v] = -np.inf, 0.0, 0.0
            y[r, :vocab], mag[r, :vocab], rnd[r, :vocab] = z, m, n
    return y, mag, rnd


def _slots(table, seq, page_size, pages, positions):
    """(page, place) of each position of a sequence; page -1 where it does not exist."""
    page = np.full(len(positions), -1, dtype=np.int64)
    if 0 <= seq < table.shape[0]:
        i = positions // page_size
        inside = i < table.shape[1]
        page[inside] = table[seq, i[inside]]
        page[(page < 0) | (page >= pages)] = -1
    return page, positions % page_size


def _sequence(t, seq_ids, table):
    return int(seq_ids[t]) if seq_ids is not None else (0 if table.shape[0] == 1 else t)


def oracle_score(q, weights, keys, table, end, row_stride, *, seq_ids=None, key_scale=None):
    """Scores [tokens, row_stride] (float64) and a bound on what float32 sums can be off by.

    The bound: a product of two operands of at most 11 bits is exact; a sum of dim products in
    float32, whatever its order and with truncated additions, is off by at most
    (dim + 8) * 2^-23 times the sum of their magnitudes; each head's weighted term and each
    addition of the sum over heads rounds once (2^-24 of the running magnitude, heads + 8 times)."""
    tokens, heads, dim = q.shape
    out = np.full((tokens, row_stride), -np.inf)
    err = np.zeros((tokens, row_stride))
    with np.errstate(invalid="ignore", over="ignore"):
        for t in range(tokens):
            n = min(max(int(end[t]), 0), row_stride)
            pos = np.arange(n)
            page, place = _slots(table, _sequence(t, seq_ids, table), keys.shape[1], keys.shape[0], pos)
            pos, page, place = pos[page >= 0], page[page >= 0], place[page >= 0]
            k = keys[page, place].astype(np.float64)
            z = q[t].astype(np.float64) @ k.T
            a = np.abs(q[t].astype(np.float64)) @ np.abs(k).T
            w = weights[t].astype(np.float64)[:, None]
            z = np.where(np.isnan(z), z, np.maximum(z, 0))
            s = key_scale[page, place].astype(np.float64) if key_scale is not None else np.ones(len(pos))
            out[t, pos] = (w * z).sum(0) * s
            err[t, pos] = ((np.abs(w) * a).sum(0) * (dim + 8) * 2.0 ** -23
                           + (np.abs(w) * z).sum(0) * (heads + 8) * 2.0 ** -24) * np.abs(s) + 2.0 ** -120
    return out, err


def oracle_attention(q, k_cache, v_cache, table, indices, end, *, block=1, seq_ids=None, scale=None, eps=2.0 ** -8):
    """(o, lse, bound on o, bound on lse) in float64; ``eps``: half a step of the operands' type.

    A score's sum of dim exact products in float32 is off by at most (dim + 8) * 2^-23 of the sum of
    magnitudes, its scaling and the subtraction of the maximum by 2^-23 of their magnitudes; powers
    of two by 2^-21.  A probability then is off by that much absolutely in the exponent (d), plus eps
    where it is rounded for the product with v (not in the sum), so
    |o - o'| <= sum_n p_n |v_n| (2 d + eps + (n + 64) * 2^-22), and one rounding of o to its type;
    lse is off by d and by the rounding of itself."""
    tokens, hq, dim = q.shape
    pages, page_size, hk, _ = k_cache.shape
    scale = dim ** -0.5 if scale is None else scale
    o = np.zeros((tokens, hq, dim))
    lse = np.full((tokens, hq), -np.inf)
    oerr, lerr = np.zeros_like(o), np.zeros_like(lse)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        for t in range(tokens):
            for g in range(hk):
                mine = indices[t, g] if indices.ndim == 3 else indices[t]
                mine = mine[mine >= 0].astype(np.int64)
                pos = (mine[:, None] * block + np.arange(block)).reshape(-1)
                pos = pos[pos < int(end[t])]
                page, place = _slots(table, _sequence(t, seq_ids, table), page_size, pages, pos)
                page, place = page[page >= 0], place[page >= 0]
                if len(page) == 0:
                    continue
                k, v = k_cache[page, place, g].astype(np.float64), v_cache[page, place, g].astype(np.float64)
                for h in range(g * (hq // hk), (g + 1) * (hq // hk)):
                    z = scale * (k @ q[t, h].astype(np.float64))
                    top = np.max(z)
                    if top == -np.inf:
                        continue
                    e = np.exp(z - top)
                    p = e / e.sum()
                    o[t, h] = p @ v
                    lse[t, h] = top + np.log(e.sum())
                    a = abs(scale) * (np.abs(k) @ np.abs(q[t, h].astype(np.float64)))
                    d = np.max(a * (dim + 8) * 2.0 ** -23 + (np.abs(z) + abs(top)) * 2.0 ** -22)
                    mag = p @ np.abs(v)
                    oerr[t, h] = mag * (2 * d + eps + (len(page) + 64) * 2.0 ** -22)
                    oerr[t, h] += (np.abs(o[t, h]) + oerr[t, h]) * eps + 2.0 ** -24 * (eps < 2.0 ** -9)
                    lerr[t, h] = d + (len(page) + 64) * 2.0 ** -22 + abs(lse[t, h]) * 2.0 ** -22
    return o, lse, oerr, lerr
