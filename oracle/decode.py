"""fp64 definitions of the decode-step operators (test infrastructure only; no
code shared with the library): block tables and slot maps, the cache append,
attention of one token over a paged cache, and the logit controls. Everything
is written out request by request from the formulas."""
from __future__ import annotations

import numpy as np

# explicit mantissa bits, smallest normal exponent, largest finite value
FLOATS = {"bf16": (7, -126, 2.0 ** 128 * (1 - 2.0 ** -8)), "f16": (10, -14, 65504.0), "e4m3": (3, -6, 448.0),
          "f32": (23, -126, 2.0 ** 128 * (1 - 2.0 ** -24))}


def round_to(x, fmt: str, saturate: bool = False):
    """x (fp64) rounded to nearest, ties to even, on the grid of a float format."""
    bits, emin, top = FLOATS[fmt]
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        _, e = np.frexp(np.where(np.isfinite(x) & (x != 0), x, 1.0))
        ulp = 2.0 ** (np.maximum(e - 1, emin) - bits)
        y = np.where(np.isfinite(x), np.round(x / ulp) * ulp, x)   # numpy rounds half to even
        over = np.abs(y) > top
        return np.where(over, np.sign(y) * (top if saturate else np.inf), y)


def kv_tables(lengths, new, page, free, table, capacity):
    """Returns (table, slots, positions, rows, offsets, lengths, counts, status)."""
    table = np.array(table, np.int64)
    width, status, taken, tokens = table.shape[1], 0, 0, 0
    slots, positions, rows = (np.full(capacity, -1, np.int64) for _ in range(3))
    offsets, out_lengths = [0], []
    for i, (n, m) in enumerate(zip(lengths, new)):
        n, m = int(n), int(m)
        if n < 0 or m < 0 or n + m > 2 ** 31 - 1:
            status |= 8
        n, m = max(n, 0), max(m, 0)
        held, last = -(-n // page), -(-(n + m) // page)
        fresh = {}
        for j in range(held, last):
            fresh[j] = int(free[taken]) if taken < len(free) else -1
            if taken >= len(free):
                status |= 1
            taken += 1
            if j < width:
                table[i, j] = fresh[j]
        if m and last > width:
            status |= 2
        for pos in range(n, n + m):
            j = pos // page
            p = -1 if j >= width else fresh.get(j, table[i, j] if j < held else -1)
            if tokens < capacity:
                slots[tokens] = p * page + pos % page if p >= 0 else -1
                positions[tokens], rows[tokens] = pos, i
            else:
                status |= 4
            tokens += 1
        offsets.append(tokens)
        out_lengths.append(n + m)
    return table, slots, positions, rows, np.array(offsets), np.array(out_lengths), np.array([tokens, taken]), status


def kv_attention(q, k, v, table, lengths, scale, window=0, k_scale=1.0, v_scale=1.0):
    """q (requests, heads, dim), k and v (pages, page, kv heads, dim) in fp64.
    Returns out, lse, and for error bounds sum_j p_j |v_j| and the largest
    sum_d |q_d k_d| scale of the row."""
    requests, heads, dim = q.shape
    pages, page, kvh, _ = k.shape
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse, big = np.full((requests, heads), -np.inf), np.zeros((requests, heads))
    for r in range(requests):
        n = min(max(int(lengths[r]), 0), table.shape[1] * page)
        js = np.arange(max(0, n - window) if window else 0, n)
        if not js.size:
            continue
        at = np.asarray(table[r], np.int64)[js // page]
        held = (at >= 0) & (at < pages)
        kk = np.where(held[:, None, None], k[np.where(held, at, 0), js % page], 0.0) * k_scale
        vv = np.where(held[:, None, None], v[np.where(held, at, 0), js % page], 0.0) * v_scale
        for h in range(heads):
            g = h // (heads // kvh)
            s = kk[:, g] @ q[r, h] * scale
            big[r, h] = np.max(np.abs(kk[:, g]) @ np.abs(q[r, h])) * abs(scale)
            m = s.max()
            if m == -np.inf:
                continue
            p = np.exp(s - m)
            lse[r, h] = m + np.log(p.sum())
            out[r, h] = p @ vv[:, g] / p.sum()
            mag[r, h] = p @ np.abs(vv[:, g]) / p.sum()
    return out, lse, mag, big


def logits_process(x, history=None, history_lengths=None, prompt_lengths=None, repetition=None, presence=None,
                   frequency=None, bias=None, mask=None, mask_rows=None):
    """x (rows, vocab) fp64; bias: a list of {token: value} per row; mask: bool (mask rows, vocab)."""
    x = np.array(x, np.float64)
    rows, vocab = x.shape
    for b in range(rows):
        if history is not None:
            n = min(max(int(history_lengths[b]), 0), history.shape[1])
            p = max(int(prompt_lengths[b]), 0) if prompt_lengths is not None else 0
            h = [int(t) for t in history[b][:n]]
            r = 1.0 if repetition is None else float(repetition[b])
            for t in set(h):
                if 0 <= t < vocab:
                    x[b, t] = x[b, t] / r if x[b, t] > 0 else x[b, t] * r
            for t in set(h[p:]):
                if 0 <= t < vocab:
                    c = h[p:].count(t)
                    x[b, t] -= (0 if frequency is None else float(frequency[b])) * c
                    x[b, t] -= 0 if presence is None else float(presence[b])
        if bias is not None:
            for t, val in bias[b].items():
                if 0 <= t < vocab:
                    x[b, t] += val
        if mask is not None:
            row = b if mask_rows is None else int(mask_rows[b])
            if 0 <= row < len(mask):
                x[b, ~mask[row]] = -np.inf
    return x
