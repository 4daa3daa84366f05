"""fp64 definitions of the operators of a layer's step (test infrastructure only;
no code shared with the library): norm, rotary positions, the gated delta rule
and the choice of the next token, written out from the formulas."""
from __future__ import annotations

import math

import numpy as np


def norm(x, residual=None, gate=None, weight=None, group=None, eps=1e-6, offset=0.0):
    """x (rows, cols) in fp64; returns the sum and the result."""
    s = np.array(x, np.float64) + (0.0 if residual is None else residual)
    out = np.empty_like(s)
    group = group or s.shape[1]
    w = np.ones(group) if weight is None else np.asarray(weight, np.float64) + offset
    for g in range(0, s.shape[1], group):
        h = s[:, g:g + group]
        out[:, g:g + group] = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w
    if gate is not None:
        with np.errstate(over="ignore"):
            out = out * (gate / (1 + np.exp(-gate)))
    return s, out


def rotary_frequencies(rotary_dim, base, scaling="none", factor=1.0, context=0.0, slow=1.0, fast=32.0):
    """Radians a position, and the magnitude."""
    f, magnitude = [], 1.0
    if scaling == "dimensions":
        magnitude = 0.1 * math.log(factor) + 1
        where = {n: rotary_dim * math.log(context / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (fast, slow)}
        low, high = max(math.floor(where[fast]), 0), min(math.ceil(where[slow]), rotary_dim - 1)
    for i in range(rotary_dim // 2):
        x = base ** (-2 * i / rotary_dim)
        share = 0.0             # of the scaled frequency
        if scaling == "linear":
            share = 1.0
        elif scaling == "dimensions":
            share = (i - low) / max(high - low, 0.001)
        elif scaling == "turns":
            share = 1 - (context * x / (2 * math.pi) - slow) / (fast - slow)
        share = min(max(share, 0.0), 1.0)
        f.append(x / factor * share + x * (1 - share))
    return np.array(f), magnitude


def rotary(x, positions, frequencies, magnitude=1.0, interleaved=False, weight=None, eps=1e-6, offset=0.0):
    """x (tokens, heads, dim) in fp64, frequencies uint64 (turns a position times 2^64, whole-number arithmetic)."""
    y = np.array(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * (np.asarray(weight, np.float64) + offset)
    z = y.copy()
    half = len(frequencies)
    for t, p in enumerate(positions):
        if p < 0:
            z[t] = np.nan       # left out
            continue
        for i, f in enumerate(frequencies):
            angle = 2 * math.pi * ((int(p) * int(f)) % 2 ** 64) / 2.0 ** 64
            j, k = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            a, b = y[t, :, j], y[t, :, k]
            z[t, :, j] = magnitude * (a * math.cos(angle) - b * math.sin(angle))
            z[t, :, k] = magnitude * (b * math.cos(angle) + a * math.sin(angle))
    return z


def gated_delta(q, k, v, log_decay, beta, state, offsets, slots, lengths=None, scale=1.0, norm_eps=None, unit=2.0 ** -24,
                floor=0.0):
    """q, k (tokens, k heads, dk), v (tokens, v heads, dv), state (slots, v heads, dk, dv) in fp64. Returns out (NaN in
    rows of no request), the states, and bounds for both of what roundings of `unit` can do: with E the 2-norm of a
    column's error, a step multiplies it by at most e^g (the rest of the step's map, I - beta k k^T, has norm 1 where
    beta |k|^2 <= 2) and adds the roundings of the products with k, of u and of the update. `floor`: what is lost of an operand
    below this part of the largest one of its column so far (state, value or u), in each of k_dim + 64 products."""
    tokens, v_heads, dv = v.shape
    dk, group = k.shape[2], v_heads // k.shape[1]
    if norm_eps is not None:
        q = q / np.sqrt((q * q).sum(-1, keepdims=True) + norm_eps)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + norm_eps)
    out, out_bound = np.full(v.shape, np.nan), np.zeros(v.shape)
    state, bound = np.array(state, np.float64), np.zeros(state.shape)
    for r, slot in enumerate(slots):
        b, e = int(offsets[r]), int(offsets[r + 1])
        if slot < 0 or slot >= len(state) or e <= b:
            continue
        for h in range(v_heads):
            s = np.zeros((dk, dv)) if lengths is not None and lengths[r] <= 0 else state[slot, h]
            err, terms, most = np.zeros(dv), dk + 16, np.abs(s).max(0)
            for t in range(b, e):
                kt, qt, g = k[t, h // group], q[t, h // group], math.exp(log_decay[t, h])
                s = g * s
                said = np.abs(s).T @ np.abs(kt)
                u = beta[t, h] * (v[t, h] - s.T @ kt)
                size = np.linalg.norm(kt)
                s = s + np.outer(kt, u)
                most = np.maximum(most, np.maximum(np.abs(s).max(0), np.maximum(np.abs(v[t, h]), np.abs(u))))
                lost = floor * (dk + 64) * most
                err = g * err + lost + unit * (4 * np.linalg.norm(s, axis=0) + terms * abs(beta[t, h]) * size * (said + np.abs(v[t, h])))
                out[t, h] = scale * (s.T @ qt)
                out_bound[t, h] = abs(scale) * (np.linalg.norm(qt) * (err + lost) + terms * unit * (np.abs(s).T @ np.abs(qt) + np.abs(u) * (np.abs(kt) @ np.abs(qt))))
            state[slot, h], bound[slot, h] = s, err
    return out, state, out_bound, bound


def sample(x, random, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row of logits in fp64; returns the token, its logprob, and how near (as a share of the largest sum) the
    nearest border of a decision was."""
    x = np.where(np.isnan(x), -np.inf, np.array(x, np.float64))
    live = np.flatnonzero(x > -np.inf)
    if not live.size:
        return -1, -np.inf, 1.0
    m = x.max()
    if not temperature > 0:
        return int(np.argmax(x)), 0.0, 1.0
    order = live[np.argsort(-x[live], kind="stable")]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x[order] == m, 1.0, np.exp((x[order] - m) / temperature))
    near = [1.0]
    if top_k > 0:
        order, w = order[:top_k], w[:top_k]
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        total = w.sum()
        near.append(np.min(np.abs(before[1:] / total - max(top_p, 0))) if len(w) > 1 and top_p > 0 else 1.0)
        keep = before < max(top_p, 0) * total
        keep[0] = True
        order, w = order[keep], w[keep]
    if min_p > 0:
        least = min(min_p, 1.0)
        near.append(np.min(np.abs(w - least)[w != 1], initial=1.0))
        order, w = order[w >= least], w[w >= least]
    places = np.argsort(order)
    order, w = order[places], w[places]
    running = np.cumsum(w)
    share = min(max(random, 0.0), 1.0)
    near.append(np.min(np.abs(running / running[-1] - share)[:-1], initial=1.0))
    at = min(int(np.searchsorted(running, share * running[-1], side="right")), len(w) - 1)
    while w[at] == 0:
        at -= 1
    return int(order[at]), float(np.log(w[at] / running[-1])), float(min(near))
