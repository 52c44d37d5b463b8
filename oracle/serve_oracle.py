"""Plain float64 definitions of the operators around the span attention: norms with rotation, attention mass, the choice
of kept positions, log probabilities.  Test infrastructure only; shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np


def norm_rope(x, weight, eps, positions, theta):
    """x [T, H, d], positions [T]: every head row over its root mean square, times weight (None: not normalised), turned
    (element j < d/2 with element j + d/2) by position * theta^(-2j/d)."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    w = float(theta) ** (-2.0 * np.arange(d // 2) / d)
    angle = np.asarray(positions, np.float64)[:, None, None] * w
    a, b = x[..., :d // 2], x[..., d // 2:]
    return np.concatenate([a * np.cos(angle) - b * np.sin(angle), b * np.cos(angle) + a * np.sin(angle)], -1)


def attn_mass(q, keys, prefix, intervals, old, decay, scale=None):
    """New mass [P + L, h_kv] of every question: keys[i] [P_i + L_i, h_kv, d], old[i] the same shape without d.  Also the
    largest sum of |q_e k_e| * scale that a visible score has (for error bounds)."""
    out, top = [], 0.0
    h_q, d = q.shape[1:]
    scale = 1 / np.sqrt(d) if scale is None else scale
    for (b, e), p, k, o in zip(intervals, prefix, keys, old):
        m, h_kv = int(e - b), k.shape[1]
        if m == 0:
            out.append(np.array(o, np.float64))
            continue
        g = h_q // h_kv
        new = np.zeros((p + m, h_kv))
        for t in range(m):
            for h in range(h_q):
                kk = k[:p + t + 1, h // g]
                z = kk @ q[b + t, h] * scale
                top = max(top, float((np.abs(kk) @ np.abs(q[b + t, h])).max() * scale))
                w = np.exp(z - z.max())
                new[:p + t + 1, h // g] += w / w.sum()
        if decay:
            new[:p] += decay * np.asarray(o, np.float64)[:p]
        out.append(new)
    return out, top


def select(mass, keep, first, last):
    """Kept positions, ascending, of one question's mass [n, h_kv]: [h_kv, min(n, keep)]."""
    n, h_kv = mass.shape
    if n <= keep:
        return np.tile(np.arange(n), (h_kv, 1))
    res = []
    for g in range(h_kv):
        middle = list(range(first, n - last))
        # NaN above everything, then larger masses, then lower positions
        middle.sort(key=lambda u: (not np.isnan(mass[u, g]), -mass[u, g] if not np.isnan(mass[u, g]) else 0.0, u))
        res.append(sorted(list(range(first)) + middle[:keep - first - last] + list(range(n - last, n))))
    return np.array(res)


def logprobs(logits, temperature, tokens, top_n):
    """(log probabilities of the tokens, entropies, top tokens, their log probabilities); NaN and -1 for rows without a
    distribution."""
    x = np.asarray(logits, np.float64)
    n, v = x.shape
    lp, ent = np.full(n, np.nan), np.full(n, np.nan)
    top, top_lp = np.full((n, top_n), -1), np.full((n, top_n), np.nan)
    for r in range(n):
        if np.isnan(x[r]).any() or x[r].max() in (np.inf, -np.inf):
            continue
        t = 1.0 if temperature is None else float(temperature[r])
        if t == 0:
            y = np.full(v, -np.inf)
            y[np.argmax(x[r])] = 0.0
        else:
            y = (x[r] - x[r].max()) / t
            y = y - np.log(np.exp(y).sum())
        p = np.exp(y)
        lp[r] = y[tokens[r]]
        ent[r] = -(p[p > 0] * y[p > 0]).sum()
        top[r] = np.lexsort((np.arange(v), -x[r]))[:top_n]
        top_lp[r] = y[top[r]]
    return lp, ent, top, top_lp
