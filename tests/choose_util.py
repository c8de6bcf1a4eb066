"""64-bit reference of a router's choice and its gradient, from the definitions (numpy)."""
from __future__ import annotations

import numpy as np


def scores(x, scoring):
    """Scores of logits [tokens, E] in 64 bits; masked logits (-infinity) score 0."""
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if scoring == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        top = np.max(x, axis=1, keepdims=True)
        e = np.exp(x - np.where(np.isfinite(top), top, 0.0))
        return e / np.maximum(e.sum(1, keepdims=True), 1e-300)


def _shares(x, scoring):
    """Scores of logits x (finite or +infinity) over their sum, also where every score is zero in 64 bits."""
    log = x if scoring == "softmax" else np.where(x >= 0, -np.log1p(np.exp(-np.abs(x))), np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x))))
    u = np.exp(log - log.max())
    return u / u.sum()


def choose(x, top_k, scoring="softmax", bias=None, groups=1, top_groups=None, group_top=1, renormalise=True, scale=1.0):
    """(ids, weights) of finite or masked logits x [tokens, E]."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    top_groups = groups if top_groups is None else top_groups
    s = scores(x, scoring)
    key = np.where(x == -np.inf, -np.inf, s if bias is None else s + np.asarray(bias, np.float64))
    key = np.where(np.isnan(key), -np.inf, key)
    ids, weights = np.full((T, top_k), -1, np.int32), np.zeros((T, top_k))
    per = E // groups
    for t in range(T):
        allowed = key[t] > -np.inf
        if top_groups < groups:
            total = np.full(groups, -np.inf)
            of = x[t] if bias is None and group_top == 1 else key[t]     # as below: a single score stands in its logit's order
            for g in range(groups):
                best = np.sort(of[g * per:(g + 1) * per])[::-1][:group_top]
                best = best[best > -np.inf]
                if best.size:
                    total[g] = best.sum()
            kept = sorted(range(groups), key=lambda g: (-total[g], g))[:top_groups]
            allowed &= np.isin(np.arange(E) // per, kept)
        # Without a bias the scores stand in the order of the logits, also where 64 bits do not tell them apart.
        order = x[t] if bias is None else key[t]
        best = [e for e in sorted(range(E), key=lambda e: (-order[e], e)) if allowed[e]][:top_k]
        ids[t, :len(best)] = best
        if best:
            w = _shares(x[t, best], scoring) if renormalise else s[t, best]
            weights[t, :len(best)] = scale * w
    return ids, weights


def grad(x, ids, d_weights, scoring="softmax", renormalise=True, scale=1.0):
    """(d_logits, the magnitudes that were added up in each) for the choice `ids` (negative: left out)."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    s = scores(x, scoring)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        js = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E and x[t, ids[t, j]] > -np.inf]
        e = ids[t, js]
        g = scale * np.asarray(d_weights, np.float64)[t, js]
        p = s[t, e]
        if renormalise:
            if not js:
                continue
            u = _shares(x[t, e], scoring)
            factor = u if scoring == "softmax" else u * (1.0 - p)
            for j, ej in enumerate(e):
                d[t, ej] += factor[j] * (g[j] - (u * g).sum())
                mag[t, ej] += factor[j] * (abs(g[j]) + (u * np.abs(g)).sum())
        elif scoring == "sigmoid":
            for j, ej in enumerate(e):
                d[t, ej] += g[j] * p[j] * (1.0 - p[j])
                mag[t, ej] += abs(g[j]) * p[j] * (1.0 - p[j])
        else:
            own, own_mag = np.zeros(E), np.zeros(E)
            np.add.at(own, e, g)
            np.add.at(own_mag, e, np.abs(g))
            d[t] = s[t] * (own - (g * p).sum())
            mag[t] = s[t] * (own_mag + (np.abs(g) * p).sum())
    return d, mag
