"""Routing on given logits and its gradient, one row at a time in float64.

TEST INFRASTRUCTURE (CPU oracle); see the package docstring.

``select_ref`` and ``select_grad_ref`` return, with their values, how far an
fp32 evaluation may be from them. U32 = 2^-24 is half a step of fp32; an
exponential of an fp32 argument a is off by |a| U32 for the argument's
rounding and by 2 U32 for its own; sums of n terms by n U32.
"""

import numpy as np

U32 = 2.0 ** -24


def scores_ref(row, scoring):
    """float64 scores of one row; masked logits (-inf, NaN) score 0."""
    x = np.where(np.isnan(row), -np.inf, np.asarray(row, dtype=np.float64))
    with np.errstate(over="ignore", invalid="ignore"):
        if scoring == "sigmoid":
            return x, np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))
        m = x.max()
        if not np.isfinite(m):
            return x, np.zeros_like(x)
        e = np.exp(x - m)
        return x, e / e.sum()


def choose_ref(key, x, k, groups=1, topk_groups=1, group_top=2):
    """Experts by descending key, equal ones by descending logit x, then the lower one, inside the best groups (by score,
    equal ones by the logit where that is one expert's key, then the lower one); keys of -inf are never chosen."""
    key = np.array(key, dtype=np.float64)
    if topk_groups < groups:
        g, l = key.reshape(groups, -1), x.reshape(groups, -1)
        best = np.lexsort((-l, -g), axis=1)[:, :group_top]  # stable: what is left goes to the lower one
        with np.errstate(invalid="ignore"):
            score = np.take_along_axis(g, best, 1).sum(axis=1)
        score = np.where(np.isnan(score), -np.inf, score)
        one = np.full(groups, -np.inf)
        if best.shape[1] == 1:
            one = np.where(score > -np.inf, np.take_along_axis(l, best, 1)[:, 0], -np.inf)
        out = np.ones(groups, dtype=bool)
        out[np.lexsort((-one, -score))[:topk_groups]] = False
        key = np.where(np.repeat(out, g.shape[1]), -np.inf, key)
    order = np.lexsort((-x, -key))[:k].tolist()
    return [i if key[i] > -np.inf else -1 for i in order] + [-1] * (k - len(order))


def _shares(x, idx, scoring):
    """Shares of the chosen scores in their sum, for any finite logits, and the span of the exponents."""
    l = x[idx]
    base = l if scoring == "softmax" else np.minimum(l, 0.0)
    m = base.max()
    num = np.exp(base - m)
    if scoring == "sigmoid":
        num = num / (1.0 + np.exp(-np.abs(l)))
    return num / num.sum(), float(np.max(np.abs(base - m))) + (0.0 if scoring == "softmax" else float(np.max(np.abs(l))))


def select_ref(logits, k, bias=None, scoring="sigmoid", groups=1, topk_groups=1, group_top=2, renormalize=True,
               routed_scale=1.0):
    """(idx [T, k], w [T, k] float64, bound [T, k]) for logits [T, E]."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    idx = np.full((T, k), -1, dtype=np.int64)
    w, bound = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        x, s = scores_ref(logits[t], scoring)
        key = np.where(x > -np.inf, s + (0.0 if bias is None else np.asarray(bias, np.float64)), -np.inf)
        key = np.where(np.isnan(key), -np.inf, key)
        idx[t] = choose_ref(key, x, k, groups, topk_groups, group_top)
        c = idx[t] >= 0
        if not c.any():
            continue
        e = idx[t][c]
        if renormalize:
            share, span = _shares(x, e, scoring)
            w[t, c] = routed_scale * share
            rel = 2 * span + k + 16
        else:
            w[t, c] = routed_scale * s[e]
            # softmax: the sum of E exponentials, each weighed by its own size
            live = x > -np.inf
            rel = 2 * np.max(np.abs(x[e] - (x.max() if scoring == "softmax" else 0))) + 16
            if scoring == "softmax":
                rel += 2 * float((s[live] * (x.max() - x[live])).sum()) + 44
        bound[t, c] = np.abs(w[t, c]) * rel * U32 + 2.0 ** -126
    return idx, w, bound


def select_grad_ref(logits, idx, grad_w, scoring="sigmoid", renormalize=True, routed_scale=1.0):
    """(grad_logits [T, E] float64, bound) of the weights of the choice idx; places outside [0, E) take no part."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    out, bound = np.zeros((T, E)), np.zeros((T, E))
    c = abs(routed_scale)
    for t in range(T):
        ok = (idx[t] >= 0) & (idx[t] < E)
        e, g = idx[t][ok], np.asarray(grad_w[t], dtype=np.float64)[ok]
        x, s = scores_ref(logits[t], scoring)
        live = x > -np.inf
        k = len(e)
        span = 2 * float(np.max(np.abs(x[e][x[e] > -np.inf]), initial=0.0)) + k + 24
        if scoring == "softmax" and not renormalize:
            if not live.any():
                continue
            dot = (g * s[e]).sum()
            out[t] = -routed_scale * s * dot
            np.add.at(out[t], e, routed_scale * s[e] * g)
            mag = s * (np.abs(g) * s[e]).sum()
            np.add.at(mag, e, s[e] * np.abs(g))
            span = 4 * float(np.max(x.max() - x[live])) + 64 + k
            bound[t] = c * mag * span * U32
            continue
        alive = x[e] > -np.inf
        e, g = e[alive], g[alive]
        if not len(e):
            continue
        if renormalize:
            u, sp = _shares(x, e, scoring)
            r = routed_scale * u * (g - (u * g).sum())
            mag = c * u * (np.abs(g) + 2 * (u * np.abs(g)).sum())
            span += 2 * sp
        else:
            u = s[e]
            r, mag = routed_scale * u * g, c * u * np.abs(g)
        if scoring == "sigmoid":
            down = scores_ref(-x[e], "sigmoid")[1]
            r, mag = r * down, mag * down
        np.add.at(out[t], e, r)
        np.add.at(bound[t], e, 2 * mag * span * U32)
    # Scores below fp32's normal numbers, 2^-126, may come out as 0 (the base-2 exponential flushes them), and then take
    # scale (gw - dot) times as much from a gradient, dot being at most the sum of the |gw| that take part.
    ok = (np.asarray(idx) >= 0) & (np.asarray(idx) < E)
    total = np.where(ok, np.abs(np.nan_to_num(np.asarray(grad_w, dtype=np.float64))), 0.0).sum(axis=1, keepdims=True)
    return out, bound + 2.0 ** -126 * (1.0 + 2.0 * c * total)
