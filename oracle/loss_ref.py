"""Losses of the lm_head over its whole vocabulary and their gradient, in float64 with all logits at hand.

TEST INFRASTRUCTURE (CPU oracle); see the package docstring.

``loss_ref`` returns each output with a bound on how far an evaluation may be
from it that sums exact products in fp32 (half a step U32 = 2^-24 each),
keeps the columns' softmax weights as fp16 times 2^15, rounded once (UF16 =
2^-11, and 2^-25 / 2^15 below fp16's range, at the block's scale and at the
row's, which is less than twice the largest weight: 3 2^-40 of that in all)
and rounds dx to bf16 (2^-8).
"""

import numpy as np

from .quant_ref import dequant_ref

U32, UF16, UBF16 = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8


def _lse(z):
    m = z.max(axis=1, keepdims=True)
    return m[:, 0] + np.log(np.exp(z - m).sum(axis=1))


def loss_ref(xq, wq, tokens, teacher=None, tau=1.0, weight=None):
    """dict of (value, bound): loss, lse, logq, dx; xq and wq are (codes, scales, global scale), tokens [T, K].

    Without a teacher K is 1 and the token has probability 1 (cross entropy). Tokens outside [0, N) are left out."""
    x, w = dequant_ref(*xq), dequant_ref(*wq)
    tokens = np.asarray(tokens)
    T, D = x.shape
    N, K = w.shape[0], tokens.shape[1]
    z = x @ w.T / tau
    ez = (D + 8) * U32 * (np.abs(x) @ np.abs(w).T) / tau  # sums of D products, and the factors' roundings
    lse = _lse(z)
    mag = np.abs(z).max(axis=1)
    elog = ez.max(axis=1) + (3 * mag + 64 + N / 64) * U32
    else_ = elog + 4 * U32 * np.abs(lse)
    valid = (tokens >= 0) & (tokens < N)
    at = np.where(valid, tokens, 0)
    rows = np.arange(T)[:, None]
    logq = np.where(valid, z[rows, at] - lse[:, None], 0.0)
    elogq = np.where(valid, ez[rows, at] + else_[:, None] + 2 * U32 * (np.abs(z[rows, at]) + np.abs(lse[:, None])), 0.0)
    none = np.zeros(T, dtype=bool)
    if teacher is None:
        p, logp, ep = valid.astype(np.float64), np.zeros((T, K)), np.zeros((T, K))
        used = valid.any(axis=1)
    else:
        t = np.where(valid, np.asarray(teacher, dtype=np.float64) / tau, -np.inf)
        none = (np.isnan(t) | (t == np.inf)).any(axis=1)  # rows whose loss and gradient are NaN
        t = np.where(none[:, None], 0.0, t)
        m = t.max(axis=1, keepdims=True)
        used = np.isfinite(m[:, 0])
        m = np.where(np.isfinite(m), m, 0.0)
        e = np.exp(t - m)
        s = np.where(used, e.sum(axis=1), 1.0)[:, None]
        p = np.where(used[:, None], e / s, 0.0)
        with np.errstate(divide="ignore"):
            logp = np.where(p > 0, np.where(valid, t, 0.0) - m - np.log(s), 0.0)
        # relative, of p; the quotients t / tau round too
        span = np.where(np.isfinite(t), np.abs(t) + np.abs(m), 0.0)
        ep = (2 * span + K + 16) * U32
    diff = np.where(p > 0, logp - logq, 0.0)
    loss = tau * tau * (p * diff).sum(axis=1) * used
    eloss = tau * tau * (p * (np.abs(diff) * (ep + (K + 8) * U32) + ep + 2 * U32 * np.abs(logp) + elogq)).sum(axis=1) * used
    # gradient
    g = np.ones(T) if weight is None else np.asarray(weight, dtype=np.float64)
    q = np.exp(z - lse[:, None])
    named = np.zeros((T, N), dtype=bool)
    for j in range(K):
        named[np.arange(T)[valid[:, j]], at[:, j][valid[:, j]]] = True
    c = q.copy()
    np.add.at(c, (np.broadcast_to(rows, (T, K)), at), np.where(valid, -p, 0.0))
    eq = q * (UF16 + 2 * elog[:, None] + ez + (mag[:, None] + 64) * U32) + 2.0 ** -40 * q.max(axis=1, keepdims=True) * 3
    ec = np.where(named, q * (2 * else_[:, None] + ez + 8 * U32), eq)
    np.add.at(ec, (np.broadcast_to(rows, (T, K)), at), np.where(valid, p * (ep + 4 * U32), 0.0))
    aw = np.abs(w)
    f = (tau * g * used)[:, None]
    dx = f * (c @ w)
    total = q.copy()
    np.add.at(total, (np.broadcast_to(rows, (T, K)), at), np.where(valid, p, 0.0))
    edx = np.abs(f) * ((ec + (N + K + 16) * U32 * total) @ aw)
    edx = edx + UBF16 * (np.abs(dx) + edx) + 2.0 ** -133  # and below bf16's normal numbers
    loss, dx = np.where(none, np.nan, loss), np.where(none[:, None], np.nan, dx)
    return {"loss": (loss, eloss + 2.0 ** -126), "lse": (lse, else_), "logq": (logq, elogq + 2.0 ** -126), "dx": (dx, edx)}


def check_outputs(name, got, want, bound, limit=8):
    """Failures (empty == pass) of got against want within bound; NaN where the other has none fails."""
    got = np.asarray(got, dtype=np.float64)
    if got.shape != want.shape:
        return [f"{name}: shape {got.shape} != {want.shape}"]
    bad = np.argwhere(~((np.abs(got - want) <= bound) | (np.isnan(got) & np.isnan(want))))
    return [f"{name}{[int(i) for i in b]}: {got[tuple(b)]!r} want {want[tuple(b)]!r} +- {np.broadcast_to(bound, want.shape)[tuple(b)]:.3g}"
            for b in bad[:limit]] + ([f"{name}: {len(bad)} in all"] if len(bad) > limit else [])
