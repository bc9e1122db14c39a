"""Penalties, biases and a mask on logits and the greedy token, one token at a time.

TEST INFRASTRUCTURE (CPU oracle); see the package docstring.

``penalize_ref`` evaluates in float64 and returns, with the logits, how far
the fp32 evaluation (each operation rounded by half a step, 2^-24 of its
result) may be from them, the rounding to bf16 apart (2^-8).
"""

import numpy as np

U32 = 2.0 ** -24


def penalize_ref(logits, history=None, prompt=None, lengths=None, repetition=None, frequency=None, presence=None,
                 bias=None, mask=None):
    """(x [T, N] float64, bound [T, N]) for logits [T, N]; bias = (start, token, value), mask 32-bit words."""
    x = np.array(logits, dtype=np.float64)
    err = np.zeros_like(x)
    T, N = x.shape
    with np.errstate(invalid="ignore", over="ignore"):
        for t in range(T):
            r = 1.0 if repetition is None else float(repetition[t])
            f = 0.0 if frequency is None else float(frequency[t])
            p = 0.0 if presence is None else float(presence[t])
            seen, made = set(), {}
            if history is not None:
                L = history.shape[1]
                n = L if lengths is None else min(max(int(lengths[t]), 0), L)
                start = 0 if prompt is None else int(prompt[t])
                for i in range(n):
                    tok = int(history[t, i])
                    if 0 <= tok < N:
                        seen.add(tok)
                        if i >= start:
                            made[tok] = made.get(tok, 0) + 1
            for tok in seen:
                x[t, tok] = x[t, tok] / r if x[t, tok] > 0 else x[t, tok] * r
                err[t, tok] += U32 * abs(x[t, tok])
            for tok, c in made.items():
                x[t, tok] -= f * c
                err[t, tok] += U32 * (abs(f * c) + abs(x[t, tok]))
                x[t, tok] -= p
                err[t, tok] += U32 * abs(x[t, tok])
            if bias is not None:
                last = {}
                for i in range(max(int(bias[0][t]), 0), min(int(bias[0][t + 1]), len(bias[1]))):
                    last[int(bias[1][i])] = float(bias[2][i])
                for tok, v in last.items():
                    if 0 <= tok < N:
                        x[t, tok] += v
                        err[t, tok] += U32 * abs(x[t, tok])
            if mask is not None:
                for n in range(N):
                    if not (int(mask[t][n // 32]) >> (n % 32)) & 1:
                        x[t, n], err[t, n] = -np.inf, 0.0
    return x, 1.01 * err


def penalize_rows(x, history=None, lengths=None, prompt=None, repetition=None, frequency=None, presence=None, bias=None,
                  mask=None):
    """penalize_ref, a row at a time instead of a token at a time: the same operations, for large inputs."""
    x = np.array(x, dtype=np.float64)
    err = np.zeros_like(x)
    T, N = x.shape

    def inside(v):
        return v[(v >= 0) & (v < N)]

    with np.errstate(invalid="ignore", over="ignore"):
        for t in range(T):
            r, f, p = (d if v is None else float(v[t]) for v, d in ((repetition, 1.0), (frequency, 0.0), (presence, 0.0)))
            h = np.zeros(0, dtype=np.int64) if history is None else history[t].astype(np.int64)
            if lengths is not None:
                h = h[:max(int(lengths[t]), 0)]
            seen = np.unique(inside(h))
            v = np.where(x[t, seen] > 0, x[t, seen] / r, x[t, seen] * r)
            x[t, seen] = v
            err[t, seen] += U32 * np.abs(v)
            made, c = np.unique(inside(h[0 if prompt is None else max(int(prompt[t]), 0):]), return_counts=True)
            v = x[t, made] - f * c
            err[t, made] += U32 * (np.abs(f * c) + np.abs(v))
            v = v - p
            x[t, made] = v
            err[t, made] += U32 * np.abs(v)
            if bias is not None:
                a, b = max(int(bias[0][t]), 0), min(int(bias[0][t + 1]), len(bias[1]))
                tok, at = np.unique(bias[1][a:max(a, b)][::-1].astype(np.int64), return_index=True)  # the last of each
                value = bias[2][a:max(a, b)][::-1][at].astype(np.float64)
                ok = (tok >= 0) & (tok < N)
                v = x[t, tok[ok]] + value[ok]
                x[t, tok[ok]] = v
                err[t, tok[ok]] += U32 * np.abs(v)
            if mask is not None:
                words = np.ascontiguousarray(mask[t], dtype=np.uint32).astype("<u4")
                off = np.unpackbits(words.view(np.uint8), bitorder="little")[:N] == 0
                x[t, off], err[t, off] = -np.inf, 0.0
    return x, 1.01 * err


def check_choice(idx, logit, x, err):
    """Failures of the greedy choice: the first maximum, or another token where the fp32 values may order them
    otherwise; -1 and -inf where nothing is above -inf."""
    out = []
    for t in range(x.shape[0]):
        ok = np.nonzero(x[t] > -np.inf)[0]  # NaN compares false
        i = int(idx[t])
        if ok.size == 0:
            if i != -1 or logit[t] != -np.inf:
                out.append(f"row {t}: ({i}, {logit[t]}) for an empty row")
            continue
        best = ok[np.argmax(x[t, ok])]
        if i not in ok:
            out.append(f"row {t}: token {i} is not allowed")
        elif i != best and not x[t, i] >= x[t, best] - err[t, i] - err[t, best] or \
                (i > best and x[t, i] == x[t, best] and err[t, i] == err[t, best] == 0):
            out.append(f"row {t}: token {i} ({x[t, i]!r}) chosen, reference {best} ({x[t, best]!r})")
        elif not (logit[t] == x[t, i] or abs(logit[t] - x[t, i]) <= err[t, i]):
            out.append(f"row {t}: logit {logit[t]!r}, reference {x[t, i]!r}")
    return out
