"""The routed experts on rows sorted by expert, written as their plain definitions.

TEST INFRASTRUCTURE (CPU oracle); see the package docstring.

Slot s = t * k + j is token t's j-th choice. ``plan_ref`` lists each expert's
slots one by one; ``swiglu_ref`` and ``combine_ref`` work on dequantized
float64 values and also return how far a correct fp32 evaluation may be off:

* a sum of n exact products, each fp32 addition rounding by half a step
  (2^-24 relative to a partial sum, which A = sum |products| bounds):
  n 2^-24 A; the scale factor, its product and the bias addition: three more
  roundings of at most 2^-24 A + 2^-24 |bias|;
* silu'(g) lies in [-0.1, 1.1], so an error dg of the gate moves silu(g) u by
  at most 1.1 dg |u|, an error du by |silu(g)| du;
* silu itself from a hardware exponential and reciprocal (one unit each) of
  g log2(e), whose rounding |g| 2^-24 is a relative error of e^-g; two
  products: (|g| + 5) 2^-23 relative;
* the rounding to bf16: half a step, 2^-8 relative (2^-134 where the result
  is subnormal).
"""

import numpy as np

from .quant_ref import dequant_ref

U32 = 2.0 ** -24
U16 = 2.0 ** -8
TINY = 2.0 ** -133


def plan_ref(topk_idx, G, first_expert=0):
    """(offsets [G + 1], rows [T * k], pos [T * k]) of the slots sorted by expert."""
    flat = [int(v) - first_expert for v in np.asarray(topk_idx).reshape(-1)]
    lists = [[] for _ in range(G)]
    for s, e in enumerate(flat):
        if 0 <= e < G:
            lists[e].append(s)
    rows = [s for lst in lists for s in lst]
    offsets = np.cumsum([0] + [len(lst) for lst in lists])
    pos = np.full(len(flat), -1)
    for p, s in enumerate(rows):
        pos[s] = p
    return offsets, np.array(rows + [-1] * (len(flat) - len(rows)), dtype=np.int64), pos


def _product(x, w, bias):
    """(y, bound of y's error) for exact fp32-accumulated products of dequantized x [n, K] and w [N, K]."""
    y, A = x @ w.T, np.abs(x) @ np.abs(w).T
    err = (x.shape[1] + 3) * U32 * A
    if bias is not None:
        b = np.asarray(bias, dtype=np.float64)
        y, err = y + b, err + U32 * (A + np.abs(b))
    return y, err


def _silu(g):
    return g / (1.0 + np.exp(np.minimum(-g, 700.0)))


def swiglu_ref(xq, wq, offsets, rows, k, bias=None):
    """(h [R, F], bound [R, F]); xq the tokens' NVFP4 tuple, wq one tuple [2F, D] per expert."""
    x = dequant_ref(*xq)
    R, F = len(rows), wq[0][0].shape[0] // 2
    h, err = np.zeros((R, F)), np.zeros((R, F))
    for g in range(len(wq)):
        a, b = int(offsets[g]), int(offsets[g + 1])
        if a == b:
            continue
        y, d = _product(x[np.asarray(rows[a:b]) // k], dequant_ref(*wq[g]), None if bias is None else bias[g])
        gate, up, dg, du = y[:, :F], y[:, F:], d[:, :F], d[:, F:]
        s = _silu(gate)
        h[a:b] = s * up
        e = 1.1 * dg * (np.abs(up) + du) + np.abs(s) * du + (np.abs(gate) + 5) * 2 * U32 * np.abs(s * up)
        err[a:b] = e + U16 * (np.abs(h[a:b]) + e) + TINY
    return h, err


def combine_ref(hq, wq, offsets, pos, topk_w, bias=None, residual=None):
    """(out [T, N], bound [T, N]); hq the sorted rows' NVFP4 tuple, wq one tuple [N, F] per expert."""
    h = dequant_ref(*hq)
    T, k = topk_w.shape
    N = wq[0][0].shape[0]
    y, err = np.zeros((h.shape[0], N)), np.zeros((h.shape[0], N))
    for g in range(len(wq)):
        a, b = int(offsets[g]), int(offsets[g + 1])
        if a < b:
            y[a:b], err[a:b] = _product(h[a:b], dequant_ref(*wq[g]), None if bias is None else bias[g])
    out = np.zeros((T, N)) if residual is None else np.array(residual, dtype=np.float64)
    mag, d = np.abs(out), np.zeros((T, N))
    for t in range(T):
        for j in range(k):
            p = int(pos[t * k + j])
            if p >= 0:
                w = float(topk_w[t, j])
                out[t] += w * y[p]
                mag[t] += np.abs(w * y[p])
                d[t] += abs(w) * err[p]
    d += 2 * (k + 1) * U32 * mag
    return out, d + U16 * (np.abs(out) + d) + TINY


def check_close(name, dev, ref, bound, limit=8):
    """Failures (empty == pass) of |dev - ref| <= bound; NaN fails."""
    dev = np.asarray(dev, dtype=np.float64)
    if dev.shape != ref.shape:
        return [f"{name}: shape {dev.shape} != {ref.shape}"]
    bad = np.argwhere(~(np.abs(dev - ref) <= bound))
    out = [f"{name}{[int(i) for i in p]}: dev {dev[tuple(p)]!r} ref {ref[tuple(p)]!r} bound {bound[tuple(p)]!r}"
           for p in bad[:limit]]
    return out + ([f"{name}: {len(bad)} of {dev.size} outside the bound"] if len(bad) > limit else [])
