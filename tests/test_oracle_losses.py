"""CPU pins of the oracles of routing on given logits and of the lm_head's losses: hand cases, differences and planted
mistakes."""

import numpy as np
import pytest

from oracle import loss_ref as lr
from oracle import select_ref as sr
from oracle.quant_ref import quantize_ref
from nvfp4_block_scaled_06_amd import workloads as wl


def test_select_hand_case():
    x = np.array([[0.0, np.log(3.0), 0.0, np.log(2.0)]])
    idx, w, _ = sr.select_ref(x, 2, scoring="softmax")
    assert idx.tolist() == [[1, 3]]
    np.testing.assert_allclose(w, [[0.6, 0.4]], rtol=1e-14)
    idx, w, _ = sr.select_ref(x, 3, scoring="softmax", renormalize=False, routed_scale=7.0)
    assert idx.tolist() == [[1, 3, 0]]  # the tie goes to the lower expert
    np.testing.assert_allclose(w, [[3.0, 2.0, 1.0]], rtol=1e-14)
    idx, w, _ = sr.select_ref(x, 2, scoring="sigmoid", bias=[1.0, 0.0, 0.0, 0.0])
    assert idx.tolist() == [[0, 1]]
    np.testing.assert_allclose(w, [[0.5 / 1.25, 0.75 / 1.25]], rtol=1e-14)


def test_groups_hand_case():
    x = np.array([[9.0, 0.0, 5.0, 5.0, 6.0, 3.0]])
    s = 1.0 / (1.0 + np.exp(-x[0]))
    for top, kept in ((1, [0, 2]), (2, [1, 2])):
        score = [np.sort(s[2 * g:2 * g + 2])[-top:].sum() for g in range(3)]
        assert sorted(np.argsort(score)[-2:].tolist()) == kept
        idx, _, _ = sr.select_ref(x, 3, groups=3, topk_groups=2, group_top=top)
        assert set(np.unique(idx // 2)) <= set(kept)
    assert sr.select_ref(x, 1, groups=3, topk_groups=2, group_top=2)[0].tolist() == [[4]]
    assert sr.select_ref(x, 1, groups=3, topk_groups=2, group_top=1)[0].tolist() == [[0]]


def test_masked_rows():
    x = np.array([[-np.inf, 1.0, np.nan, 2.0], [-np.inf] * 4])
    idx, w, _ = sr.select_ref(x, 3)
    assert idx.tolist() == [[3, 1, -1], [-1, -1, -1]]
    assert w[0, 2] == 0.0 and not w[1].any()
    low = np.full((1, 4), np.finfo(np.float32).min)
    for scoring in ("sigmoid", "softmax"):
        idx, w, _ = sr.select_ref(low, 2, scoring=scoring)
        assert idx.tolist() == [[0, 1]] and w.tolist() == [[0.5, 0.5]]


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_select_gradient_is_the_slope(scoring, renorm):
    r = np.random.default_rng(1)
    x, gw = r.standard_normal((3, 10)), r.standard_normal((3, 4))
    kw = dict(scoring=scoring, renormalize=renorm, routed_scale=1.7)
    idx, _, _ = sr.select_ref(x, 4, **kw)
    grad, _ = sr.select_grad_ref(x, idx, gw, **kw)
    h = 1e-6
    for t in range(3):
        for e in range(10):
            d = np.zeros((3, 10))
            d[t, e] = h
            up, down = sr.select_ref(x + d, 4, **kw), sr.select_ref(x - d, 4, **kw)
            assert np.array_equal(up[0], idx) and np.array_equal(down[0], idx)
            slope = ((up[1] - down[1]) * gw).sum() / (2 * h)
            assert abs(slope - grad[t, e]) < 1e-8


def operands(T, D, N, seed=0, scale=1.0):
    r = np.random.default_rng(seed)
    q = lambda rows, s: quantize_ref(wl.bf16_bits((s * r.standard_normal((rows, D))).astype(np.float32)))
    return q(T, scale), q(N, D ** -0.5)


def test_loss_hand_case():
    # x of zeros: every token has probability 1 / N.
    zero = quantize_ref(np.zeros((2, 32), dtype=np.uint16))
    _, wq = operands(1, 32, 8)
    r = lr.loss_ref(zero, wq, np.array([[3], [-100]]))
    np.testing.assert_allclose(r["loss"][0], [np.log(8.0), 0.0], rtol=1e-14)
    np.testing.assert_allclose(r["lse"][0], np.log(8.0), rtol=1e-14)
    w = lr.dequant_ref(*wq)
    np.testing.assert_allclose(r["dx"][0][0], w.mean(axis=0) - w[3], atol=1e-15)
    assert not r["dx"][0][1].any()


def test_a_teacher_of_one_token_is_cross_entropy():
    xq, wq = operands(4, 64, 50, 2)
    tok = np.array([[7], [49], [50], [-1]])
    a = lr.loss_ref(xq, wq, tok)
    b = lr.loss_ref(xq, wq, tok, teacher=np.array([[5.0], [-2.0], [1.0], [0.0]]))
    for k in ("loss", "lse", "logq", "dx"):
        np.testing.assert_allclose(a[k][0], b[k][0], rtol=1e-13, atol=1e-14)


def test_a_teacher_that_is_the_head_has_no_loss():
    xq, wq = operands(3, 64, 20, 3)
    z = lr.dequant_ref(*xq) @ lr.dequant_ref(*wq).T
    for tau in (0.5, 3.0):
        r = lr.loss_ref(xq, wq, np.tile(np.arange(20), (3, 1)), teacher=z, tau=tau)
        assert np.abs(r["loss"][0]).max() < 1e-12 and np.abs(r["dx"][0]).max() < 1e-12


def test_teacher_places_left_out():
    xq, wq = operands(4, 64, 20, 4)
    tok = np.array([[3, -1, 5], [-1, 20, -7], [2, 4, 6], [9, 9, 1]])
    te = np.array([[1.0, np.nan, 2.0], [1.0, 2.0, np.inf], [-np.inf] * 3, [0.5, 1.5, 0.0]])
    r = lr.loss_ref(xq, wq, tok, teacher=te)
    assert r["loss"][0][1] == 0 and r["loss"][0][2] == 0 and not r["dx"][0][1:3].any()
    nan = lr.loss_ref(xq, wq, tok, teacher=np.where(np.arange(4)[:, None] == 3, [np.inf, 0.0, 0.0], te))
    assert np.isnan(nan["loss"][0][3]) and np.isnan(nan["dx"][0][3]).all()
    np.testing.assert_array_equal(nan["loss"][0][:3], r["loss"][0][:3])
    merged = lr.loss_ref(xq, wq, np.array([[9, 1]] * 4), teacher=np.tile([np.logaddexp(0.5, 1.5), 0.0], (4, 1)))
    np.testing.assert_allclose(r["dx"][0][3], merged["dx"][0][3], atol=1e-14)


@pytest.mark.parametrize("tau,teacher", [(1.0, False), (2.5, True)])
def test_loss_gradient_is_the_slope(tau, teacher):
    """Against differences of the loss along the unquantized x (the oracle with x given in float64)."""
    r = np.random.default_rng(5)
    xq, wq = operands(2, 32, 12, 6)
    x, w = lr.dequant_ref(*xq), lr.dequant_ref(*wq)
    tok = np.array([[1, 4], [7, 7]]) if teacher else np.array([[3], [11]])
    te = r.standard_normal((2, 2)) if teacher else None
    g = np.array([0.3, -2.0])

    def total(x):
        z = x @ w.T / tau
        logq = z - lr._lse(z)[:, None]
        p = np.ones((2, 1)) if te is None else np.exp(te / tau) / np.exp(te / tau).sum(axis=1, keepdims=True)
        return (g * tau * tau * (p * (np.log(p) - np.take_along_axis(logq, tok, 1))).sum(axis=1)).sum()

    ref = lr.loss_ref(xq, wq, tok, teacher=te, tau=tau, weight=g)
    assert abs(total(x) - (g * ref["loss"][0]).sum()) < 1e-12
    for t in range(2):
        for d in range(32):
            e = np.zeros_like(x)
            e[t, d] = 1e-6
            slope = (total(x + e) - total(x - e)) / 2e-6
            assert abs(slope - ref["dx"][0][t, d]) < 1e-8


def test_planted_mistakes_are_caught():
    xq, wq = operands(5, 128, 300, 7)
    tok = np.array([[3], [299], [0], [150], [-100]])
    r = lr.loss_ref(xq, wq, tok)
    loss, bound = r["loss"]
    assert not lr.check_outputs("loss", loss, loss, bound)
    for wrong in (loss + 1e-3, np.where(tok[:, 0] < 0, r["lse"][0], loss), np.roll(loss, 1)):
        assert lr.check_outputs("loss", wrong, loss, bound)
    dx, bound = r["dx"]
    q_only = lr.loss_ref(xq, wq, np.array([[-1]] * 5))  # no token at all: all zeros
    w = lr.dequant_ref(*wq)
    for wrong in (dx * 1.02, q_only["dx"][0], dx + 0.05 * np.abs(dx).max(), np.where(np.arange(128) == 17, 0.0, dx),
                  dx + w[3] * (np.arange(5) == 0)[:, None] * 0.02):
        assert lr.check_outputs("dx", wrong, dx, bound)
    assert lr.check_outputs("dx", np.full_like(dx, np.nan), dx, bound)
