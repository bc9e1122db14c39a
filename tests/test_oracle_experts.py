"""CPU pins of the routed experts' and the logits' oracles: hand cases and planted mistakes."""

import numpy as np
import pytest

from conftest import bf16_exact
from oracle import experts_ref as er
from oracle import penalize_ref as pr
from oracle.quant_ref import quantize_ref


def test_plan_hand_case():
    idx = np.array([[2, 0], [0, 5], [-1, 2]])
    off, rows, pos = er.plan_ref(idx, G=3)
    assert off.tolist() == [0, 2, 2, 4]
    assert rows.tolist() == [1, 2, 0, 5, -1, -1]
    assert pos.tolist() == [2, 0, 1, -1, -1, 3]
    off, rows, pos = er.plan_ref(idx, G=1, first_expert=5)
    assert off.tolist() == [0, 1] and rows.tolist() == [3] + 5 * [-1] and pos.tolist() == [-1, -1, -1, 0, -1, -1]


def onehot(rows, D, at, v):
    x = np.zeros((rows, D), dtype=np.uint16)
    for r, (c, val) in enumerate(zip(at, v)):
        x[r, c] = bf16_exact([val])[0]
    return x


def test_swiglu_and_combine_hand_case():
    # x = 6 e0 and 3 e1; one expert, gate row e0 + e1, up row 2 e0: gsa and gsw drop out of one-hot products.
    xq = quantize_ref(onehot(2, 32, [0, 1], [6.0, 3.0]))
    w = np.zeros((2, 32), dtype=np.uint16)
    w[0, 0] = w[0, 1] = bf16_exact([1.0])[0]
    w[1, 0] = bf16_exact([2.0])[0]
    h, err = er.swiglu_ref(xq, [quantize_ref(w)], [0, 2], np.array([0, 1]), k=1)
    assert h.shape == (2, 1)
    np.testing.assert_allclose(h[0, 0], 6.0 / (1 + np.exp(-6.0)) * 12.0, rtol=1e-6)
    assert h[1, 0] == 0.0
    h, _ = er.swiglu_ref(xq, [quantize_ref(w)], [0, 2], np.array([0, 1]), k=1, bias=np.array([[1.0, 0.5]]))
    np.testing.assert_allclose(h[1, 0], 4.0 / (1 + np.exp(-4.0)) * 0.5, rtol=1e-6)
    hq = quantize_ref(onehot(2, 32, [0, 0], [1.0, 2.0]))
    w2 = [quantize_ref(onehot(1, 32, [0], [4.0]))]
    out, _ = er.combine_ref(hq, w2, [0, 2], [1, 0, -1, -1], np.array([[0.5, 2.0], [np.nan, 1.0]]),
                            residual=np.array([[10.0], [7.0]]))
    np.testing.assert_allclose(out, [[10.0 + 0.5 * 8.0 + 2.0 * 4.0], [7.0]], rtol=1e-6)


@pytest.mark.parametrize("plant", ["value", "nan", "none"])
def test_close_check_catches_mistakes(plant):
    rng = np.random.default_rng(3)
    ref = rng.standard_normal((4, 8))
    bound = er.U16 * np.abs(ref)
    dev = ref.copy()
    if plant == "value":
        dev[1, 2] += 2 * bound[1, 2]
    if plant == "nan":
        dev[1, 2] = np.nan
    assert bool(er.check_close("x", dev, ref, bound)) == (plant != "none")


def test_penalize_hand_case():
    x = np.array([[4.0, -4.0, 1.0, 2.0, 0.5]])
    hist = np.array([[0, 1, 2, 2, 9, -3]])
    out, err = pr.penalize_ref(x, history=hist, prompt=[2], repetition=[2.0], frequency=[0.25], presence=[1.0],
                               bias=([0, 3], [4, 4, 7], [9.0, 3.0, 1.0]), mask=[[0b10111]])
    assert out[0, :3].tolist() == [2.0, -8.0, 0.5 - 0.5 - 1.0]  # token 2: made twice
    assert out[0, 3] == -np.inf and out[0, 4] == 3.5  # the last of the repeated biases
    assert not pr.check_choice([4], [3.5], out, err)
    assert pr.check_choice([3], [2.0], out, err) and pr.check_choice([0], [2.0], out, err)
    empty, e = pr.penalize_ref(x, mask=[[0]])
    assert not pr.check_choice([-1], [-np.inf], empty, e) and pr.check_choice([0], [4.0], empty, e)
    tie, e = pr.penalize_ref(np.array([[1.0, 3.0, 3.0]]))
    assert not pr.check_choice([1], [3.0], tie, e) and pr.check_choice([2], [3.0], tie, e)


@pytest.mark.parametrize("T,N,L,nbias,mask", [(3, 70, 90, 40, True), (2, 33, 5, 0, True), (4, 64, 0, 12, False),
                                              (3, 40, 300, 80, False)])
def test_penalize_by_rows_is_penalize(T, N, L, nbias, mask):
    rng = np.random.default_rng(N)
    x = 3 * rng.standard_normal((T, N))
    x[0, :3] = np.nan, np.inf, -np.inf
    a = dict(repetition=rng.uniform(0.8, 1.5, T), frequency=rng.uniform(-0.5, 0.5, T), presence=rng.uniform(-1, 1, T))
    if L:
        a.update(history=rng.integers(-2, N + 2, (T, L)), lengths=rng.integers(-1, L + 3, T),
                 prompt=rng.integers(-1, L + 3, T))
    if nbias:
        start = np.concatenate([[0], np.cumsum(rng.integers(0, nbias, T))])
        start[1] = -3  # an empty row, and one from the list's beginning
        a["bias"] = (start, rng.integers(-1, N + 1, start[-1]), rng.standard_normal(start[-1]))
    if mask:
        a["mask"] = rng.integers(0, 2 ** 32, (T, (N + 31) // 32), dtype=np.uint32)
    for got, want in zip(pr.penalize_rows(x, **a), pr.penalize_ref(x, **a)):
        np.testing.assert_array_equal(got, want)
