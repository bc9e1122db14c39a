"""GPU tests of router_select where its order is hard to decide: large keys that cancel, saturated scores, infinite biases."""

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_06_amd import router as rt
from oracle import loss_ref as lr
from oracle import select_ref as sr

pytestmark = pytest.mark.gpu

def log(msg):
    print(f"[gpu-select-limits] {msg}", flush=True)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    rt.load_library()
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def up(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def check(x, b, k, got, **kw):
    idx, w = got[0].cpu().numpy(), got[1].cpu().numpy()
    ref, rw, bound = sr.select_ref(x, k, bias=b, **kw)
    bad = np.argwhere((idx != ref).any(axis=1))[:, 0]
    assert not len(bad), (len(bad), bad[:5], idx[bad[:3]], ref[bad[:3]])
    fails = lr.check_outputs("w", w, rw, bound)
    assert not fails, "\n".join(fails)


# A wavefront to a row, and four rows to one.
ROWS = [3, 6200]


@pytest.mark.parametrize("T", [4000, 6200])
@pytest.mark.parametrize("big", [64.0, 1e4])
def test_group_border_of_keys_that_cancel(dev, T, big):
    """Groups of one forced and one banned expert: their scores, the sums of two large keys, are about 1 and differ by
    steps of the keys' own size in 32 bits, or less."""
    G = 16
    r = np.random.default_rng(int(big) + T)
    x = np.empty((T, 2 * G))
    s1 = r.uniform(0.2, 0.8, (T, G))
    s2 = 1.1 - s1 + r.uniform(-0.5, 0.5, (T, G)) * big * 2.0 ** -20
    x[:, 0::2], x[:, 1::2] = np.log(s1 / (1 - s1)), np.log(s2 / (1 - s2))
    x = x.astype(np.float32)
    b = np.tile([big, -big], G).astype(np.float32)
    kw = dict(groups=G, topk_groups=5, group_top=2)
    log(f"border T={T} big={big}")
    got = rt.select(up(x, dev), 8, bias=up(b, dev), **kw)
    torch.cuda.synchronize()
    check(x, b, 8, got, **kw)


def saturated(T, E, scoring, seed):
    """Rows of which many scores, or all, are the same number in 64 bits although their logits differ, and some not."""
    r = np.random.default_rng(seed)
    x = r.uniform(38.0, 60.0, (T, E)) if scoring == "sigmoid" else r.uniform(-1200.0, -900.0, (T, E))
    x = np.round(x * 8) / 8  # equal logits too
    x[:, ::7] = r.uniform(-2.0, 2.0, x[:, ::7].shape)
    x[T // 2:, 1::3] = -np.inf
    if scoring == "softmax":
        x[:, 3] = 1.0
    return x.astype(np.float32)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k", [(3, 48, 12), (4, 256, 8), (5, 500, 32), (2100, 48, 12), (6200, 256, 8), (6200, 384, 16)])
def test_saturated_scores(dev, T, E, k, scoring):
    """Equal keys go to the larger logit, so a bias of zeros chooses what no bias chooses: the order of the logits."""
    x = saturated(T, E, scoring, T + E)
    log(f"saturated T={T} E={E} k={k} {scoring}")
    zeros = torch.zeros(E, device=dev)
    want = np.argsort(np.where(x > -np.inf, -x, np.inf), axis=1, kind="stable")[:, :k]
    for groups, kept, top in ((1, 1, 1), (4, 2, 1), (4, 4, 2)):
        if k > kept * (E // groups):
            continue
        kw = dict(scoring=scoring, groups=groups, topk_groups=kept, group_top=top, renormalize=False)
        a, b = rt.select(up(x, dev), k, **kw), rt.select(up(x, dev), k, bias=zeros, **kw)
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0])
        if kept == groups:
            assert np.array_equal(a[0].cpu().numpy(), want)
        check(x, None, k, a, **kw)  # each row count has its own order of sums, so the weights are not the same bits
        check(x, np.zeros(E, np.float32), k, b, **kw)
    if E % 4 == 0 and k <= E // 2:  # sums of two saturated scores
        kw = dict(scoring=scoring, groups=4, topk_groups=2, group_top=2)
        a, b = rt.select(up(x, dev), k, **kw), rt.select(up(x, dev), k, bias=zeros, **kw)
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0])
        check(x, None, k, a, **kw)


@pytest.mark.parametrize("T", ROWS)
def test_equal_keys_of_different_biases(dev, T):
    """A key that is the same number in 64 bits by a larger score and a smaller bias: the larger logit comes first."""
    x = np.tile(np.array([0.0, 50.0, 50.0, 0.0, 60.0, -np.inf], np.float32), (T, 4))
    b = np.tile(np.array([1.0, 0.5, 0.5, 1.0, 0.5, 3.0], np.float32), 4)
    log(f"equal keys T={T}")
    for kw in (dict(), dict(groups=4, topk_groups=2, group_top=1), dict(groups=2, topk_groups=1, group_top=2)):
        got = rt.select(up(x, dev), 7, bias=up(b, dev), **kw)
        torch.cuda.synchronize()
        check(x, b, 7, got, **kw)
        if not kw:
            assert got[0].cpu().numpy().tolist() == [[4, 10, 16, 22, 1, 2, 7]] * T


@pytest.mark.parametrize("k", [1, 4, 9])
@pytest.mark.parametrize("T", ROWS)
def test_infinite_biases(dev, T, k):
    """Experts forced by a bias of +infinity, as many as are chosen, fewer and more; banned and masked ones beside them."""
    E = 128
    x = np.random.default_rng(k).standard_normal((T, E)).astype(np.float32)
    for forced in (1, 4, 9, 40, 128):
        log(f"infinite biases T={T} k={k} forced={forced}")
        b = np.zeros(E, np.float32)
        b[np.random.default_rng(forced).permutation(E)[:forced]] = np.inf
        b[5] = -np.inf
        x[:, 11] = -np.inf
        for kw in (dict(), dict(scoring="softmax"), dict(groups=8, topk_groups=3, group_top=2),
                   dict(groups=8, topk_groups=3, group_top=1)):
            got = rt.select(up(x, dev), k, bias=up(b, dev), **kw)
            torch.cuda.synchronize()
            check(x, b, k, got, **kw)


@pytest.mark.parametrize("T", ROWS)
def test_infinite_logits(dev, T):
    """+infinity is the largest logit; softmax scores of its row are NaN, and other rows do not feel it."""
    E, k = 64, 4
    x = np.random.default_rng(1).standard_normal((T, E)).astype(np.float32)
    x[1, 20] = np.inf
    rest = [t for t in range(T) if t != 1]
    for bias in (None, torch.zeros(E, device=dev)):
        got = rt.select(up(x, dev), k, bias=bias)
        torch.cuda.synchronize()
        check(x, None, k, got)
        idx, w = rt.select(up(x, dev), k, bias=bias, scoring="softmax")
        torch.cuda.synchronize()
        if bias is None:
            assert idx[1].tolist() == got[0][1].tolist() and torch.isnan(w[1]).all()
        else:
            assert (idx[1] == -1).all() and not w[1].any()
        check(x[rest], None, k, (idx[rest], w[rest]), scoring="softmax")


@pytest.mark.parametrize("T", ROWS)
def test_biases_of_the_lowest_value(dev, T):
    """Experts banned by the type's lowest value and by less: sums of two such keys, beyond 32 bits, still have an order, and
    come before groups of masked experts."""
    G, E = 8, 32
    low = np.finfo(np.float32).min
    x = np.random.default_rng(T).standard_normal((T, E)).astype(np.float32)
    b = np.full(E, low, np.float32)
    b[20:22] = low / 2   # group 5: the largest of the sums
    b[26] = low / 3      # group 6: the second
    x[:, 0:4] = -np.inf  # group 0: nothing to choose
    log(f"lowest biases T={T}")
    for kept, top in ((1, 2), (2, 2), (7, 2), (2, 1)):
        kw = dict(groups=G, topk_groups=kept, group_top=top)
        got = rt.select(up(x, dev), 4, bias=up(b, dev), **kw)
        torch.cuda.synchronize()
        check(x, b, 4, got, **kw)
