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
