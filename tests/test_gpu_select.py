"""GPU parity of router_select and router_select_backward against the CPU oracle, through the C ABI."""

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_06_amd import router as rt
from nvfp4_block_scaled_06_amd import workloads as wl
from oracle import loss_ref as lr
from oracle import select_ref as sr

pytestmark = pytest.mark.gpu
UBF16 = 2.0 ** -8


def log(msg):
    print(f"[gpu-select] {msg}", flush=True)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    rt.load_library()
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def make(T, E, dtype, seed, kind="normal", bias=True):
    r = np.random.default_rng(seed)
    x = (1.5 * r.standard_normal((T, E))).astype(np.float32)
    if kind == "wide":
        x *= 30.0
    elif kind == "equal":
        x[:] = 0.25
    elif kind == "few":  # a handful of values: ties everywhere
        x = np.round(x).astype(np.float32)
    elif kind == "masked":
        x[r.random((T, E)) < 0.9] = -np.inf
        x[r.random((T, E)) < 0.02] = np.nan
        x[0] = -np.inf
        x[-1] = np.finfo(np.float32).min
    elif kind == "near":  # keys closer than fp32 tells apart, and their ties
        x = (1.0 + r.integers(0, 40, (T, E)) * 2.0 ** -23).astype(np.float32)
    if dtype == torch.bfloat16:
        with np.errstate(over="ignore", invalid="ignore"):
            x = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
    b = (0.001 * r.integers(-100, 101, E)).astype(np.float32) if bias else None
    return x, b


def up(a, dev, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    return t if dtype is None else t.to(dtype)


def check(x, b, k, got, kw):
    idx, w = got[0].cpu().numpy(), got[1].cpu().numpy()
    ref, rw, bound = sr.select_ref(x, k, bias=b, **kw)
    bad = np.argwhere((idx != ref).any(axis=1))[:, 0]
    assert not len(bad), (bad[:5], idx[bad[:3]], ref[bad[:3]])
    fails = lr.check_outputs("w", w, rw, bound)
    assert not fails, "\n".join(fails)


def check_grad(x, idx, gw, got, kw, dtype):
    ref, bound = sr.select_grad_ref(x, idx, gw, **kw)
    if dtype == torch.bfloat16:
        bound = bound + UBF16 * (np.abs(ref) + bound) + 2.0 ** -133
    fails = lr.check_outputs("grad", got.float().cpu().numpy(), ref, bound)
    assert not fails, "\n".join(fails)


RULES = [dict(scoring="sigmoid"), dict(scoring="softmax"), dict(scoring="sigmoid", renormalize=False, routed_scale=0.7),
         dict(scoring="softmax", renormalize=False, routed_scale=2.5)]


@pytest.mark.parametrize("rule", range(4))
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 5, 5), (3, 33, 32), (2, 64, 8), (1, 128, 6), (5, 200, 17),
                                   (1, 256, 8), (2, 385, 9), (7, 512, 32), (1024, 16, 4), (1025, 61, 13), (1100, 96, 6),
                                   (1030, 130, 8), (2050, 256, 8), (1029, 384, 8), (1024, 510, 16), (1027, 260, 32)])
def test_parity(dev, T, E, k, rule):
    kw = RULES[rule]
    for dtype, bias in ((torch.float32, True), (torch.float32, False), (torch.bfloat16, rule % 2 == 0)):
        x, b = make(T, E, dtype, 100 * T + E + rule, bias=bias)
        log(f"parity T={T} E={E} k={k} {kw} {dtype} bias={bias}")
        xd = up(x, dev, dtype)
        got = rt.select(xd, k, bias=None if b is None else up(b, dev), **kw)
        torch.cuda.synchronize()
        check(x, b, k, got, kw)
        gw = np.random.default_rng(1).standard_normal((T, k)).astype(np.float32)
        grad = rt.select_backward(xd, got[0], up(gw, dev), **kw)
        torch.cuda.synchronize()
        assert grad.dtype == dtype
        check_grad(x, got[0].cpu().numpy(), gw, grad, kw, dtype)


@pytest.mark.parametrize("kind", ["normal", "few", "equal", "masked", "near", "wide"])
@pytest.mark.parametrize("T", [3, 1040])
@pytest.mark.parametrize("E,groups,kept,top,k", [(256, 8, 4, 2, 8), (256, 8, 4, 1, 8), (60, 6, 3, 2, 6), (64, 64, 9, 2, 7),
                                                 (96, 2, 1, 1, 5), (24, 12, 5, 2, 10), (340, 5, 2, 2, 16)])
def test_groups(dev, T, E, groups, kept, top, k, kind):
    for rule, bias in ((0, True), (1, False), (0, False), (3, True)):
        kw = dict(RULES[rule], groups=groups, topk_groups=kept, group_top=top)
        x, b = make(T, E, torch.float32, E + rule, kind, bias)
        log(f"groups T={T} E={E} {kind} {kw} bias={bias}")
        got = rt.select(up(x, dev), k, bias=None if b is None else up(b, dev), **kw)
        torch.cuda.synchronize()
        check(x, b, k, got, kw)


@pytest.mark.parametrize("kind", ["few", "equal", "masked", "near", "wide"])
@pytest.mark.parametrize("T,E,k", [(2, 40, 8), (3, 256, 8), (1025, 40, 12), (1025, 256, 8), (1024, 512, 16)])
def test_hard_rows(dev, T, E, k, kind):
    """Ties, masks that leave nothing, the type's lowest value, saturated scores, keys that 32 bits cannot order."""
    for rule, kw in enumerate(RULES):
        for bias in (True, False):
            x, b = make(T, E, torch.float32, 7 * E + rule, kind, bias)
            log(f"hard rows T={T} E={E} {kind} {kw} bias={bias}")
            xd = up(x, dev)
            got = rt.select(xd, k, bias=None if b is None else up(b, dev), **kw)
            torch.cuda.synchronize()
            check(x, b, k, got, kw)
            gw = np.random.default_rng(2).standard_normal((T, k)).astype(np.float32)
            gw[got[0].cpu().numpy() < 0] = np.nan  # places of no expert: never read into a result
            grad = rt.select_backward(xd, got[0], up(gw, dev), **kw)
            torch.cuda.synchronize()
            check_grad(x, got[0].cpu().numpy(), gw, grad, kw, torch.float32)


@pytest.mark.parametrize("T,E,k", [(2048, 61, 13), (6150, 256, 8), (6147, 384, 8), (6200, 510, 16), (8193, 96, 6),
                                   (8200, 130, 12), (8192, 256, 17)])
def test_many_rows(dev, T, E, k):
    """Row counts where four rows share a wavefront."""
    for rule, kw in enumerate(RULES):
        for bias in (True, False):
            x, b = make(T, E, torch.float32, T + E + rule, "few" if rule == 2 else "normal", bias)
            x[5::97] = make(1, E, torch.float32, 3, "masked")[0]
            log(f"many rows T={T} E={E} k={k} {kw} bias={bias}")
            xd = up(x, dev)
            got = rt.select(xd, k, bias=None if b is None else up(b, dev), **kw)
            torch.cuda.synchronize()
            check(x, b, k, got, kw)
            gw = np.random.default_rng(4).standard_normal((T, k)).astype(np.float32)
            grad = rt.select_backward(xd, got[0], up(gw, dev), **kw)
            torch.cuda.synchronize()
            check_grad(x, got[0].cpu().numpy(), gw, grad, kw, torch.float32)


@pytest.mark.parametrize("kind", ["normal", "few", "masked", "near"])
@pytest.mark.parametrize("E,groups,kept,top,k", [(256, 8, 4, 2, 8), (60, 6, 3, 1, 6), (96, 16, 9, 2, 7), (340, 5, 2, 2, 16)])
def test_groups_many_rows(dev, E, groups, kept, top, k, kind):
    T = 6150
    for rule, bias in ((0, True), (3, False)):
        kw = dict(RULES[rule], groups=groups, topk_groups=kept, group_top=top)
        x, b = make(T, E, torch.float32, E + rule, kind, bias)
        log(f"groups T={T} E={E} {kind} {kw} bias={bias}")
        got = rt.select(up(x, dev), k, bias=None if b is None else up(b, dev), **kw)
        torch.cuda.synchronize()
        check(x, b, k, got, kw)


def test_bias_special_values(dev):
    x, b = make(4, 64, torch.float32, 3)
    b[5], b[6], b[7] = -np.inf, np.nan, 50.0
    got = rt.select(up(x, dev), 8, bias=up(b, dev))
    torch.cuda.synchronize()
    assert (got[0][:, 0] == 7).all() and not ((got[0] == 5) | (got[0] == 6)).any()
    check(x, b, 8, got, {})


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [5, 1030])
def test_row_strides(dev, dtype, T):
    """Logits and gradients as columns of wider matrices, odd strides and starts among them; what lies between is kept."""
    for E, ld, first in ((96, 100, 2), (96, 128, 32), (130, 131, 1), (256, 264, 8), (256, 260, 4)):
        x, b = make(T, E, dtype, ld)
        log(f"strides T={T} E={E} ld={ld} first={first} {dtype}")
        wide = torch.full((T, ld), float("nan"), dtype=dtype, device=dev)
        wide[:, first:first + E] = up(x, dev, dtype)
        xd = wide[:, first:first + E]
        got = rt.select(xd, 6, bias=up(b, dev))
        gw = np.random.default_rng(3).standard_normal((T, 6)).astype(np.float32)
        out = torch.full((T, ld), 7.0, dtype=dtype, device=dev)
        rt.select_backward(xd, got[0], up(gw, dev), out=out[:, first:first + E])
        torch.cuda.synchronize()
        check(x, b, 6, got, {})
        check_grad(x, got[0].cpu().numpy(), gw, out[:, first:first + E], {}, dtype)
        assert (out[:, :first] == 7).all() and (out[:, first + E:] == 7).all()


@pytest.mark.parametrize("rule", range(4))
@pytest.mark.parametrize("T", [3, 1030])
def test_backward_of_any_indices(dev, T, rule):
    """Places outside [0, E), the same expert twice, rows without any."""
    E, k = 40, 7
    x, _ = make(T, E, torch.float32, 11)
    r = np.random.default_rng(12)
    idx = r.integers(-2, E + 2, (T, k)).astype(np.int32)
    idx[:, 3] = idx[:, 1]
    idx[0] = -1
    idx[1] = 5
    idx[2, :] = np.iinfo(np.int32).max
    gw = r.standard_normal((T, k)).astype(np.float32)
    log(f"any indices T={T} {RULES[rule]}")
    grad = rt.select_backward(up(x, dev), up(idx, dev), up(gw, dev), **RULES[rule])
    torch.cuda.synchronize()
    check_grad(x, idx, gw, grad, RULES[rule], torch.float32)


def test_gradient_against_differences(dev):
    """Central differences of the device's own weights: the choice must not change, and fp32 weights near 1 differ by
    2^-24 steps, so a difference over 2 h = 2^-5 is good to 2^-18 of the weights' scale and h^2 of the third slope."""
    T, E, k, h = 1, 24, 4, 2.0 ** -6
    for kw in RULES:
        x, _ = make(T, E, torch.float32, 21)
        gw = np.random.default_rng(4).standard_normal((T, k)).astype(np.float32)
        idx, _ = rt.select(up(x, dev), k, **kw)
        grad = rt.select_backward(up(x, dev), idx, up(gw, dev), **kw).cpu().numpy()
        steps = np.concatenate([x + h * np.eye(E, dtype=np.float32), x - h * np.eye(E, dtype=np.float32)])
        i2, w2 = rt.select(up(steps, dev), k, **kw)
        i2, w2 = i2.cpu().numpy(), w2.cpu().numpy().astype(np.float64)
        order = np.argsort(idx.cpu().numpy()[0])
        assert all(np.array_equal(np.sort(i), np.sort(i2[0])) for i in i2)  # the same experts, in whatever order
        by = np.take_along_axis(w2, np.argsort(i2, axis=1), 1)
        slope = ((by[:E] - by[E:]) * gw[0][order]).sum(axis=1) / (2 * h)
        scale = kw.get("routed_scale", 1.0) * np.abs(gw).sum()
        assert np.abs(slope - grad[0]).max() <= scale * (2.0 ** -18 * 2 + h * h)


def test_no_rows(dev):
    x = torch.empty((0, 64), device=dev)
    idx, w = rt.select(x, 4)
    assert idx.shape == w.shape == (0, 4)
    assert rt.select_backward(x, idx, w).shape == (0, 64)


def test_far_rows(dev):
    """Logits beyond 2^31 bytes and 2^31 elements from the start."""
    T, E, ld = 1100, 64, 2 * 10 ** 6
    x, b = make(T, E, torch.bfloat16, 5)
    wide = torch.empty((T, ld), dtype=torch.bfloat16, device=dev)
    wide[:, 4:4 + E] = up(x, dev, torch.bfloat16)
    got = rt.select(wide[:, 4:4 + E], 6, bias=up(b, dev))
    torch.cuda.synchronize()
    check(x, b, 6, got, {})


def test_agrees_with_the_fused_router(dev):
    """On router_gate_topk's own logits, its rule."""
    T, D, E, k = 70, 512, 64, 6
    ws = rt.Workspace(rt.workspace_bytes(T, D, E, k), dev)
    r = np.random.default_rng(8)
    bits = lambda s: up(wl.bf16_bits(r.standard_normal(s).astype(np.float32)).view(np.int16), dev)
    xq, wq = rt.quantize(bits((T, D)), ws), rt.quantize(bits((E, D)), ws)
    bias = up(r.uniform(-0.1, 0.1, E).astype(np.float32), dev)
    idx, w, logits = rt.gate_topk(xq, wq, bias, k, 2.5, ws, want_logits=True)
    i2, w2 = rt.select(logits, k, bias=bias, routed_scale=2.5)
    torch.cuda.synchronize()
    assert torch.equal(idx, i2)
    assert (w - w2).abs().max() <= 2.5e-5


@pytest.mark.parametrize("T", [4, 1030])
def test_graph_streams_and_repeatability(dev, T):
    E, k = 256, 8
    x, b = make(T, E, torch.float32, 31)
    xd, bd = up(x, dev), up(b, dev)
    gw = torch.randn((T, k), device=dev)
    kw = dict(bias=bd, groups=8, topk_groups=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = rt.select(xd, k, **kw)
        ga = rt.select_backward(xd, a[0], gw)
    torch.cuda.synchronize()
    check(x, b, k, a, dict(groups=8, topk_groups=4))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = rt.select(xd, k, **kw)
        gc = rt.select_backward(xd, c[0], gw)
    for i in range(3):
        xd.copy_(up(make(T, E, torch.float32, 40 + i)[0], dev))
        graph.replay()
        torch.cuda.synchronize()
        e = rt.select(xd, k, **kw)
        ge = rt.select_backward(xd, e[0], gw)
        torch.cuda.synchronize()
        assert torch.equal(c[0], e[0]) and torch.equal(c[1], e[1]) and torch.equal(gc, ge), i


@pytest.mark.parametrize("E,k", [(4, 2), (20, 17)])
def test_most_rows(dev, E, k):
    """The most rows of a call: its first and last rows are those of calls of their own."""
    T = 1 << 25
    g = torch.Generator(device=dev).manual_seed(E)
    x = torch.randn((T, E), generator=g, device=dev)
    gw = torch.randn((T, k), generator=g, device=dev)
    log(f"most rows E={E} k={k}")
    idx, w = rt.select(x, k)
    grad = rt.select_backward(x, idx, gw)
    torch.cuda.synchronize()
    # Sums of k terms in two orders, up to 6 steps each, and a quotient: weights 2 (6 + 2) 2^-24 apart; a gradient's
    # products with grad_w, whose sum it leaves out, 2 (8 + 7 + 2) 2^-24 max|grad_w|.
    atol = 40 * 2.0 ** -24 * float(gw.abs().max())
    for rows in (slice(0, 3000), slice(T - 3001, T)):
        i, v = rt.select(x[rows], k)
        assert torch.equal(i, idx[rows]) and torch.allclose(v, w[rows], rtol=2.0 ** -20, atol=0.0)
        assert torch.allclose(rt.select_backward(x[rows], i, gw[rows]), grad[rows], rtol=0.0, atol=atol)
    with pytest.raises(rt.RouterError):
        rt.select(torch.empty((T + 1, 1), device=dev), 1)


def test_binding_refusals(dev):
    x = torch.zeros((4, 64), device=dev)
    idx, w = rt.select(x, 4)
    bad = [
        lambda: rt.select(x.double(), 4),
        lambda: rt.select(x[0], 4),
        lambda: rt.select(x.t(), 4),
        lambda: rt.select(x, 0),
        lambda: rt.select(x, 65),
        lambda: rt.select(x, 4, scoring="tanh"),
        lambda: rt.select(x, 4, groups=7),
        lambda: rt.select(x, 4, groups=8, topk_groups=9),
        lambda: rt.select(x, 9, groups=8, topk_groups=1),
        lambda: rt.select(x, 4, group_top=3),
        lambda: rt.select(x, 4, bias=torch.zeros(63, device=dev)),
        lambda: rt.select(x, 4, bias=torch.zeros(64)),
        lambda: rt.select(x, 4, bias=torch.zeros(64, device=dev, dtype=torch.bfloat16)),
        lambda: rt.select(x, 4, out=(idx[:3], w)),
        lambda: rt.select(x, 4, out=(idx, w.half())),
        lambda: rt.select(torch.zeros((2, 600), device=dev), 4),
        lambda: rt.select_backward(x, idx.long(), w),
        lambda: rt.select_backward(x, idx, w[:, :3]),
        lambda: rt.select_backward(x, idx[:3], w),
        lambda: rt.select_backward(x, idx, w, out=torch.empty((4, 64), device=dev, dtype=torch.bfloat16)),
        lambda: rt.select_backward(x, idx, w, out=torch.empty((4, 65), device=dev)),
        lambda: rt.select_backward(x, idx, w, scoring=None),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(rt.RouterError):
            f()
            pytest.fail(f"call {i} was not refused")
