"""GPU parity of the lm_head's losses and their gradient against the CPU oracle, through the C ABI."""

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_06_amd import router as rt
from nvfp4_block_scaled_06_amd import workloads as wl
from oracle import loss_ref as lr

pytestmark = pytest.mark.gpu


def log(msg):
    print(f"[gpu-loss] {msg}", flush=True)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    rt.load_library()
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def up(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def quantized(a, dev):
    """fp32 rows as NVFP4 tensors by the library's own quantizer (bit-exact by its own tests)."""
    ws = rt.Workspace(rt.workspace_bytes(a.shape[0], a.shape[1], 1, 1), dev)
    return rt.quantize(up(wl.bf16_bits(a.astype(np.float32)).view(np.int16), dev), ws)


def host(q, rows=slice(None)):
    return q.codes[rows].cpu().numpy(), q.scales[rows].cpu().numpy(), q.gscale.cpu().numpy()[0]


def operands(T, D, N, seed, dev, x_scale=1.0, ramp=None):
    """x and the lm_head; ramp: a factor of each weight row."""
    r = np.random.default_rng(seed)
    w = r.standard_normal((N, D)) * 1.5 * D ** -0.5
    if ramp is not None:
        w *= ramp[:, None]
    return quantized(x_scale * r.standard_normal((T, D)), dev), quantized(w, dev)


def workspace(T, D, N, grad, dev):
    return rt.Workspace(rt.lmhead_loss_workspace_bytes(T, D, N, grad), dev)


def compare(got, ref, rows=slice(None)):
    fails = []
    for k, g in got.items():
        if g is not None:
            fails += lr.check_outputs(k, g[rows].double().cpu().numpy(), *ref[k])
    assert not fails, "\n".join(fails)


def make_targets(T, N, seed):
    r = np.random.default_rng(seed)
    y = r.integers(0, N, T).astype(np.int32)
    y[r.random(T) < 0.2] = -100
    if T > 3:
        y[0], y[1], y[2], y[3] = 0, N - 1, N, np.iinfo(np.int32).min
    else:
        y[0] = N - 1
    return y


# Few rows: 16- and 32-row streams (D a multiple of 256, of 64, of 32); many: wide tiles of 1 to 4 row tiles; odd and
# tiny vocabularies; blocks, tiles and steps that end inside.
SIZES = [(1, 32, 1), (1, 32, 2), (2, 64, 33), (3, 96, 127), (1, 256, 1000), (16, 256, 513), (16, 992, 400), (17, 512, 700),
         (32, 320, 1001), (31, 1056, 300), (33, 256, 600), (40, 96, 5000), (63, 64, 30000), (65, 512, 13000),
         (96, 160, 13001), (97, 544, 12500), (130, 288, 9000), (200, 256, 6500), (257, 96, 5121), (129, 1312, 9001)]


@pytest.mark.parametrize("T,D,N", SIZES)
def test_cross_entropy(dev, T, D, N):
    log(f"cross entropy T={T} D={D} N={N}")
    xq, wq = operands(T, D, N, T + D + N, dev)
    y = make_targets(T, N, T)
    weight = np.random.default_rng(T).standard_normal(T).astype(np.float32)
    ref = lr.loss_ref(host(xq), host(wq), y[:, None], weight=weight)
    loss, lse, dx = rt.lmhead_loss(xq, wq, up(y, dev), workspace(T, D, N, True, dev), weight=up(weight, dev), want_grad=True)
    torch.cuda.synchronize()
    compare(dict(loss=loss, lse=lse, dx=dx), ref)
    loss, lse, none = rt.lmhead_loss(xq, wq, up(y, dev), workspace(T, D, N, False, dev))
    torch.cuda.synchronize()
    assert none is None
    compare(dict(loss=loss, lse=lse), ref)


# Each tile of the logits with each way of its scales (D a multiple of 256, of 64, of 32): streams of 16 rows with two K
# groups, of 32 rows, alone on their weights and not; 64-row wide tiles, one round of 128-row ones, several rounds.
TILES = [(5, 1280, 700), (16, 1088, 900), (3, 1056, 500), (40, 1280, 1100), (33, 1088, 900), (20, 96, 900), (40, 1536, 13000),
         (64, 1600, 8300), (36, 1120, 11897),
         (200, 256, 32003), (250, 64, 32500), (195, 96, 32003),
         (96, 256, 100000), (128, 256, 99999), (200, 64, 65000), (180, 96, 65000), (260, 320, 40000), (270, 512, 40001),
         (400, 256, 50000), (500, 64, 40003), (420, 160, 45007)]


@pytest.mark.parametrize("T,D,N", TILES)
def test_every_tile(dev, T, D, N):
    log(f"every tile T={T} D={D} N={N}")
    xq, wq = operands(T, D, N, T + D + N, dev)
    y = make_targets(T, N, T)
    ref = lr.loss_ref(host(xq), host(wq), y[:, None])
    loss, lse, dx = rt.lmhead_loss(xq, wq, up(y, dev), workspace(T, D, N, True, dev), want_grad=True)
    alone = rt.lmhead_loss(xq, wq, up(y, dev), workspace(T, D, N, False, dev))
    torch.cuda.synchronize()
    compare(dict(loss=loss, lse=lse, dx=dx), ref)
    compare(dict(loss=alone[0], lse=alone[1]), ref)


def make_teacher(T, K, N, dtype, seed):
    r = np.random.default_rng(seed)
    tok = r.integers(0, N, (T, K)).astype(np.int32)
    te = (4.0 * r.standard_normal((T, K))).astype(np.float32)
    te[r.random((T, K)) < 0.05] = -np.inf
    te[r.random((T, K)) < 0.02] = np.finfo(np.float32).min / 4
    out = r.random((T, K)) < 0.2
    tok[out] = r.choice([-1, N, np.iinfo(np.int32).min, np.iinfo(np.int32).max], out.sum())
    te[out] = r.choice([np.nan, np.inf, 1e30, 0.0], out.sum())
    if K > 1:
        tok[:, K // 2] = tok[:, 0]  # named twice
    if T > 3:
        tok[1] = -1               # no entry
        te[2] = -np.inf           # nothing but masked ones
        tok[3] = tok[3, 0]        # one token alone
    if dtype == torch.bfloat16:
        te = torch.from_numpy(te).to(dtype).float().numpy()
    return tok, te


@pytest.mark.parametrize("T,D,N,K,tau", [(1, 32, 5, 1, 1.0), (2, 96, 50, 3, 0.5), (5, 256, 900, 4, 2.0),
                                         (16, 320, 700, 5, 1.0), (20, 288, 800, 65, 1.5), (32, 256, 600, 256, 4.0),
                                         (4, 64, 2000, 1024, 1.0), (40, 512, 700, 17, 0.25), (70, 160, 13003, 64, 1.0),
                                         (150, 256, 9000, 100, 3.0), (260, 96, 5500, 4, 1.0), (33, 64, 30000, 33, 2.0)])
def test_distillation(dev, T, D, N, K, tau):
    for dtype in (torch.float32, torch.bfloat16):
        log(f"distillation T={T} D={D} N={N} K={K} tau={tau} {dtype}")
        xq, wq = operands(T, D, N, T + K, dev)
        tok, te = make_teacher(T, K, N, dtype, K)
        weight = np.random.default_rng(T).standard_normal(T).astype(np.float32)
        ref = lr.loss_ref(host(xq), host(wq), tok, teacher=te, tau=tau, weight=weight)
        args = (xq, wq, up(tok, dev), up(te, dev).to(dtype))
        loss, lse, logq, dx = rt.lmhead_distill(*args, workspace(T, D, N, True, dev), temperature=tau,
                                                weight=up(weight, dev), want_grad=True)
        torch.cuda.synchronize()
        compare(dict(loss=loss, lse=lse, logq=logq, dx=dx), ref)
        loss, lse, logq, none = rt.lmhead_distill(*args, workspace(T, D, N, False, dev), temperature=tau)
        torch.cuda.synchronize()
        assert none is None
        compare(dict(loss=loss, lse=lse, logq=logq), ref)


@pytest.mark.parametrize("T,D,N", [(3, 256, 700), (20, 96, 5000), (70, 128, 13000)])
@pytest.mark.parametrize("kind", ["peaked", "rising", "falling", "zero"])
def test_hard_distributions(dev, T, D, N, kind):
    """One token with nearly all of the probability, maxima that rise or fall along the vocabulary, x of zeros."""
    ramp = {"rising": np.linspace(0.1, 3.0, N), "falling": np.linspace(3.0, 0.1, N)}.get(kind)
    scale = {"peaked": 60.0, "zero": 0.0}.get(kind, 6.0)
    log(f"{kind} T={T} D={D} N={N}")
    xq, wq = operands(T, D, N, 3, dev, scale, ramp)
    z = lr.dequant_ref(*host(xq)) @ lr.dequant_ref(*host(wq)).T
    y = np.where(np.arange(T) % 2, z.argmax(axis=1), make_targets(T, N, 1)).astype(np.int32)
    ref = lr.loss_ref(host(xq), host(wq), y[:, None])
    got = rt.lmhead_loss(xq, wq, up(y, dev), workspace(T, D, N, True, dev), want_grad=True)
    torch.cuda.synchronize()
    compare(dict(zip(("loss", "lse", "dx"), got)), ref)


@pytest.mark.parametrize("D", [32, 96, 128])
@pytest.mark.parametrize("kind", ["even", "rising"])
def test_pieces_of_the_vocabulary(dev, D, kind):
    """More rows than one piece's softmax weights have room for: three pieces, with maxima that rise from one to the
    next. Sampled rows against the oracle, the tile borders among them."""
    T, N = 66000, 10007
    log(f"pieces T={T} D={D} N={N} {kind}")
    xq, wq = operands(T, D, N, D, dev, 3.0, np.linspace(0.2, 2.5, N) if kind == "rising" else None)
    y = make_targets(T, N, 5)
    ws = workspace(T, D, N, True, dev)
    loss, lse, dx = rt.lmhead_loss(xq, wq, up(y, dev), ws, want_grad=True)
    torch.cuda.synchronize()
    rows = np.unique(np.concatenate([[0, 1, 2, 3, 127, 128, 32767, 32768, T - 81, T - 80, T - 1],
                                     np.random.default_rng(0).integers(0, T, 30)]))
    ref = lr.loss_ref(host(xq, rows), host(wq), y[rows][:, None])
    compare(dict(loss=loss, lse=lse, dx=dx), ref, up(rows, dev))


@pytest.mark.parametrize("T", [1, 4, 64, 300])
def test_full_vocabulary_sampled(dev, T):
    """The full 129280 x 7168 lm_head: every row's logsumexp and loss against the same sums in float64 on the GPU, and
    sampled columns of the gradient."""
    D, N = 7168, 129280
    g = torch.Generator(device=dev).manual_seed(T)
    ws = rt.Workspace(max(rt.workspace_bytes(N, D, 1, 1), rt.lmhead_loss_workspace_bytes(T, D, N, True)), dev)
    wq = rt.quantize((0.02 * torch.randn((N, D), generator=g, device=dev)).to(torch.bfloat16), ws)
    xq = rt.quantize(torch.randn((T, D), generator=g, device=dev).to(torch.bfloat16), ws)
    y = torch.randint(0, N, (T,), generator=g, device=dev, dtype=torch.int32)
    log(f"full vocabulary T={T}")
    loss, lse, dx = rt.lmhead_loss(xq, wq, y, ws, want_grad=True)
    torch.cuda.synchronize()
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=dev)

    def wide(q, rows, cols=slice(None)):
        v = torch.stack((lut[(q.codes[rows] & 15).long()], lut[(q.codes[rows] >> 4).long()]), -1).flatten(1)
        return (v * q.scales[rows].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1))[:, cols] * q.gscale.double()

    x = wide(xq, slice(None))
    z = torch.cat([torch.mm(x, wide(wq, slice(a, a + 8192)).t().contiguous()) for a in range(0, N, 8192)], 1)
    A = 40.0 * x.norm(dim=1).max() * 0.02  # well above sum |x w| / sqrt(D)
    tol = float(D * 2.0 ** -24 * A) + 1e-5
    ref = torch.logsumexp(z, 1)
    assert (lse.double() - ref).abs().max() <= tol
    assert (loss.double() - (ref - z.gather(1, y.long()[:, None])[:, 0])).abs().max() <= 2 * tol
    p = (z - ref[:, None]).exp()
    p[torch.arange(T, device=dev), y.long()] -= 1.0
    cols = torch.tensor([0, 1, 15, 16, 1023, 1024, 3583, 5000, 7167], device=dev)
    want = torch.zeros((T, len(cols)), dtype=torch.float64, device=dev)
    mag = torch.zeros_like(want)
    for a in range(0, N, 8192):
        w = wide(wq, slice(a, a + 8192), cols)
        want += torch.mm(p[:, a:a + 8192].contiguous(), w)
        mag += torch.mm(p[:, a:a + 8192].abs().contiguous(), w.abs())
    # bf16's half step, and the fp16 weights' three roundings against the sum of magnitudes
    assert ((dx[:, cols].double() - want).abs() <= 2.0 ** -8 * want.abs() + (3 * 2.0 ** -11 + 2 * tol + 1e-4) * mag).all()


def test_agrees_with_the_greedy_head(dev):
    """On lmhead_argmax's own logits."""
    T, D, N = 4, 1024, 5003
    xq, wq = operands(T, D, N, 1, dev)
    ws = rt.Workspace(max(rt.lmhead_workspace_bytes(T, D, N), rt.lmhead_loss_workspace_bytes(T, D, N)), dev)
    idx, top, logits = rt.lmhead_argmax(xq, wq, ws, want_logits=True)
    loss, lse, _ = rt.lmhead_loss(xq, wq, idx, ws)
    loss1, lse1, logq, _ = rt.lmhead_distill(xq, wq, idx[:, None].contiguous(), torch.zeros((T, 1), device=dev), ws)
    torch.cuda.synchronize()
    z = logits.double()
    assert (lse.double() - torch.logsumexp(z, 1)).abs().max() <= 1e-5
    assert (loss.double() - (torch.logsumexp(z, 1) - top.double())).abs().max() <= 1e-5
    assert torch.equal(lse, lse1) and torch.allclose(loss, -logq[:, 0], atol=1e-6) and torch.allclose(loss1, loss, atol=1e-6)


@pytest.mark.parametrize("T,D,N", [(4, 256, 900), (70, 128, 13000)])
def test_gradient_against_differences(dev, T, D, N):
    """Differences of the device's loss for x moved by whole code steps along one element."""
    xq, wq = operands(T, D, N, 9, dev, 2.0)
    y = make_targets(T, N, 9)
    ws = workspace(T, D, N, True, dev)
    _, _, dx = rt.lmhead_loss(xq, wq, up(y, dev), ws, want_grad=True)
    dx = dx.float().cpu().numpy()
    codes, scales, gsa = host(xq)
    for d in (0, 17, D - 1):
        moved = []
        for code in (2, 3):  # 1.0 and 1.5 of the block's scale
            c = codes.copy()
            c[:, d // 2] = (c[:, d // 2] & 0xF0) | code if d % 2 == 0 else (c[:, d // 2] & 0x0F) | (code << 4)
            q = rt.NVFP4Tensor(up(c, dev), xq.scales, xq.gscale)
            loss, _, g = rt.lmhead_loss(q, wq, up(y, dev), ws, want_grad=True)
            moved.append((loss.double().cpu().numpy(), g[:, d].double().cpu().numpy()))
        h = 0.5 * lr.dequant_ref(np.full((T, D // 2), 0x22, np.uint8), scales, gsa)[:, d]
        # The mean of the ends' slopes, off by h^2 / 12 of the third derivative: at most 6 max|w|^3.
        wmax = np.abs(lr.dequant_ref(*host(wq))[:, d]).max()
        slope = (moved[0][1] + moved[1][1]) / 2
        bound = 2 ** -8 * np.abs(slope) + h ** 2 / 12 * 6 * wmax ** 3 + 4e-6 * 12 / np.maximum(h, 1e-9) + 1e-3 * wmax
        ok = h > 0
        assert (np.abs((moved[1][0] - moved[0][0]) / np.maximum(h, 1e-9) - slope) <= bound)[ok].all()
    assert np.isfinite(dx).all()


@pytest.mark.parametrize("T", [1, 20, 80])
def test_graph_streams_and_repeatability(dev, T):
    """Captured and replayed with eager calls on the same workspace in between; another stream; no atomics in floats, so
    every run gives the same bits."""
    D, N, K = 256, 13000, 9
    xq, wq = operands(T, D, N, T, dev)
    tok, te = make_teacher(T, K, N, torch.float32, T)
    tok, te = up(tok, dev), up(te, dev)
    y = up(make_targets(T, N, T), dev)
    wsg, wse = workspace(T, D, N, True, dev), workspace(T, D, N, True, dev)

    def both(ws):
        return rt.lmhead_loss(xq, wq, y, ws, want_grad=True) + rt.lmhead_distill(xq, wq, tok, te, ws, temperature=2.0,
                                                                                 want_grad=True)

    want = both(wse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = both(wsg)
    torch.cuda.synchronize()
    same = lambda a, b: all(torch.equal(torch.nan_to_num(u.float()), torch.nan_to_num(v.float())) for u, v in zip(a, b))
    assert same(want, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(wsg)
    for i in range(3):
        fresh = quantized(np.random.default_rng(50 + i).standard_normal((T, D)), dev)
        xq.codes.copy_(fresh.codes), xq.scales.copy_(fresh.scales), xq.gscale.copy_(fresh.gscale)
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, both(wse)), i
        assert same(out, both(wsg)), i  # eager on the graph's own workspace, in order


def test_two_calls_at_once(dev):
    """Two streams, a workspace each."""
    D, N = 256, 6000
    jobs = []
    for T, seed in ((50, 1), (24, 2)):
        xq, wq = operands(T, D, N, seed, dev)
        y = up(make_targets(T, N, seed), dev)
        jobs.append((xq, wq, y, workspace(T, D, N, True, dev), torch.cuda.Stream()))
    want = [rt.lmhead_loss(*j[:4], want_grad=True) for j in jobs]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for xq, wq, y, ws, stream in jobs:
            with torch.cuda.stream(stream):
                got.append(rt.lmhead_loss(xq, wq, y, ws, want_grad=True))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_state_prefix_and_outputs(dev):
    """The workspace's state prefix stays zero; `out` is written; other rows' workspace contents do not matter."""
    T, D, N = 40, 128, 13000
    xq, wq = operands(T, D, N, 4, dev)
    y = up(make_targets(T, N, 4), dev)
    ws = workspace(T, D, N, True, dev)
    a = rt.lmhead_loss(xq, wq, y, ws, want_grad=True)
    ws.buf[4096 + 131072:].fill_(0xFF)  # NaN everywhere
    out = torch.full((T, D), float("nan"), dtype=torch.bfloat16, device=dev)
    b = rt.lmhead_loss(xq, wq, y, ws, want_grad=True, out=out)
    torch.cuda.synchronize()
    assert b[2] is out and all(torch.equal(u, v) for u, v in zip(a, b))
    assert not ws.buf[:4096 + 131072].any()


@pytest.mark.parametrize("T,D,N", [(3, 96, 300), (20, 256, 900), (40, 512, 700), (80, 128, 13000)])
def test_workspace_contents_do_not_matter(dev, T, D, N):
    xq, wq = operands(T, D, N, 6, dev)
    tok, te = make_teacher(T, 7, N, torch.float32, 6)
    want = None
    for fill in (0x00, 0xFF, 0x7C):
        for grad in (False, True):
            ws = workspace(T, D, N, grad, dev)
            ws.buf[4096 + 131072:].fill_(fill)
            got = rt.lmhead_distill(xq, wq, up(tok, dev), up(te, dev), ws, want_grad=grad)
            torch.cuda.synchronize()
            if grad:
                want = want or got
                assert all(torch.equal(torch.nan_to_num(u), torch.nan_to_num(v)) for u, v in zip(got, want)), fill


def test_nan_teachers_stay_in_their_rows(dev):
    T, D, N, K = 6, 64, 200, 5
    xq, wq = operands(T, D, N, 8, dev)
    r = np.random.default_rng(8)
    tok, te = r.integers(0, N, (T, K)).astype(np.int32), r.standard_normal((T, K)).astype(np.float32)
    ws = workspace(T, D, N, True, dev)
    want = rt.lmhead_distill(xq, wq, up(tok, dev), up(te, dev), ws, want_grad=True)
    te[2, 1], te[4, 0] = np.nan, np.inf
    got = rt.lmhead_distill(xq, wq, up(tok, dev), up(te, dev), ws, want_grad=True)
    torch.cuda.synchronize()
    for t in range(T):
        for u, v in zip(got, want):
            if t in (2, 4) and u.dim() != 1:
                continue
            if t in (2, 4):
                continue
            assert torch.equal(u[t], v[t]), t
    assert torch.isnan(got[0][[2, 4]]).all() and torch.isnan(got[3][[2, 4]].float()).all()


def test_no_rows(dev):
    D, N = 64, 100
    _, wq = operands(1, D, N, 1, dev)
    xq = rt.empty_nvfp4(0, D, dev)
    ws = workspace(0, D, N, True, dev)
    loss, lse, dx = rt.lmhead_loss(xq, wq, torch.empty(0, dtype=torch.int32, device=dev), ws, want_grad=True)
    assert loss.shape == lse.shape == (0,) and dx.shape == (0, D)
    out = rt.lmhead_distill(xq, wq, torch.empty((0, 3), dtype=torch.int32, device=dev), torch.empty((0, 3), device=dev), ws)
    assert out[2].shape == (0, 3) and out[3] is None


def test_last_layer_together(dev):
    """A decoder's last layer as these calls make it: choice, plan, experts, quantizer, loss with its gradient, and the
    choice's own gradient; captured and replayed as well."""
    T, D, E, k, F, N = 70, 512, 32, 4, 256, 13000
    r = np.random.default_rng(17)
    x = up(wl.bf16_bits(r.standard_normal((T, D)).astype(np.float32)).view(np.int16), dev)
    ws = rt.Workspace(max(rt.workspace_bytes(T * k, D, E, k), rt.grouped_workspace_bytes(T, k, E, D, F),
                          rt.lmhead_loss_workspace_bytes(T, D, N, True)), dev)
    bits = lambda s, v: up(wl.bf16_bits((v * r.standard_normal(s)).astype(np.float32)).view(np.int16), dev)
    gate, head = rt.quantize(bits((E, D), 0.05), ws), rt.quantize(bits((N, D), 0.05), ws)
    w13 = rt.quantize_grouped_weights(bits((E, 2 * F, D), D ** -0.5), ws)
    w2 = rt.quantize_grouped_weights(bits((E, D, F), F ** -0.5), ws)
    bias = up(r.uniform(-0.01, 0.01, E).astype(np.float32), dev)
    y, gw = up(make_targets(T, N, 2), dev), up(r.standard_normal((T, k)).astype(np.float32), dev)

    def step():
        xq = rt.quantize(x, ws)
        _, _, logits = rt.gate_topk(xq, gate, bias, k, 1.0, ws, want_logits=True)
        idx, w = rt.select(logits, k, bias=bias, groups=4, topk_groups=2, routed_scale=2.5)
        plan = rt.grouped_plan(idx, E, ws)
        h = rt.grouped_swiglu(xq, w13, plan)
        out = rt.grouped_combine(rt.quantize(h, ws), w2, plan, w, ws, residual=x.view(torch.bfloat16))
        oq = rt.quantize(out, ws)
        return rt.lmhead_loss(oq, head, y, ws, want_grad=True) + (rt.select_backward(logits, idx, gw, routed_scale=2.5),
                                                                  idx, oq.codes, oq.scales, oq.gscale)

    first = step()
    torch.cuda.synchronize()
    loss, lse, dx, grad, idx, codes, scales, gs = first
    ref = lr.loss_ref((codes.cpu().numpy(), scales.cpu().numpy(), gs.cpu().numpy()[0]), host(head), y.cpu().numpy()[:, None])
    compare(dict(loss=loss, lse=lse, dx=dx), ref)
    assert (idx >= 0).all() and torch.isfinite(grad).all() and ((idx // 8).sort(1).values.diff(dim=1) > 0).sum(1).max() <= 1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        x.copy_(up(wl.bf16_bits(np.random.default_rng(i).standard_normal((T, D)).astype(np.float32)).view(np.int16), dev))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_binding_refusals(dev):
    T, D, N = 4, 64, 100
    xq, wq = operands(T, D, N, 1, dev)
    y = torch.zeros(T, dtype=torch.int32, device=dev)
    tok, te = torch.zeros((T, 3), dtype=torch.int32, device=dev), torch.zeros((T, 3), device=dev)
    ws, small = workspace(T, D, N, True, dev), workspace(T, D, N, False, dev)
    _, wide = operands(1, 2 * D, N, 1, dev)
    bad = [
        lambda: rt.lmhead_loss(xq, wide, y, ws),
        lambda: rt.lmhead_loss(xq, wq, y.long(), ws),
        lambda: rt.lmhead_loss(xq, wq, y[:3], ws),
        lambda: rt.lmhead_loss(xq, wq, y.cpu(), ws),
        lambda: rt.lmhead_loss(xq, wq, y, None),
        lambda: rt.lmhead_loss(xq, wq, y, small, want_grad=True),
        lambda: rt.lmhead_loss(xq, wq, y, ws, weight=torch.ones(T, device=dev, dtype=torch.bfloat16)),
        lambda: rt.lmhead_loss(xq, wq, y, ws, weight=torch.ones(T + 1, device=dev)),
        lambda: rt.lmhead_loss(xq, wq, y, ws, out=torch.empty((T, D), dtype=torch.bfloat16, device=dev)),
        lambda: rt.lmhead_loss(xq, wq, y, ws, want_grad=True, out=torch.empty((T, D), device=dev)),
        lambda: rt.lmhead_loss(xq, rt.NVFP4Tensor(wq.codes, wq.scales[:50], wq.gscale), y, ws),
        lambda: rt.lmhead_loss(rt.NVFP4Tensor(xq.codes.t(), xq.scales, xq.gscale), wq, y, ws),
        lambda: rt.lmhead_distill(xq, wq, tok, te[:, :2], ws),
        lambda: rt.lmhead_distill(xq, wq, tok.long(), te, ws),
        lambda: rt.lmhead_distill(xq, wq, tok, te.half(), ws),
        lambda: rt.lmhead_distill(xq, wq, tok, te, ws, temperature=0.0),
        lambda: rt.lmhead_distill(xq, wq, tok[0], te, ws),
        lambda: rt.lmhead_distill(xq, wq, torch.zeros((T, 1025), dtype=torch.int32, device=dev),
                                  torch.zeros((T, 1025), device=dev), ws),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(rt.RouterError):
            f()
            pytest.fail(f"call {i} was not refused")


@pytest.mark.parametrize("T", [3, 20])
def test_codes_beyond_32_bits(dev, T):
    """Weight codes of more than 2^31 bytes, taken in two pieces also where rows are few; against float64 on the GPU."""
    D, N = 1 << 20, 4500
    g = torch.Generator(device=dev).manual_seed(T)
    byte = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=dev, dtype=torch.uint8)
    wq = rt.NVFP4Tensor(byte(0, 256, N, D // 2), byte(0x18, 0x30, N, D // 16), torch.tensor([3e-4], device=dev))
    xq = rt.NVFP4Tensor(byte(0, 256, T, D // 2), byte(0x18, 0x30, T, D // 16), torch.tensor([0.04], device=dev))
    y = torch.randint(0, N, (T,), generator=g, device=dev, dtype=torch.int32)
    y[0] = N - 1
    log(f"codes beyond 32 bits T={T}")
    ws = workspace(T, D, N, True, dev)
    alone = rt.lmhead_loss(xq, wq, y, ws)
    loss, lse, dx = rt.lmhead_loss(xq, wq, y, ws, want_grad=True)
    torch.cuda.synchronize()
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=dev)

    def wide(q, rows, a, b):
        c = q.codes[rows, a // 2:b // 2]
        v = torch.stack((lut[(c & 15).long()], lut[(c >> 4).long()]), -1).flatten(1)
        return v * q.scales[rows, a // 16:b // 16].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1) * q.gscale.double()

    z = torch.zeros((T, N), dtype=torch.float64, device=dev)
    mag = torch.zeros((T, N), dtype=torch.float64, device=dev)
    step = 1 << 15
    for a in range(0, D, step):
        u, v = wide(xq, slice(None), a, a + step), wide(wq, slice(None), a, a + step)
        z += torch.mm(u, v.t().contiguous())
        mag += torch.mm(u.abs(), v.abs().t().contiguous())
    # Random signs: a sum of D products in fp32 is off by sqrt(D) half steps of its largest partial sum, not D; partial
    # sums stay below 6 sqrt(D) products' size.
    tol = float(6 * 2.0 ** -24 * mag.max()) + 1e-4
    ref = torch.logsumexp(z, 1)
    assert (lse.double() - ref).abs().max() <= tol and (alone[1].double() - ref).abs().max() <= tol
    want = ref - z.gather(1, y.long()[:, None])[:, 0]
    assert (loss.double() - want).abs().max() <= 2 * tol and (alone[0].double() - want).abs().max() <= 2 * tol
    p = (z - ref[:, None]).exp()
    p[torch.arange(T, device=dev), y.long()] -= 1.0
    for a in (0, 16384, D // 2 + 1024, D - 1024):
        w = wide(wq, slice(None), a, a + 1024)
        bound = 2.0 ** -8 * torch.mm(p, w).abs() + (3 * 2.0 ** -11 + 4 * tol) * torch.mm(p.abs(), w.abs())
        assert ((dx[:, a:a + 1024].double() - torch.mm(p, w)).abs() <= bound).all(), a


def test_most_rows(dev):
    """The most rows of a call, and a vocabulary that takes more than one launch with them; a few rows against float64."""
    T, D, N = 1 << 18, 32, (1 << 20) + 700
    g = torch.Generator(device=dev).manual_seed(2)
    byte = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=dev, dtype=torch.uint8)
    wq = rt.NVFP4Tensor(byte(0, 256, N, D // 2), byte(0x18, 0x30, N, D // 16), torch.tensor([0.5], device=dev))
    xq = rt.NVFP4Tensor(byte(0, 256, T, D // 2), byte(0x18, 0x30, T, D // 16), torch.tensor([0.5], device=dev))
    y = torch.randint(0, N, (T,), generator=g, device=dev, dtype=torch.int32)
    rows = torch.tensor([0, 1, 127, 131072, T - 129, T - 1], device=dev)
    y[-1] = N - 1
    log(f"most rows T={T} D={D} N={N}")
    loss, lse, _ = rt.lmhead_loss(xq, wq, y, workspace(T, D, N, False, dev))
    torch.cuda.synchronize()
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=dev)

    def wide(q, at):
        c = q.codes[at]
        v = torch.stack((lut[(c & 15).long()], lut[(c >> 4).long()]), -1).flatten(1)
        return v * q.scales[at].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1) * q.gscale.double()

    u, v = wide(xq, rows), wide(wq, slice(None))
    z = torch.mm(u, v.t().contiguous())
    # D products in fp32, and sums of exponentials in a tree of fp32 over N (a block's 64 in 6 steps, then 64 and more
    # blocks in a thread, each exponential off by a few steps): 2^-24 (D |x||w| + 128) bounds the logarithm.
    tol = 2.0 ** -24 * (D * float(torch.mm(u.abs(), v.abs().t().contiguous()).max()) + 128 + 8 * float(z.abs().max()))
    ref = torch.logsumexp(z, 1)
    assert (lse[rows].double() - ref).abs().max() <= tol
    want = ref - z.gather(1, y[rows].long()[:, None])[:, 0]
    assert (loss[rows].double() - want).abs().max() <= 2 * tol
