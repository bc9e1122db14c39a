"""GPU parity of the routed experts (grouped_plan, grouped_swiglu, grouped_combine) against the CPU oracle, through
the C ABI: every tile path, odd sizes, ragged and empty experts, slots of no expert, and a whole layer."""

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_06_amd import router as rt
from nvfp4_block_scaled_06_amd import workloads as wl
from oracle import experts_ref as er
from oracle import quant_ref, router_ref

pytestmark = pytest.mark.gpu

STATE = 4096 + 131072  # ROUTER_WORKSPACE_STATE_BYTES


def log(msg):
    print(f"[gpu-experts] {msg}", flush=True)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    rt.load_library()
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


@pytest.fixture(scope="module")
def ws(dev):
    return rt.Workspace(256 << 20, dev)


def bits(shape, seed, scale=1.0):
    return wl.bf16_bits((np.random.default_rng(seed).standard_normal(shape) * scale).astype(np.float32))


def to_dev(b, dev):
    return torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).to(dev)


def routing(T, k, E, seed, kind="skewed"):
    """[T, k] distinct experts of E, some more popular than others; or a special pattern."""
    r = np.random.default_rng(seed)
    if kind == "one":  # every slot to expert E - 1
        return np.full((T, k), E - 1, dtype=np.int32)
    if kind == "none":
        return np.full((T, k), -1, dtype=np.int32)
    if kind == "repeat":  # a token may name an expert several times
        return r.integers(0, max(E // 3, 1), (T, k)).astype(np.int32)
    score = r.standard_normal((T, E)) + r.standard_normal(E)
    idx = np.argsort(-score, axis=1)[:, :k].astype(np.int32)
    if kind == "holes":  # padded tokens, and stray values
        idx[r.random((T, k)) < 0.3] = -1
        idx[r.random((T, k)) < 0.1] = 2 ** 31 - 1
        idx[r.random((T, k)) < 0.1] = -2 ** 31
        idx[T // 2] = -1
    return idx


def make_plan(idx, G, first, ws, dev):
    p = rt.grouped_plan(torch.from_numpy(idx).to(dev), G, ws, first_expert=first)
    torch.cuda.synchronize()
    return p


@pytest.mark.parametrize("T,k,E,first,G,kind", [
    (1, 1, 1, 0, 1, "skewed"), (1, 8, 256, 0, 256, "skewed"), (3, 2, 5, 0, 5, "repeat"), (64, 8, 256, 0, 256, "skewed"),
    (512, 8, 64, 0, 64, "skewed"), (513, 8, 64, 0, 64, "skewed"), (1003, 6, 96, 17, 24, "skewed"),
    (5000, 8, 512, 0, 512, "skewed"), (700, 32, 300, 299, 1, "holes"), (900, 7, 31, 4, 20, "holes"),
    (2000, 4, 9, 0, 9, "one"), (300, 4, 9, 0, 9, "none"), (77, 5, 130, 100, 400, "skewed"), (2, 2, 8, 50, 8, "skewed"),
    (40001, 3, 384, 1, 383, "repeat"),
])
def test_plan(dev, ws, T, k, E, first, G, kind):
    log(f"plan T={T} k={k} E={E} first={first} G={G} {kind}")
    idx = routing(T, k, E, T + E, kind)
    p = make_plan(idx, G, first, ws, dev)
    off, rows, pos = er.plan_ref(idx, G, first)
    assert np.array_equal(p.offsets.cpu().numpy(), off)
    assert np.array_equal(p.rows.cpu().numpy(), rows)
    assert np.array_equal(p.pos.cpu().numpy(), pos)


def test_plan_of_many_slots(dev):
    """More slots than 256 chunks of 4096: the chunks grow."""
    T, k, E = 140000, 8, 300
    idx = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    wsl = rt.Workspace(rt.grouped_workspace_bytes(0, k, E, 32, 32) + (4 << 20), dev)
    log(f"plan T={T} k={k}")
    p = rt.grouped_plan(idx.to(dev), E, wsl)
    torch.cuda.synchronize()
    order = torch.argsort(idx.reshape(-1), stable=True)
    assert torch.equal(p.rows.cpu().long(), order)
    assert torch.equal(p.pos.cpu()[order], torch.arange(T * k, dtype=torch.int32))
    assert torch.equal(p.offsets.cpu().long(), torch.cat((torch.zeros(1, dtype=torch.long),
                                                          torch.bincount(idx.reshape(-1), minlength=E).cumsum(0))))


def test_plan_of_no_tokens(dev, ws):
    p = rt.grouped_plan(torch.empty((0, 8), dtype=torch.int32, device=dev), 16, ws)
    assert p.offsets.cpu().tolist() == 17 * [0]


def host(q):
    return q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.gscale.cpu().numpy()[0]


def host_groups(wg):
    c, s, g = wg.codes.cpu().numpy(), wg.scales.cpu().numpy(), wg.gscale.cpu().numpy()
    return [(c[i], s[i], g[i]) for i in range(len(g))]


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


# T, k, E, first, G, F, D, routing, bias: one line per path and edge.
SWIGLU = [
    # Up to 8 slots per expert: 16-row tiles.
    (1, 8, 64, 0, 64, 64, 1024, "skewed", False),
    (1, 2, 4, 0, 4, 16, 32, "repeat", True),          # the smallest sizes
    (2, 4, 32, 0, 32, 48, 2080, "skewed", True),      # D % 256 != 0
    (3, 8, 40, 0, 40, 80, 7168, "skewed", False),
    (2, 3, 16, 0, 16, 32, 16384, "skewed", True),
    (2, 8, 2, 0, 2, 64, 16416, "repeat", False),
    (33, 4, 64, 10, 40, 112, 512, "holes", True),     # some slots of no expert
    (4, 8, 256, 0, 256, 32, 256, "one", False),       # all rows in one of many experts
    (200, 8, 200, 0, 200, 144, 768, "one", True),     # 1600 rows of it, 100 tiles
    (9, 3, 512, 5, 500, 48, 288, "skewed", False),    # many experts
    (40, 8, 96, 0, 96, 288, 416, "skewed", True),     # more workgroups than compute units, D % 256 != 0
    (32, 2, 64, 60, 64, 160, 768, "none", False),     # no rows, few slots
    # Up to 16: 32-row tiles, and 16-row tiles for few work items.
    (64, 4, 16, 0, 16, 1040, 512, "skewed", True),
    (50, 4, 16, 0, 16, 1040, 448, "skewed", False),
    (80, 4, 16, 0, 16, 1056, 352, "skewed", True),
    (37, 3, 9, 2, 3, 640, 1600, "holes", True),
    (64, 4, 16, 0, 16, 144, 512, "skewed", True),
    (50, 4, 16, 0, 16, 64, 1056, "skewed", False),
    (16, 16, 16, 0, 16, 16, 32, "repeat", True),
    (300, 3, 32, 1, 30, 176, 992, "holes", True),
    # More: shared by size, all small here (too few rows to fill the GPU with 128-row tiles) ...
    (100, 4, 12, 2, 8, 80, 768, "holes", True),
    (200, 2, 8, 0, 8, 208, 2080, "skewed", False),
    (129, 1, 3, 0, 1, 128, 256, "one", False),        # an expert without rows
    (40, 8, 4, 0, 4, 32, 256, "none", True),          # no rows at all
    # ... (a rank's part: only the device knows that they are) ...
    (600, 8, 128, 10, 16, 640, 512, "skewed", False),
    # ... with 64-row tiles, one for each compute unit at most ...
    (300, 7, 40, 0, 40, 1024, 256, "skewed", True),
    (260, 8, 30, 2, 24, 1200, 352, "holes", False),
    # ... and with enough of those tiles and small experts beside them, scale rows 16-byte aligned and not, and so
    # many work items that the small experts' workgroups take several.
    (1400, 8, 40, 0, 40, 2080, 256, "skewed", False),
    (1300, 8, 44, 3, 38, 2144, 96, "holes", True),
    (1400, 8, 40, 0, 40, 704, 512, "skewed", True),
    (1300, 8, 44, 3, 38, 1408, 416, "holes", True),
]


@pytest.mark.parametrize("T,k,E,first,G,F,D,kind,with_bias", SWIGLU)
def test_swiglu(dev, ws, T, k, E, first, G, F, D, kind, with_bias):
    log(f"swiglu T={T} k={k} E={E} first={first} G={G} F={F} D={D} {kind} bias={with_bias}")
    idx = routing(T, k, E, T + F, kind)
    off, rows, _ = er.plan_ref(idx, G, first)
    plan = make_plan(idx, G, first, ws, dev)
    xq = rt.quantize(to_dev(bits((T, D), T, 2.0), dev), ws)
    wg = rt.quantize_grouped_weights(to_dev(bits((G, 2 * F, D), D, D ** -0.5), dev), ws)
    bias = np.random.default_rng(1).standard_normal((G, 2 * F)).astype(np.float32) if with_bias else None
    out = torch.full((T * k, F), float("nan"), dtype=torch.bfloat16, device=dev)
    rt.grouped_swiglu(xq, wg, plan, bias=None if bias is None else torch.from_numpy(bias).to(dev), out=out)
    torch.cuda.synchronize()
    ref, bound = er.swiglu_ref(host(xq), host_groups(wg), off, rows, k, bias)
    fails = er.check_close("h", f64(out), ref, bound)
    assert not fails, "\n".join(fails)
    assert torch.all(out[int(off[-1]):] == 0)  # rows of no expert


COMBINE = [(T, k, E, first, G, max(16, F), 32 * max(1, D // 64), kind, b, i % 2 == 0)
           for i, (T, k, E, first, G, F, D, kind, b) in enumerate(SWIGLU[:-4])]
COMBINE += [(300, 7, 40, 0, 40, 2048, 256, "skewed", True, True), (260, 8, 30, 2, 24, 2400, 352, "holes", False, False),
            (60, 8, 96, 0, 96, 288, 768, "skewed", True, True), (1400, 8, 40, 0, 40, 4160, 256, "skewed", False, True),
            (1300, 8, 44, 3, 38, 4288, 96, "holes", True, False), (1400, 8, 40, 0, 40, 1360, 512, "skewed", True, True),
            (1300, 8, 44, 3, 38, 2816, 352, "holes", True, False)]


@pytest.mark.parametrize("T,k,E,first,G,N,F,kind,with_bias,with_residual", COMBINE)
def test_combine(dev, ws, T, k, E, first, G, N, F, kind, with_bias, with_residual):
    log(f"combine T={T} k={k} E={E} first={first} G={G} N={N} F={F} {kind} bias={with_bias} res={with_residual}")
    r = np.random.default_rng(T + N)
    idx = routing(T, k, E, T + N, kind)
    off, _, pos = er.plan_ref(idx, G, first)
    plan = make_plan(idx, G, first, ws, dev)
    hq = rt.quantize(to_dev(bits((T * k, F), T, 0.5), dev), ws)
    wg = rt.quantize_grouped_weights(to_dev(bits((G, N, F), F, F ** -0.5), dev), ws)
    w = r.uniform(0.05, 0.6, (T, k)).astype(np.float32)
    w[pos.reshape(T, k) < 0] = np.nan  # weights of slots held elsewhere are not read
    bias = r.standard_normal((G, N)).astype(np.float32) if with_bias else None
    res = bits((T, N), 5) if with_residual else None
    out = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device=dev)
    rt.grouped_combine(hq, wg, plan, torch.from_numpy(w).to(dev), ws,
                       bias=None if bias is None else torch.from_numpy(bias).to(dev),
                       residual=None if res is None else to_dev(res, dev).view(torch.bfloat16), out=out)
    torch.cuda.synchronize()
    ref, bound = er.combine_ref(host(hq), host_groups(wg), off, pos, w, bias,
                                None if res is None else quant_ref.bf16_bits_to_f64(res))
    fails = er.check_close("out", f64(out), ref, bound)
    assert not fails, "\n".join(fails)


def layer_inputs(dev, ws, T, D, E, k, F, seed=0):
    x = to_dev(bits((T, D), seed), dev)
    gate = rt.quantize(to_dev(bits((E, D), seed + 1, 0.02), dev), ws)
    bias = torch.from_numpy(np.random.default_rng(seed).uniform(-0.01, 0.01, E).astype(np.float32)).to(dev)
    w13 = rt.quantize_grouped_weights(to_dev(bits((E, 2 * F, D), seed + 2, D ** -0.5), dev), ws)
    w2 = rt.quantize_grouped_weights(to_dev(bits((E, D, F), seed + 3, F ** -0.5), dev), ws)
    return x, gate, bias, w13, w2


def run_layer(x, gate, bias, w13, w2, k, ws, parts=None):
    """The whole expert layer, x as its residual; parts: (first, G) of an expert-parallel rank, no residual."""
    xq, (idx, w, _) = rt.forward(x, gate, bias, k, 2.5, ws)
    plan = rt.grouped_plan(idx, w13.G, ws, first_expert=parts[0] if parts else 0)
    h = rt.grouped_swiglu(xq, w13, plan)
    hq = rt.quantize(h, ws)
    out = rt.grouped_combine(hq, w2, plan, w, ws, residual=None if parts else x.view(torch.bfloat16))
    return xq, idx, w, plan, h, hq, out


@pytest.mark.parametrize("T", [1, 2, 7, 64, 300])
def test_layer(dev, ws, T):
    D, E, k, F = 1024, 32, 4, 256
    x, gate, bias, w13, w2 = layer_inputs(dev, ws, T, D, E, k, F, seed=T)
    log(f"layer T={T} D={D} E={E} k={k} F={F}")
    xq, idx, w, plan, h, hq, out = run_layer(x, gate, bias, w13, w2, k, ws)
    torch.cuda.synchronize()
    off, rows, pos = er.plan_ref(idx.cpu().numpy(), E)
    ref, bound = er.swiglu_ref(host(xq), host_groups(w13), off, rows, k)
    fails = er.check_close("h", f64(h), ref, bound)
    res = quant_ref.bf16_bits_to_f64(x.cpu().numpy().view(np.uint16))
    ref, bound = er.combine_ref(host(hq), host_groups(w2), off, pos, w.cpu().numpy(), residual=res)
    fails += er.check_close("out", f64(out), ref, bound)
    assert not fails, "\n".join(fails)


@pytest.mark.parametrize("T", [1, 64, 300])
def test_layer_replays_in_a_graph(dev, ws, T):
    """The whole layer captured once and replayed, with other eager calls on the same workspace in between; the
    residual is also written in place."""
    D, E, k, F = 512, 16, 4, 128
    x, gate, bias, w13, w2 = layer_inputs(dev, ws, T, D, E, k, F, seed=3)
    wsg = rt.Workspace(max(rt.workspace_bytes(T, D, E, k), rt.grouped_workspace_bytes(T, k, E, D, F)), dev)
    log(f"layer in a graph T={T}")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run_layer(x, gate, bias, w13, w2, k, wsg)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run_layer(x, gate, bias, w13, w2, k, wsg)[-1]
    for i in range(3):
        x.copy_(to_dev(bits((T, D), 100 + i), dev))
        graph.replay()
        torch.cuda.synchronize()
        want = run_layer(x, gate, bias, w13, w2, k, wsg)[-1]
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_residual_in_place(dev, ws):
    T, D, E, k, F = 20, 256, 8, 2, 64
    x, gate, bias, w13, w2 = layer_inputs(dev, ws, T, D, E, k, F)
    _, _, w, plan, _, hq, want = run_layer(x, gate, bias, w13, w2, k, ws)
    inout = x.view(torch.bfloat16).clone()
    rt.grouped_combine(hq, w2, plan, w, ws, residual=inout, out=inout)
    torch.cuda.synchronize()
    assert torch.equal(inout, want)


def test_ranks_add_up_to_the_layer(dev, ws):
    """Expert-parallel ranks of different sizes: their rows are the whole layer's, and their sums add up to it."""
    T, D, E, k, F = 150, 512, 24, 4, 128
    x, gate, bias, w13, w2 = layer_inputs(dev, ws, T, D, E, k, F, seed=9)
    _, idx, w, plan, h, hq, _ = run_layer(x, gate, bias, w13, w2, k, ws)
    whole = rt.grouped_combine(hq, w2, plan, w, ws).double()
    xq = rt.quantize(x, ws)
    total, step = torch.zeros((T, D), dtype=torch.float64, device=dev), er.U16 * whole.abs()
    for first, G in ((0, 5), (5, 1), (6, 18)):
        def part(q):
            return rt.GroupedWeights(q.codes[first:first + G], q.scales[first:first + G], q.gscale[first:first + G])

        p = rt.grouped_plan(idx, G, ws, first_expert=first)
        off, rows, _ = er.plan_ref(idx.cpu().numpy(), G, first)
        ref, bound = er.swiglu_ref(host(xq), host_groups(part(w13)), off, rows, k)
        fails = er.check_close("h", f64(rt.grouped_swiglu(xq, part(w13), p)), ref, bound)
        assert not fails, "\n".join(fails)
        # The whole layer's codes of these experts' rows, so that the outputs differ by fp32 sums and roundings only.
        n, s = int(off[-1]), int(plan.offsets[first])
        q = rt.NVFP4Tensor(torch.zeros_like(hq.codes), torch.zeros_like(hq.scales), hq.gscale)
        q.codes[:n], q.scales[:n] = hq.codes[s:s + n], hq.scales[s:s + n]
        o = rt.grouped_combine(q, part(w2), p, w, ws).double()
        total, step = total + o, step + er.U16 * o.abs()
    # Each rank's output is rounded to bf16 once and the whole one once. The fp32 sums' errors, F 2^-24 of the
    # products' magnitudes, stay below a hundredth of the largest output's rounding step.
    assert torch.all((total - whole).abs() <= step + 0.01 * er.U16 * whole.abs().amax())


def test_other_stream_and_repeatability(dev, ws):
    T, D, E, k, F = 90, 768, 12, 4, 160
    x, gate, bias, w13, w2 = layer_inputs(dev, ws, T, D, E, k, F, seed=4)
    want = run_layer(x, gate, bias, w13, w2, k, ws)[-1]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = run_layer(x, gate, bias, w13, w2, k, ws)[-1]
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def shifted(t, by):
    """The same values, `by` bytes past a 16-byte boundary."""
    buf = torch.empty(t.numel() + 16, dtype=torch.uint8, device=t.device)
    view = buf[by:by + t.numel()].view(t.shape)
    assert view.data_ptr() % 16 == by
    return view.copy_(t)


@pytest.mark.parametrize("T,k,E,F,D", [
    (2, 4, 16, 48, 64), (30, 4, 24, 96, 448), (50, 4, 16, 176, 256), (40, 4, 16, 144, 832), (1400, 8, 40, 704, 192),
    (1400, 8, 40, 704, 256), (1400, 8, 40, 704, 576), (1400, 8, 40, 704, 544), (20, 4, 16, 48, 352),
])
def test_scale_alignment(dev, ws, T, k, E, F, D):
    """D a multiple of 256, 64 or 32, the weights' scales at every alignment: the same bits each time, few rows and
    many; scales that no 4-byte load may touch are refused."""
    log(f"scale alignment T={T} k={k} E={E} F={F} D={D}")
    idx = routing(T, k, E, T + F, "skewed")
    off, rows, pos = er.plan_ref(idx, E)
    plan = make_plan(idx, E, 0, ws, dev)
    xq = rt.quantize(to_dev(bits((T, D), T, 2.0), dev), ws)
    hq = rt.quantize(to_dev(bits((T * k, D), T, 0.5), dev), ws)
    wg = rt.quantize_grouped_weights(to_dev(bits((E, 2 * F, D), D, D ** -0.5), dev), ws)
    w = np.random.default_rng(T).uniform(0.05, 0.6, (T, k)).astype(np.float32)
    wt = torch.from_numpy(w).to(dev)
    h, out = rt.grouped_swiglu(xq, wg, plan), rt.grouped_combine(hq, wg, plan, wt, ws)
    torch.cuda.synchronize()
    ref, bound = er.swiglu_ref(host(xq), host_groups(wg), off, rows, k)
    fails = er.check_close("h", f64(h), ref, bound)
    ref, bound = er.combine_ref(host(hq), host_groups(wg), off, pos, w)
    fails += er.check_close("out", f64(out), ref, bound)
    assert not fails, "\n".join(fails)
    for call in (lambda w2: rt.grouped_swiglu(xq, w2, plan), lambda w2: rt.grouped_combine(hq, w2, plan, wt, ws)):
        with pytest.raises(rt.RouterError):
            call(rt.GroupedWeights(wg.codes, shifted(wg.scales, 2), wg.gscale))
    for by in (4, 8, 12):
        wb = rt.GroupedWeights(wg.codes, shifted(wg.scales, by), wg.gscale)
        log(f"weight scales at {by} bytes")
        assert torch.equal(rt.grouped_swiglu(xq, wb, plan), h), by
        assert torch.equal(rt.grouped_combine(hq, wb, plan, wt, ws), out), by
        torch.cuda.synchronize()


@pytest.mark.parametrize("T,k,E,F,D", [
    (2, 4, 8, 48, 448), (2, 4, 8, 48, 352), (2, 4, 8, 80, 1120), (40, 8, 96, 288, 448), (40, 8, 96, 288, 416),
    (40, 8, 96, 288, 1056), (64, 4, 16, 1040, 448), (64, 4, 16, 1040, 352), (300, 7, 40, 1024, 192),
    (1400, 8, 40, 704, 832), (1400, 8, 40, 704, 544), (1400, 8, 40, 704, 288), (1400, 8, 40, 2080, 96),
    (1400, 8, 40, 704, 256), (2, 4, 8, 48, 512),
])
def test_a_nan_scale_stays_in_its_row(dev, ws, T, k, E, F, D):
    """Weight rows whose scales are all NaN make their own outputs NaN and change no bit of the others, at every K: two
    K groups, 16- and 32-row tiles, 64- and 128-row tiles, small experts beside them. So does a token's row of x."""
    log(f"nan scales T={T} k={k} E={E} F={F} D={D}")
    idx = routing(T, k, E, T + F, "skewed")
    off, rows, _ = er.plan_ref(idx, E)
    plan = make_plan(idx, E, 0, ws, dev)
    xq = rt.quantize(to_dev(bits((T, D), T, 2.0), dev), ws)
    hq = rt.quantize(to_dev(bits((T * k, D), T, 0.5), dev), ws)
    wg = rt.quantize_grouped_weights(to_dev(bits((E, 2 * F, D), D, D ** -0.5), dev), ws)
    w = torch.from_numpy(np.random.default_rng(T).uniform(0.05, 0.6, (T, k)).astype(np.float32)).to(dev)

    def both(x, h, wt):
        return rt.grouped_swiglu(x, wt, plan), rt.grouped_combine(h, wt, plan, w, ws)

    clean = both(xq, hq, wg)
    bad_row = 1 + 37 * np.arange(E) % (2 * F - 1)  # one of each expert's rows; the row before it is sound
    scales = wg.scales.clone()
    scales[torch.arange(E), torch.from_numpy(bad_row)] = torch.tensor([0x7F, 0xFF], dtype=torch.uint8,
                                                                      device=dev).repeat(D // 32)
    bad = both(xq, hq, rt.GroupedWeights(wg.codes, scales, wg.gscale))
    expert = np.repeat(np.arange(E), np.diff(off))
    nan_h, nan_out = np.zeros((T * k, F), bool), np.zeros((T, 2 * F), bool)
    nan_h[np.arange(T * k), bad_row[expert] % F] = True
    nan_out[rows // k, bad_row[expert]] = True
    t = T // 2
    xs, hs = xq.scales.clone(), hq.scales.clone()
    xs[t, 0] = hs[int(off[-1]) // 2, -1] = 0x7F
    one = both(rt.NVFP4Tensor(xq.codes, xs, xq.gscale), rt.NVFP4Tensor(hq.codes, hs, hq.gscale), wg)
    torch.cuda.synchronize()
    nan_x, nan_t = np.zeros((T * k, F), bool), np.zeros((T, 2 * F), bool)
    nan_x[rows // k == t] = True
    nan_t[rows[int(off[-1]) // 2] // k] = True
    for what, got, want, nan in (("h", bad[0], clean[0], nan_h), ("out", bad[1], clean[1], nan_out),
                                 ("h of x", one[0], clean[0], nan_x), ("out of h", one[1], clean[1], nan_t)):
        nan = torch.from_numpy(nan).to(dev)
        assert not torch.any(torch.isnan(want))
        assert torch.equal(torch.isnan(got), nan), (what, int(torch.isnan(got).sum()), int(nan.sum()))
        assert torch.equal(got[~nan], want[~nan]), what


@pytest.mark.parametrize("T,k,G,F,D", [(2, 4, 8, 48, 352), (64, 4, 16, 1040, 448), (300, 7, 40, 1024, 192),
                                       (1400, 8, 40, 704, 288), (1400, 8, 40, 2080, 96)])
@pytest.mark.parametrize("kind", ["every other", "stray", "falling", "past the end"])
def test_offsets_that_no_plan_gives(dev, ws, T, k, G, F, D, kind):
    """Offsets, rows and positions of no plan: their results are undefined, what lies around the outputs is untouched,
    and the next call with a plan is right."""
    log(f"offsets {kind} T={T} k={k} G={G} F={F} D={D}")
    R, r = T * k, np.random.default_rng(G)
    lo, hi = np.iinfo(np.int32).min, np.iinfo(np.int32).max
    off = {"every other": np.arange(G + 1) % 2 * R, "stray": r.integers(lo, hi, G + 1),
           "falling": R - np.arange(G + 1) * (R // G), "past the end": np.arange(G + 1) * R}[kind].astype(np.int32)
    idx = routing(T, k, G, T + F, "skewed")
    plan = make_plan(idx, G, 0, ws, dev)
    stray = [torch.from_numpy(v.astype(np.int32)).to(dev) for v in (off, r.integers(lo, hi, R), r.integers(lo, hi, R))]
    bad = [rt.GroupedPlan(*stray, T, k), rt.GroupedPlan(stray[0], plan.rows, plan.pos, T, k)]
    xq = rt.quantize(to_dev(bits((T, D), T, 2.0), dev), ws)
    hq = rt.quantize(to_dev(bits((R, D), T, 0.5), dev), ws)
    wg = rt.quantize_grouped_weights(to_dev(bits((G, 2 * F, D), D, D ** -0.5), dev), ws)
    w = torch.from_numpy(r.uniform(0.05, 0.6, (T, k)).astype(np.float32)).to(dev)
    used = rt.grouped_workspace_bytes(T, k, G, 2 * F, D)
    wsl = rt.Workspace(used + (1 << 20), dev)
    wsl.buf[used:] = 77
    want = rt.grouped_swiglu(xq, wg, plan), rt.grouped_combine(hq, wg, plan, w, ws)
    guard = 1 << 16
    outs = []
    for rows, cols in ((R, F), (T, 2 * F)):
        buf = torch.full((2 * guard + rows * cols,), 7.0, dtype=torch.bfloat16, device=dev)
        outs.append((buf, buf[guard:guard + rows * cols].view(rows, cols)))
    torch.cuda.synchronize()
    for p in bad + [plan]:
        rt.grouped_swiglu(xq, wg, p, out=outs[0][1])
        rt.grouped_combine(hq, wg, p, w, wsl, out=outs[1][1])
        torch.cuda.synchronize()
        for buf, _ in outs:
            assert torch.all(buf[:guard] == 7.0) and torch.all(buf[-guard:] == 7.0)
        assert torch.all(wsl.buf[used:] == 77) and torch.all(wsl.buf[:STATE] == 0)
    assert torch.equal(outs[0][1], want[0]) and torch.equal(outs[1][1], want[1])


def test_binding_refusals(dev, ws):
    T, D, E, k, F = 4, 64, 4, 2, 32
    x, gate, bias, w13, w2 = layer_inputs(dev, ws, T, D, E, k, F)
    xq, idx, w, plan, h, hq, out = run_layer(x, gate, bias, w13, w2, k, ws)
    bad = [
        lambda: rt.grouped_plan(idx.long(), E, ws),
        lambda: rt.grouped_plan(idx.t(), E, ws),
        lambda: rt.grouped_plan(idx, 0, ws),
        lambda: rt.grouped_plan(idx, E, ws, out=rt.empty_plan(T + 1, k, E, dev)),
        lambda: rt.grouped_plan(idx, E, ws, out=rt.empty_plan(T, k, E + 1, dev)),
        lambda: rt.grouped_swiglu(xq, w2, plan),
        lambda: rt.grouped_swiglu(hq, w13, plan),
        lambda: rt.grouped_swiglu(xq, w13, rt.empty_plan(T, k, E + 1, dev)),
        lambda: rt.grouped_swiglu(xq, w13, plan, bias=torch.zeros((E, F), device=dev)),
        lambda: rt.grouped_swiglu(xq, w13, plan, out=torch.empty((T * k, 2 * F), dtype=torch.bfloat16, device=dev)),
        lambda: rt.grouped_swiglu(xq, w13, plan, out=torch.empty((T * k, F), dtype=torch.float32, device=dev)),
        lambda: rt.grouped_combine(xq, w2, plan, w, ws),
        lambda: rt.grouped_combine(hq, w2, plan, w[:, :1], ws),
        lambda: rt.grouped_combine(hq, w2, plan, w, ws, residual=torch.zeros((T, D), device=dev)),
        lambda: rt.grouped_combine(hq, w2, plan, w, ws, bias=torch.zeros(D, device=dev)),
        lambda: rt.grouped_combine(hq, w2, plan, w, rt.Workspace(1 << 16, dev)),
        lambda: rt.grouped_combine(hq, w2, plan, w.cpu(), ws),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(rt.RouterError):
            f()
            pytest.fail(f"call {i} was not refused")


@pytest.mark.parametrize("T,D,E,k,F", [(2048, 2048, 32, 8, 768), (1200, 2080, 16, 6, 1312)])
def test_large_layer_sampled(dev, T, D, E, k, F):
    """Prefill sizes: sampled rows and tokens against the oracle."""
    wsl = rt.Workspace(max(rt.workspace_bytes(T, D, E, k), rt.grouped_workspace_bytes(T, k, E, D, F)), dev)
    x, gate, bias, w13, w2 = layer_inputs(dev, wsl, T, D, E, k, F, seed=11)
    log(f"large layer T={T} D={D} E={E} k={k} F={F}")
    xq, idx, w, plan, h, hq, out = run_layer(x, gate, bias, w13, w2, k, wsl)
    torch.cuda.synchronize()
    off, rows, pos = er.plan_ref(idx.cpu().numpy(), E)
    assert np.array_equal(plan.rows.cpu().numpy(), rows)
    xh, hh, w13h, w2h = host(xq), host(hq), host_groups(w13), host_groups(w2)
    fails = []
    for g in (0, 7, E - 1):
        a, b = int(off[g]), int(off[g + 1])
        pick = np.unique(np.concatenate([np.arange(a, min(a + 3, b)), np.arange(max(b - 3, a), b)]))
        ref, bound = er.swiglu_ref(xh, [w13h[g]], [0, len(pick)], rows[pick], k)
        fails += er.check_close(f"h of expert {g}", f64(h)[pick], ref, bound)
    toks = np.array([0, 1, 777, T - 1])
    slots = (toks[:, None] * k + np.arange(k)).reshape(-1)
    p = pos[slots]
    # One row per slot, each with its own expert's weights.
    e = np.searchsorted(off, p, side="right") - 1
    ref, bound = er.combine_ref((hh[0][p], hh[1][p], hh[2]), [w2h[i] for i in e], np.arange(len(p) + 1),
                                np.arange(len(p)), w.cpu().numpy()[toks],
                                residual=quant_ref.bf16_bits_to_f64(x.cpu().numpy().view(np.uint16)[toks]))
    fails += er.check_close("out", f64(out)[toks], ref, bound)
    assert not fails, "\n".join(fails)
