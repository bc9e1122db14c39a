"""GPU parity of lmhead_penalize against the CPU oracle, through the C ABI."""

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_06_amd import router as rt
from nvfp4_block_scaled_06_amd import workloads as wl
from oracle import penalize_ref as pr

pytestmark = pytest.mark.gpu


def log(msg):
    print(f"[gpu-penalize] {msg}", flush=True)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    rt.load_library()
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    return d


def make(T, N, L, nbias, mask, dtype, seed, dev):
    r = np.random.default_rng(seed)
    x = (3 * r.standard_normal((T, N))).astype(np.float32)
    if dtype == torch.bfloat16:
        x = wl.bf16_to_f32(wl.bf16_bits(x))
    a = {}
    if L:
        a["history"] = (N ** r.random((T, L)) - 1).astype(np.int32)
        a["history"][r.random((T, L)) < 0.05] = -1
        a["history"][r.random((T, L)) < 0.05] = N
        a["history"][0, 0] = np.iinfo(np.int32).min
        a["lengths"] = r.integers(0, L + 1, T).astype(np.int32)
        a["lengths"][0] = L
        a["prompt"] = r.integers(0, L + 1, T).astype(np.int32)
    a["repetition"] = r.uniform(0.8, 1.5, T).astype(np.float32)
    a["frequency"] = r.uniform(-0.5, 0.5, T).astype(np.float32)
    a["presence"] = r.uniform(-0.5, 0.5, T).astype(np.float32)
    if nbias:
        n = r.integers(0, nbias + 1, T)
        tok = r.integers(-1, N + 1, n.sum()).astype(np.int32)  # repeated and stray tokens among them
        a["bias"] = (np.concatenate([[0], np.cumsum(n)]).astype(np.int32), tok,
                     r.standard_normal(n.sum()).astype(np.float32))
    if mask:
        a["mask"] = r.integers(0, 2 ** 32, (T, (N + 31) // 32), dtype=np.uint32)
    return x, a


def on_dev(a, dev):
    up = lambda v: torch.from_numpy(np.ascontiguousarray(v).view(np.int32) if v.dtype == np.uint32 else v).to(dev)
    return {k: tuple(up(x) for x in v) if isinstance(v, tuple) else up(v) for k, v in a.items()}


def check(x, a, dtype, idx, logit, out):
    ref, err = pr.penalize_ref(x, **a)
    idx, logit, out = idx.cpu().numpy(), logit.cpu().numpy().astype(np.float64), out.float().cpu().numpy()
    fails = pr.check_choice(idx, logit, ref, err)
    bound = err + (2.0 ** -8 * (np.abs(ref) + err) if dtype == torch.bfloat16 else 0.0)
    with np.errstate(invalid="ignore"):
        ok = (out == ref) | (np.abs(out - ref) <= bound) | (np.isnan(out) & np.isnan(ref))
    assert not fails, "\n".join(fails)
    assert np.all(ok), (np.argwhere(~ok)[:5], out[~ok][:5], ref[~ok][:5])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N,L,nbias,mask", [
    (1, 1, 1, 0, False), (2, 31, 5, 3, True), (3, 4096, 100, 10, True), (2, 4097, 700, 40, True),
    (4, 8192, 64, 0, False), (5, 9001, 2000, 64, True), (1, 20000, 0, 5, True), (3, 12292, 300, 0, False),
])
def test_parity(dev, T, N, L, nbias, mask, dtype):
    log(f"T={T} N={N} L={L} nbias={nbias} mask={mask} {dtype}")
    x, a = make(T, N, L, nbias, mask, dtype, N, dev)
    ws = rt.Workspace(rt.lmhead_penalize_workspace_bytes(T, N), dev)
    xd = torch.from_numpy(x).to(dev).to(dtype)
    idx, logit, out = rt.lmhead_penalize(xd, ws, **on_dev(a, dev))
    torch.cuda.synchronize()
    check(x, a, dtype, idx, logit, out)
    again = xd.clone()  # in place
    i2, l2, o2 = rt.lmhead_penalize(again, ws, out=again, **on_dev(a, dev))
    torch.cuda.synchronize()
    assert o2 is again and torch.equal(again, out) and torch.equal(i2, idx) and torch.equal(l2, logit)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_row_strides(dev, dtype):
    """Rows longer than the vocabulary, and rows that no 16-byte access may touch; what lies between stays."""
    T, N = 3, 5003
    for ld, shift in ((5008, 0), (5009, 0), (5008, 1)):
        x, a = make(T, N, 50, 8, True, dtype, ld, dev)
        buf = torch.full((T * ld + shift + 16,), 7.0, dtype=dtype, device=dev)
        view = buf[shift:shift + T * ld].view(T, ld)[:, :N]
        view.copy_(torch.from_numpy(x).to(dev))
        wide = on_dev(a, dev)
        wide["history"] = torch.nn.functional.pad(wide["history"], (0, 9))[:, :50]
        wide["mask"] = torch.nn.functional.pad(wide["mask"], (0, 3))
        ws = rt.Workspace(rt.lmhead_penalize_workspace_bytes(T, N), dev)
        log(f"row stride {ld}, shift {shift}, {dtype}")
        idx, logit, out = rt.lmhead_penalize(view, ws, out=view, **wide)
        torch.cuda.synchronize()
        check(x, a, dtype, idx, logit, out)
        rest = torch.ones_like(buf, dtype=torch.bool)
        rest[shift:shift + T * ld].view(T, ld)[:, :N] = False
        assert torch.all(buf[rest] == 7.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ldo", [5003, 5008, 5016])
def test_logits_of_every_position(dev, dtype, ldo):
    """The last position's logits of [T, S, N]: the output's rows have a stride of their own."""
    T, S, N = 3, 4, 5003
    x, a = make(T, N, 50, 8, True, dtype, ldo, dev)
    every = torch.full((T, S, N), 7.0, dtype=dtype, device=dev)
    every[:, -1] = torch.from_numpy(x).to(dev)
    ws = rt.Workspace(rt.lmhead_penalize_workspace_bytes(T, N), dev)
    wide = on_dev(a, dev)
    log(f"output stride {ldo}, {dtype}")
    idx, logit, out = rt.lmhead_penalize(every[:, -1], ws, **wide)
    assert out.is_contiguous()
    buf = torch.full((T, ldo), 7.0, dtype=dtype, device=dev)
    i2, l2, o2 = rt.lmhead_penalize(every[:, -1], ws, out=buf[:, :N], **wide)
    torch.cuda.synchronize()
    check(x, a, dtype, idx, logit, out)
    assert torch.equal(o2.nan_to_num(), out.nan_to_num()) and torch.equal(i2, idx) and torch.equal(l2, logit)
    assert torch.all(buf[:, N:] == 7.0)
    assert torch.equal(every[:, -1].cpu(), torch.from_numpy(x).to(dtype)) and torch.all(every[:, :-1] == 7.0)


def check_rows(x, a, dtype, idx, logit, out):
    """check() with the oracle that takes a row at a time."""
    ref, err = pr.penalize_rows(x, **a)
    out = out.float().cpu().numpy()
    fails = pr.check_choice(idx.cpu().numpy(), logit.cpu().numpy().astype(np.float64), ref, err)
    assert not fails, "\n".join(fails[:5])
    bound = err + (2.0 ** -8 * (np.abs(ref) + err) if dtype == torch.bfloat16 else 0.0)
    with np.errstate(invalid="ignore"):
        ok = (out == ref) | (np.abs(out - ref) <= bound)
    assert np.all(ok), (np.argwhere(~ok)[:5], out[~ok][:5], ref[~ok][:5])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N,L,nbias", [(5, 9001, 4097, 513), (5, 9001, 9000, 1500), (9, 4096, 4608, 1024),
                                         (70, 49160, 4500, 700)])
def test_long_lists(dev, T, N, L, nbias, dtype):
    """Histories past the 4096 tokens, and biases past the 512 of a row, that stay in registers: prompts that end on
    either side of the 4096th token, tokens biased on both sides of the 512th entry, whose last value counts."""
    log(f"T={T} N={N} L={L} nbias={nbias} {dtype}")
    x, a = make(T, N, L, 0, True, dtype, N + L, dev)
    r = np.random.default_rng(L)
    a["lengths"][:5] = L, L, L, 4096, 4097
    a["prompt"][:5] = 0, 4095, 4097, 4000, 4096
    tok = r.integers(-1, N + 1, (T, nbias)).astype(np.int32)
    tok[:, 512:] = np.where(r.random((T, nbias - 512)) < 0.5, tok[:, :nbias - 512], tok[:, 512:])
    tok[:, 512], tok[:, -1] = tok[:, 0], tok[:, 511]
    a["bias"] = (np.arange(0, T * nbias + 1, nbias, dtype=np.int32), tok.reshape(-1),
                 r.standard_normal(T * nbias).astype(np.float32))
    ws = rt.Workspace(rt.lmhead_penalize_workspace_bytes(T, N), dev)
    got = rt.lmhead_penalize(torch.from_numpy(x).to(dev).to(dtype), ws, **on_dev(a, dev))
    torch.cuda.synchronize()
    check_rows(x, a, dtype, *got)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N", [(100, 65541), (257, 16389), (780, 8195)])
def test_workgroups_of_several_chunks(dev, T, N, dtype, shift):
    """More chunks of 4096 tokens than resident workgroups: each takes several in turn, of a row's (17, 5 and 3) that one
    or several workgroups share; 16 bytes and one element at a time, out of place and in place."""
    log(f"T={T} N={N} {dtype} shift {shift}")
    x, a = make(T, N, 700, 40, True, dtype, N, dev)
    ld = (N + 15) // 8 * 8
    buf = torch.full((T * ld + 16,), 7.0, dtype=dtype, device=dev)
    view = buf[shift:shift + T * ld].view(T, ld)[:, :N]
    view.copy_(torch.from_numpy(x).to(dev))
    ws = rt.Workspace(rt.lmhead_penalize_workspace_bytes(T, N), dev)
    up = on_dev(a, dev)
    idx, logit, out = rt.lmhead_penalize(view, ws, **up)
    i2, l2, _ = rt.lmhead_penalize(view, ws, out=view, **up)
    torch.cuda.synchronize()
    check_rows(x, a, dtype, idx, logit, out)
    assert torch.equal(view, out) and torch.equal(i2, idx) and torch.equal(l2, logit)
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[shift:shift + T * ld].view(T, ld)[:, :N] = False
    assert torch.all(buf[rest] == 7.0)


def test_bias_starts_out_of_range(dev):
    """Starts that no list has are clamped to its ends; a row that ends before it starts has no biases."""
    lo, hi = np.iinfo(np.int32).min, np.iinfo(np.int32).max
    n, N, r = 700, 9001, np.random.default_rng(3)
    starts = np.array([hi, -5, hi - 300, 3, lo, n + 1, 650, 640, hi, lo, lo, n - 1, hi, hi], dtype=np.int32)
    rows = np.clip(starts, 0, n)
    T = len(starts) - 1
    tok = r.permutation(N)[:n].astype(np.int32)
    val = r.standard_normal(n).astype(np.float32)
    x = r.standard_normal((T, N)).astype(np.float32)
    parts = [np.arange(rows[t], max(rows[t + 1], rows[t])) for t in range(T)]
    assert [len(q) for q in parts] == [0, 700, 0, 0, 700, 0, 0, 60, 0, 0, 699, 1, 0]
    listed = np.concatenate(parts)
    want = (np.concatenate([[0], np.cumsum([len(q) for q in parts])]), tok[listed], val[listed])
    ws = rt.Workspace(rt.lmhead_penalize_workspace_bytes(T, N), dev)
    log("bias starts out of range")
    got = rt.lmhead_penalize(torch.from_numpy(x).to(dev), ws, **on_dev({"bias": (starts, tok, val)}, dev))
    torch.cuda.synchronize()
    check(x, {"bias": want}, torch.float32, *got)
    none = rt.lmhead_penalize(torch.from_numpy(x).to(dev), ws, **on_dev({"bias": (starts, tok[:0], val[:0])}, dev))
    torch.cuda.synchronize()
    check(x, {}, torch.float32, *none)


def test_special_values(dev):
    """Masked infinities and NaN, rows that the mask empties, ties, and nothing but the logits."""
    N = 4100
    x = np.zeros((6, N), dtype=np.float32)
    x[0, 10], x[0, 20], x[0, 30] = np.nan, np.inf, 5.0  # NaN and inf where the mask forbids them
    x[1] = np.nan
    x[2] = -np.inf
    x[3] = np.inf
    x[4, 7] = x[4, 4099] = 2.0
    x[5] = np.finfo(np.float32).min
    x[5, 4098] = -np.inf
    mask = np.full((6, (N + 31) // 32), 0xFFFFFFFF, dtype=np.uint32)
    mask[0, 0] &= ~np.uint32((1 << 10) | (1 << 20))
    mask[3] = 0
    mask[5, 0] = 0
    ws = rt.Workspace(rt.lmhead_penalize_workspace_bytes(6, N), dev)
    log("special values")
    xd = torch.from_numpy(x).to(dev)
    idx, logit, out = rt.lmhead_penalize(xd, ws, mask=torch.from_numpy(mask.view(np.int32)).to(dev))
    torch.cuda.synchronize()
    assert idx.cpu().tolist() == [30, -1, -1, -1, 7, 32]
    assert logit.cpu().tolist()[:1] == [5.0] and logit.cpu().tolist()[1:4] == 3 * [-np.inf]
    o = out.cpu().numpy()
    assert o[0, 10] == -np.inf and o[0, 20] == -np.inf and np.all(np.isnan(o[1])) and np.all(o[3] == -np.inf)
    assert np.array_equal(o[4], x[4])
    assert np.all(o[5, :32] == -np.inf) and np.array_equal(o[5, 32:], x[5, 32:])


def test_more_rows_than_counters(dev):
    T, N = 1030, 4500
    x, a = make(T, N, 8, 2, False, torch.float32, 7, dev)
    ws = rt.Workspace(rt.lmhead_penalize_workspace_bytes(T, N), dev)
    log(f"T={T} N={N}")
    idx, logit, out = rt.lmhead_penalize(torch.from_numpy(x).to(dev), ws, **on_dev(a, dev))
    torch.cuda.synchronize()
    check(x, a, torch.float32, idx, logit, out)


def test_replays_in_a_graph_beside_the_lm_head(dev):
    """lmhead_argmax's logits constrained in place, captured once and replayed on the workspace of eager calls."""
    T, D, N, L = 2, 512, 9000, 40
    ws = rt.Workspace(max(rt.workspace_bytes(T, D, 8, 1), rt.lmhead_workspace_bytes(T, D, N),
                          rt.lmhead_penalize_workspace_bytes(T, N), rt.workspace_bytes(N, D, 8, 1)), dev)
    r = np.random.default_rng(5)
    x = torch.from_numpy(r.standard_normal((T, D)).astype(np.float32)).to(dev).to(torch.bfloat16)
    wq = rt.quantize(torch.from_numpy(r.standard_normal((N, D)).astype(np.float32)).to(dev).to(torch.bfloat16), ws)
    _, a = make(T, N, L, 5, True, torch.float32, 6, dev)
    a = on_dev(a, dev)

    def step():
        xq = rt.quantize(x, ws)
        _, _, logits = rt.lmhead_argmax(xq, wq, ws, want_logits=True)
        return rt.lmhead_penalize(logits, ws, out=logits, **a)

    log("graph")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for i in range(3):
        x.copy_(torch.from_numpy(r.standard_normal((T, D)).astype(np.float32)).to(dev).to(torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for p, q in zip(got, want):
            assert torch.equal(p, q), i


def test_binding_refusals(dev):
    T, N = 2, 5000
    ws = rt.Workspace(rt.lmhead_penalize_workspace_bytes(T, N), dev)
    x = torch.zeros((T, N), device=dev)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    bad = [
        dict(logits=x.half()), dict(logits=x[0]), dict(logits=x.t()), dict(history=i32(T + 1, 4)),
        dict(history=i32(T, 4).long()), dict(lengths=i32(T)), dict(history=i32(T, 4), lengths=i32(T + 1)),
        dict(repetition=i32(T)), dict(frequency=torch.zeros(T)), dict(presence=torch.zeros(1, device=dev)),
        dict(bias=(i32(T), i32(3), torch.zeros(3, device=dev))), dict(bias=(i32(T + 1), i32(3), i32(3))),
        dict(bias=(i32(T + 1), i32(3), torch.zeros(2, device=dev))), dict(mask=i32(T, 156)), dict(mask=i32(1, 157)),
        dict(out=torch.zeros((T, N + 1), device=dev)), dict(out=x.to(torch.bfloat16)), dict(out=x.cpu()),
        dict(workspace=rt.Workspace(1 << 12, dev)),
    ]
    for kw in bad:
        a = dict(logits=x, workspace=ws)
        a.update(kw)
        with pytest.raises(rt.RouterError):
            rt.lmhead_penalize(**a)
            pytest.fail(f"{list(kw)} was not refused")
