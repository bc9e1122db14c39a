"""GPU tests of the lm_head's losses where they lose something most easily: NaN, near-certain tokens, cold temperatures,
roundings, workspaces made for more rows."""

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_06_amd import router as rt
from nvfp4_block_scaled_06_amd import workloads as wl
from oracle import loss_ref as lr

pytestmark = pytest.mark.gpu

NAN8 = 0x7F  # an E4M3 scale that is NaN


def log(msg):
    print(f"[gpu-loss-limits] {msg}", flush=True)


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
    ws = rt.Workspace(rt.workspace_bytes(a.shape[0], a.shape[1], 1, 1), dev)
    return rt.quantize(up(wl.bf16_bits(a.astype(np.float32)).view(np.int16), dev), ws)


def operands(T, D, N, seed, dev, scale=1.0):
    r = np.random.default_rng(seed)
    return quantized(scale * r.standard_normal((T, D)), dev), quantized(1.5 * D ** -0.5 * r.standard_normal((N, D)), dev)


def workspace(T, D, N, grad, dev):
    return rt.Workspace(rt.lmhead_loss_workspace_bytes(T, D, N, grad), dev)


def host(q):
    return q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.gscale.cpu().numpy()[0]


def copy(q):
    return rt.NVFP4Tensor(q.codes.clone(), q.scales.clone(), q.gscale.clone())


# Streams of 16 rows, of 32 rows, and wide tiles.
NAN_SIZES = [(4, 96, 2000), (20, 256, 1500), (70, 128, 13000)]


@pytest.mark.parametrize("T,D,N", NAN_SIZES)
def test_rows_of_nan(dev, T, D, N):
    """A row of x with NaN has NaN for everything but an ignored target's loss and gradient; the others keep their bits."""
    xq, wq = operands(T, D, N, 1, dev)
    y = np.random.default_rng(2).integers(0, N, T).astype(np.int32)
    y[2] = -100
    bad = [1, 2, T - 1]
    xn = copy(xq)
    xn.scales[bad] = NAN8
    log(f"rows of NaN T={T} D={D} N={N}")
    for grad in (False, True):
        ws = workspace(T, D, N, grad, dev)
        want = rt.lmhead_loss(xq, wq, up(y, dev), ws, want_grad=grad)
        got = rt.lmhead_loss(xn, wq, up(y, dev), ws, want_grad=grad)
        torch.cuda.synchronize()
        rest = [t for t in range(T) if t not in bad]
        for u, v in zip(got, want):
            assert u is v is None or torch.equal(u[rest], v[rest])
        assert torch.isnan(got[1][bad]).all()
        assert torch.isnan(got[0][[1, T - 1]]).all() and got[0][2] == 0
        if grad:
            assert torch.isnan(got[2][[1, T - 1]].float()).all() and not got[2][2].any()


@pytest.mark.parametrize("T,D,N", NAN_SIZES)
def test_columns_of_nan(dev, T, D, N):
    """Weight rows of NaN, wherever they lie and whatever they fill, make every row's sum NaN."""
    xq, wq = operands(T, D, N, 3, dev)
    y = up(np.random.default_rng(4).integers(0, 5, T).astype(np.int32), dev)
    for a, b in ((7, 8), (64, 96), (64, 80), (96, 112), (128, 192), (512, 1024), (N - 3, N), (N - N % 64, N), (0, N)):
        wn = copy(wq)
        wn.scales[a:b] = NAN8
        log(f"columns of NaN T={T} D={D} N={N} {a}:{b}")
        for grad in (False, True):
            loss, lse, dx = rt.lmhead_loss(xq, wn, y, workspace(T, D, N, grad, dev), want_grad=grad)
            torch.cuda.synchronize()
            assert torch.isnan(lse).all() and torch.isnan(loss).all(), (a, b, grad)
            assert not grad or torch.isnan(dx.float()).all(), (a, b)


@pytest.mark.parametrize("T,D,N", NAN_SIZES)
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_global_scales_that_are_not_finite(dev, T, D, N, value):
    xq, wq = operands(T, D, N, 5, dev)
    y = torch.full((T,), -100, dtype=torch.int32, device=dev)
    for which in (0, 1):
        q = [copy(xq), copy(wq)]
        q[which].gscale.fill_(value)
        loss, lse, _ = rt.lmhead_loss(*q, y, workspace(T, D, N, False, dev))
        torch.cuda.synchronize()
        assert torch.isnan(lse).all() and not loss.any()


def test_teacher_nan_is_kept(dev):
    """A NaN of a token that counts makes its row NaN, wherever it stands and whatever else the row holds; lse and logq,
    which do not depend on the teacher, are those of a row without it."""
    T, D, N, K = 12, 64, 300, 200
    xq, wq = operands(T, D, N, 6, dev)
    r = np.random.default_rng(7)
    tok = r.integers(0, N, (T, K)).astype(np.int32)
    tok[:, 5] = 17  # named by every row
    clean = r.standard_normal((T, K)).astype(np.float32)
    clean[1::2] = -np.inf  # nothing else in the row counts
    clean[1::2, 150] = 1.0
    te = clean.copy()
    at = [0, 1, 5, 5, 63, 64, 69, 69, 128, 191, 199, 199]
    for t in range(T):
        te[t] = np.where(np.isinf(te[t]) | (t % 2 == 1), -np.inf, te[t])
        te[t, at[t]] = np.nan
        tok[t, at[t]] = 100 + t
    ws = workspace(T, D, N, True, dev)
    want = rt.lmhead_distill(xq, wq, up(tok, dev), up(clean, dev), ws, want_grad=True)
    got = rt.lmhead_distill(xq, wq, up(tok, dev), up(te, dev), ws, want_grad=True)
    torch.cuda.synchronize()
    assert torch.isnan(got[0]).all() and torch.isnan(got[3].float()).all()
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    assert torch.isfinite(want[0]).all() and torch.isfinite(got[1]).all() and torch.isfinite(got[2]).all()
    tok[:, 5] = -1
    for t in range(T):
        tok[t, at[t]] = -1  # left out: whatever its teacher's logit is
    got = rt.lmhead_distill(xq, wq, up(tok, dev), up(te, dev), ws, want_grad=True)
    torch.cuda.synchronize()
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[3].float()).all()


@pytest.mark.parametrize("T,N", [(1, 192), (20, 192), (64, 30016)])
def test_softmax_weights_are_rounded_once(dev, T, N):
    """Three levels of logits, 7, 2.1 and 1.1667 in base 2, of which the lowest shares its block with the second and 57 of its
    columns cancel one of the highest in dx: what is left shows how often the weights 2^-5.83 were rounded to 11 bits. (Once
    with the block's own scale, once as that is brought to the row's and once as both are multiplied: 2.5 half steps.)"""
    D = 64
    wc, ws8 = np.zeros((N, D // 2), np.uint8), np.full((N, D // 16), 0x38, np.uint8)
    wc[:64, 0], ws8[:64, 0] = 7, 0x3A          # 6 * 1.25
    wc[64:128, 0], ws8[64:128, 0] = 2, 0x3A    # 1 * 1.25
    wc[[64, 80], 0], ws8[[64, 80], 0] = 7, 0x2C  # 6 * 0.375, in each block of 32 of these 64
    low = [n for n in range(64, 128) if n not in (64, 80)][:57]
    wc[5, 16:24], wc[low, 16:24] = 0x77, 0xFF  # +6 and -6 where x is 0
    xc, xs = np.zeros((T, D // 2), np.uint8), np.full((T, D // 16), 0x38, np.uint8)
    xc[:, 0] = 7
    gsa = np.float32(7.0 / (np.log2(np.e) * 6 * 7.5))
    q = lambda c, s, g: rt.NVFP4Tensor(up(c, dev), up(s, dev), torch.tensor([g], device=dev))
    xq, wq = q(xc, xs, gsa), q(wc, ws8, 1.0)
    y = np.full((T, 1), 130, np.int32)
    log(f"one rounding T={T} N={N}")
    _, _, dx = rt.lmhead_loss(xq, wq, up(y[:, 0], dev), workspace(T, D, N, True, dev), want_grad=True)
    torch.cuda.synchronize()
    want = lr.loss_ref(host(xq), host(wq), y)["dx"][0][:, 32:48]
    z = lr.dequant_ref(*host(xq))[:1] @ lr.dequant_ref(*host(wq)).T
    p = np.exp(z - lr._lse(z)[:, None])[0]
    share = 6 * p[low].sum()
    # One half step of 11 bits, 2^-11; 2^-17 for the exponential of arguments up to 7 and the sums in fp32; bf16 at the end.
    bound = share * (2.0 ** -11 + 2.0 ** -17) + 2.0 ** -8 * np.abs(want)
    assert np.abs(want).max() < 0.01 * share
    err = np.abs(dx[:, 32:48].double().cpu().numpy() - want)
    assert (err <= bound).all(), (err.max() / share * 2048, bound.max() / share * 2048)


CONF_SIZES = [(4, 256, 900), (16, 1280, 700), (20, 96, 5000), (40, 1056, 1100), (70, 128, 13000), (130, 288, 9000)]


@pytest.mark.parametrize("T,D,N", CONF_SIZES)
@pytest.mark.parametrize("scale", [1.0, 60.0])
def test_no_probability_exceeds_one(dev, T, D, N, scale):
    """The row's own best token: its loss is a logarithm of 1 and more, so not below 0, at any temperature; where the
    second best is far behind both are 0 but for a few steps of 1, however large the logits over the temperature are."""
    xq, wq = operands(T, D, N, 11, dev, scale)
    z = lr.dequant_ref(*host(xq)) @ lr.dequant_ref(*host(wq)).T
    top = np.sort(z, axis=1)[:, -2:]
    err = (D + 8) * 2.0 ** -24 * (np.abs(lr.dequant_ref(*host(xq))) @ np.abs(lr.dequant_ref(*host(wq))).T).max(axis=1)
    best = z.argmax(axis=1).astype(np.int32)
    ws = workspace(T, D, N, True, dev)
    wmax = np.abs(lr.dequant_ref(*host(wq))).sum(axis=0)
    log(f"confident T={T} D={D} N={N} scale={scale}")
    loss, lse, dx = rt.lmhead_loss(xq, wq, up(best, dev), ws, want_grad=True)
    torch.cuda.synchronize()
    assert (loss >= 0).all()
    for K in (1, 3, 9):
        tok = np.tile(best[:, None], (1, K))
        tok[:, 1:] = np.random.default_rng(K).integers(0, N, (T, K - 1))
        te = np.full((T, K), -np.inf, np.float32)
        te[:, 0] = 3.0
        for tau in (2.0 ** -6, 2.0 ** -10, 2.0 ** -15, 2.0 ** -20):
            loss, lse, logq, dx = rt.lmhead_distill(xq, wq, up(tok, dev), up(te, dev), ws, temperature=tau, want_grad=True)
            torch.cuda.synchronize()
            loss, logq, dx = loss.double().cpu().numpy(), logq.double().cpu().numpy(), dx.double().cpu().numpy()
            assert (logq <= 0).all() and (loss >= 0).all(), (K, tau, logq.max(), loss.min())
            sure = (top[:, 1] - top[:, 0] - 2 * err) / tau > 40.0  # N e^-40 is below 2^-24
            # The sum's roundings: at most 2^-24 for each of the 64 and more steps of its tree.
            assert (-logq[sure, 0] <= 2.0 ** -18).all() and (loss[sure] <= tau * tau * 2.0 ** -18).all()
            assert (np.abs(dx[sure]) <= tau * 2.0 ** -18 * wmax + 2.0 ** -133).all()
            if tau <= 2.0 ** -10 and scale > 1:
                assert sure.any()


@pytest.mark.parametrize("tau", [2.0 ** -4, 2.0 ** -8])
def test_cold_temperatures(dev, tau):
    """Against float64 on the logits that the device itself sums, whose roundings the temperature magnifies for any
    evaluation: they are taken from lmhead_argmax and counted; the quotients by the temperature are not."""
    T, D, N, K = 4, 1024, 5003, 6
    xq, wq = operands(T, D, N, 12, dev, 2.0)
    ws = rt.Workspace(max(rt.lmhead_workspace_bytes(T, D, N), rt.lmhead_loss_workspace_bytes(T, D, N, True)), dev)
    _, _, logits = rt.lmhead_argmax(xq, wq, ws, want_logits=True)
    torch.cuda.synchronize()
    z = logits.double().cpu().numpy()
    order = np.argsort(-z, axis=1)
    tok = order[:, :K].astype(np.int32)
    te = np.take_along_axis(z, tok, 1).astype(np.float32) + np.random.default_rng(1).uniform(-tau, tau, (T, K)).astype(np.float32)
    loss, lse, logq, _ = rt.lmhead_distill(xq, wq, up(tok, dev), up(te, dev), ws, temperature=tau, want_grad=True)
    torch.cuda.synchronize()
    # Two sums of D products in fp32 with random signs: partial sums stay below 6 times the products' norm, and at most D
    # roundings of half a step of those, with random signs too, add up to sqrt(D) of them.
    norm = np.sqrt((lr.dequant_ref(*host(xq)) ** 2) @ (lr.dequant_ref(*host(wq)) ** 2).T).max()
    err = 2 * D ** 0.5 * 2.0 ** -24 * 6 * norm / tau
    zt = z / tau
    ref = lr._lse(zt)
    want = np.take_along_axis(zt, tok, 1) - ref[:, None]
    got = logq.double().cpu().numpy()
    bound = 2 * err + 2.0 ** -18 + 2.0 ** -21 * np.abs(want)
    assert (np.abs(got - want) <= bound).all(), (np.abs(got - want) / bound).max()
    t = te.astype(np.float64) / tau
    p = np.exp(t - lr._lse(t)[:, None])
    kl = (p * (t - lr._lse(t)[:, None] - want)).sum(axis=1)
    assert (np.abs(loss.double().cpu().numpy() - tau * tau * kl) <= tau * tau * (bound.max() + 2.0 ** -18)).all()


def test_largest_teacher_logits(dev):
    """Finite teacher logits give finite losses, also where their quotients by the temperature would not be."""
    T, D, N, K = 3, 64, 200, 4
    xq, wq = operands(T, D, N, 13, dev)
    big = np.finfo(np.float32).max
    te = np.tile(np.array([[big, 0.0, -big, big]], np.float32), (T, 1))
    tok = np.tile(np.array([[3, 4, 5, 6]], np.int32), (T, 1))
    loss, _, logq, dx = rt.lmhead_distill(xq, wq, up(tok, dev), up(te, dev), workspace(T, D, N, True, dev), temperature=0.5,
                                          want_grad=True)
    torch.cuda.synchronize()
    want = 0.25 * (-np.log(2.0) - logq.double().cpu().numpy()[:, [0, 3]].mean(axis=1))
    assert np.abs(loss.double().cpu().numpy() - want).max() <= 1e-5 and torch.isfinite(dx.float()).all()


@pytest.mark.parametrize("D,N,most", [(96, 13000, 130), (256, 6000, 300), (1024, 2000, 140)])
def test_a_workspace_for_more_rows(dev, D, N, most):
    """A workspace made for the most rows, with the gradient, takes every call with fewer, with the gradient and without."""
    _, wq = operands(1, D, N, 20, dev)
    xq = quantized(np.random.default_rng(21).standard_normal((most, D)), dev)
    y = up(np.random.default_rng(22).integers(0, N, most).astype(np.int32), dev)
    ws = workspace(most, D, N, True, dev)
    for T in (0, 1, 16, 17, 32, 33, 64, 65, 96, 128, 129, most):
        if T > most:
            continue
        log(f"workspace for {most} rows, T={T} D={D} N={N}")
        part = rt.NVFP4Tensor(xq.codes[:T], xq.scales[:T], xq.gscale)
        got = rt.lmhead_loss(part, wq, y[:T], ws, want_grad=True)
        alone = rt.lmhead_loss(part, wq, y[:T], ws)
        want = rt.lmhead_loss(part, wq, y[:T], workspace(T, D, N, True, dev), want_grad=True)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert alone[2] is None and torch.allclose(alone[0], got[0], rtol=1e-5, atol=1e-5)
