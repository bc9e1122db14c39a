"""CPU checks of the entry points of routing on given logits and of the lm_head's losses: sizes, refusals and empty
calls. No call here reaches a kernel launch."""

import ctypes
import os

import pytest
import torch

from nvfp4_block_scaled_06_amd import router as rt

P = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: validation fails first
STATE = 4096 + 128 * 1024
EINVAL, EUNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(rt.LIB_PATH):
        from nvfp4_block_scaled_06_amd import build

        build.build()
    return rt.load_library()


def off(by):
    return ctypes.c_void_p((1 << 20) + by)


class Call:
    def __init__(self, fn, **args):
        self.fn, self.args = fn, args

    def __call__(self, **kw):
        assert set(kw) <= set(self.args)
        return self.fn(*{**self.args, **kw}.values())


def test_select_refusals(lib):
    c = Call(lib.router_select, logits=P, dtype=0, T=4, E=64, ld=64, bias=P, scoring=0, groups=8, kept=4, top=2,
             renorm=1, scale=1.0, k=8, idx=P, w=P, s=None)
    for bad in [dict(dtype=2), dict(dtype=-1), dict(scoring=2), dict(scoring=-1), dict(T=-1), dict(E=0), dict(k=0),
                dict(k=65), dict(ld=63), dict(groups=0), dict(groups=7), dict(kept=0), dict(kept=9), dict(top=0),
                dict(top=3), dict(kept=1, k=9), dict(logits=None), dict(idx=None), dict(w=None),
                dict(logits=off(2)), dict(dtype=1, logits=off(1)), dict(bias=off(2)), dict(idx=off(2)), dict(w=off(1))]:
        assert c(**bad) == EINVAL, bad
    for bad in [dict(E=1024, ld=1024), dict(k=33, kept=8), dict(k=33, kept=4), dict(T=1 << 31), dict(ld=1 << 31),
                dict(E=130, ld=130, groups=65, kept=65, k=1), dict(E=520, ld=520, groups=65, kept=65)]:
        assert c(**bad) == EUNSUPPORTED, bad
    assert c(T=0) == 0
    assert c(T=0, logits=None, bias=None, idx=None, w=None) == 0


def test_select_most_rows(lib):
    """More rows than a launch takes are refused, by both calls."""
    a = dict(logits=P, dtype=0, T=(1 << 25) + 1, E=64, ld=64, bias=P, scoring=0, groups=8, kept=4, top=2, renorm=1,
             scale=1.0, k=8, idx=P, w=P, s=None)
    assert lib.router_select(*a.values()) == EUNSUPPORTED
    b = dict(logits=P, dtype=0, T=(1 << 25) + 1, E=64, ld=64, idx=P, gw=P, scoring=1, renorm=0, scale=1.0, k=8,
             out=off(1 << 20), ldo=64, s=None)
    assert lib.router_select_backward(*b.values()) == EUNSUPPORTED


def test_select_backward_refusals(lib):
    c = Call(lib.router_select_backward, logits=P, dtype=0, T=4, E=64, ld=64, idx=P, gw=P, scoring=1, renorm=0,
             scale=1.0, k=8, out=off(1 << 20), ldo=64, s=None)
    for bad in [dict(dtype=2), dict(scoring=2), dict(T=-1), dict(E=0), dict(k=0), dict(k=65), dict(ld=63),
                dict(ldo=63), dict(logits=None), dict(idx=None), dict(gw=None), dict(out=None), dict(logits=off(2)),
                dict(idx=off(2)), dict(gw=off(2)), dict(out=off(2)), dict(dtype=1, out=off(1))]:
        assert c(**bad) == EINVAL, bad
    for bad in [dict(E=1024, ld=1024, ldo=1024), dict(k=33), dict(T=1 << 31), dict(ldo=1 << 31)]:
        assert c(**bad) == EUNSUPPORTED, bad
    assert c(T=0, logits=None, idx=None, gw=None, out=None) == 0


def test_loss_workspace_sizes(lib):
    f = lib.lmhead_loss_workspace_bytes
    assert f(0, 32, 1, 0) >= STATE and f(0, 32, 1, 1) >= STATE
    for T, D, N in [(1, 7168, 129280), (64, 7168, 129280), (4096, 7168, 129280), (7, 32, 1), (300, 1056, 50021)]:
        fwd, bwd = f(T, D, N, 0), f(T, D, N, 1)
        assert STATE < fwd < bwd
        assert fwd < STATE + (1 << 16) + T * (N + 1024)  # maxima and sums of blocks of columns
        # Never the T x N logits: at most 512 MB of a piece's weights, or 4608 columns of them.
        assert bwd < (1 << 20) + 2 * max(T * 5120, 1 << 28) + T * (N + 16384) + 65 * T * D * 4 + (1 << 27)
        assert rt.lmhead_loss_workspace_bytes(T, D, N) == fwd and rt.lmhead_loss_workspace_bytes(T, D, N, True) == bwd
    assert f(1 << 18, 7168, 129280, 1) < 64 << 30
    for bad in [(-1, 32, 10), (1, 0, 10), (1, 48, 10), (1, 16, 10), (1, 32, 0), ((1 << 18) + 1, 32, 10),
                (1, (1 << 22) + 32, 10), (1, 32, (1 << 30) + 1)]:
        assert f(*bad, 0) == 0 and f(*bad, 1) == 0, bad
        with pytest.raises(rt.RouterError):
            rt.lmhead_loss_workspace_bytes(*bad)


def loss_call(lib, **kw):
    need = lib.lmhead_loss_workspace_bytes(4, 256, 1000, 1)
    return Call(lib.lmhead_loss, xc=P, xs=P, gsa=P, wc=P, ws=P, gsw=P, targets=P, weight=P, T=4, D=256, N=1000, loss=P,
                lse=P, dx=P, work=P, nbytes=need, s=None)


def distill_call(lib):
    need = lib.lmhead_loss_workspace_bytes(4, 256, 1000, 1)
    return Call(lib.lmhead_distill, xc=P, xs=P, gsa=P, wc=P, ws=P, gsw=P, tokens=P, teacher=P, dtype=0, K=8, tau=1.0,
                weight=P, T=4, D=256, N=1000, loss=P, lse=P, logq=P, dx=P, work=P, nbytes=need, s=None)


@pytest.mark.parametrize("which", [loss_call, distill_call])
def test_loss_refusals(lib, which):
    c = which(lib)
    names = "targets" if which is loss_call else "tokens"
    for bad in [dict(T=-1), dict(D=0), dict(D=16), dict(D=48), dict(N=0), dict(xc=None), dict(xs=None), dict(gsa=None),
                dict(wc=None), dict(ws=None), dict(gsw=None), {names: None}, dict(loss=None), dict(lse=None),
                dict(work=None), dict(nbytes=STATE), dict(work=off(128)), dict(xc=off(8)), dict(wc=off(8)),
                dict(xs=off(1)), dict(ws=off(2)), dict(gsa=off(2)), dict(gsw=off(2)), {names: off(2)},
                dict(weight=off(2)), dict(loss=off(2)), dict(lse=off(2)), dict(dx=off(8))]:
        assert c(**bad) == EINVAL, bad
    for bad in [dict(T=(1 << 18) + 1), dict(D=(1 << 22) + 32), dict(N=(1 << 30) + 1)]:
        assert c(**bad) == EUNSUPPORTED, bad
    # The gradient needs more workspace than the loss alone.
    assert lib.lmhead_loss_workspace_bytes(4, 256, 1000, 0) < c.args["nbytes"]
    assert c(nbytes=lib.lmhead_loss_workspace_bytes(4, 256, 1000, 0)) == EINVAL
    assert c(T=0, xc=None, xs=None, loss=None, lse=None, dx=None, work=None, nbytes=0, weight=None, **{names: None}) == 0


def test_distill_refusals(lib):
    c = distill_call(lib)
    for bad in [dict(dtype=2), dict(K=0), dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")), dict(tau=2.0 ** 21),
                dict(tau=2.0 ** -21), dict(tau=float("inf")), dict(teacher=None), dict(logq=None), dict(teacher=off(2)),
                dict(dtype=1, teacher=off(1)), dict(logq=off(2))]:
        assert c(**bad) == EINVAL, bad
    assert c(K=1025) == EUNSUPPORTED


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((4, 8))
    idx = torch.zeros((4, 2), dtype=torch.int32)
    q, w = rt.empty_nvfp4(4, 32, "cpu"), rt.empty_nvfp4(10, 32, "cpu")
    for f in (lambda: rt.select(x, 2), lambda: rt.select_backward(x, idx, torch.zeros((4, 2))),
              lambda: rt.lmhead_loss(q, w, torch.zeros(4, dtype=torch.int32), None),
              lambda: rt.lmhead_distill(q, w, idx, torch.zeros((4, 2)), None)):
        with pytest.raises(rt.RouterError):
            f()
