"""CPU checks of the expert layer's and the logits' entry points: sizes, refusals and empty calls. No call here
reaches a kernel launch."""

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


def test_workspace_sizes(lib):
    assert lib.grouped_workspace_bytes(1, 8, 256, 7168, 2048) >= STATE + 8 * 7168 * 4
    assert rt.grouped_workspace_bytes(0, 1, 1, 32, 32) >= STATE
    for bad in [(-1, 8, 256, 7168, 2048), (1, 0, 256, 7168, 2048), (1, 33, 256, 7168, 2048), (1, 8, 0, 7168, 2048),
                (1, 8, 513, 7168, 2048), (1, 8, 256, 0, 2048), (1, 8, 256, 7168, 0), (1 << 31, 1, 1, 32, 32)]:
        assert lib.grouped_workspace_bytes(*bad) == 0, bad
        with pytest.raises(rt.RouterError):
            rt.grouped_workspace_bytes(*bad)
    assert lib.lmhead_penalize_workspace_bytes(0, 1) >= STATE
    assert lib.lmhead_penalize_workspace_bytes(4, 129280) >= lib.lmhead_penalize_workspace_bytes(1, 129280)
    for bad in [(-1, 10), (1, 0), (1, (1 << 30) + 1)]:
        assert lib.lmhead_penalize_workspace_bytes(*bad) == 0, bad


def test_workspace_sizes_are_the_calls_sizes(lib):
    """Zero for just the sizes that both products refuse."""
    swiglu = Call(lib.grouped_swiglu, xc=P, xs=P, gsa=None, wc=P, ws=P, gsw=P, bias=None, offsets=P, rows=P, T=4, k=2,
                  G=8, F=64, D=256, out=P, s=None)
    combine = Call(lib.grouped_combine, hc=P, hs=P, gsh=None, wc=P, ws=P, gsw=P, bias=None, offsets=P, pos=P, w=P,
                   residual=None, T=4, k=2, G=8, D=64, F=256, out=P, work=P, nbytes=1 << 20, s=None)
    taken = []
    for D, F in [(17, 32), (32, 33), (8, 32), (32, 8), (40, 40), (48, 32), (32, 48), (48, 48), (32, 1360), (16, 32),
                 (32, 16), (16, 16), (1 << 16, 1 << 17), (1 << 17, 1 << 16), (1 << 22, 512), (512, 1 << 22),
                 (32, (1 << 22) + 32), ((1 << 22) + 32, 32), (1 << 15, 1 << 16), (2048, 7168)]:
        # A missing scale is refused as EINVAL, after the sizes; sizes that the layouts allow but that are too large
        # or no multiple of 32 are unsupported.
        a, b = swiglu(D=D, F=F), combine(D=D, F=F)
        ok = [a == EINVAL and F >= 16 and F % 16 == 0 and D >= 16 and D % 16 == 0,
              b == EINVAL and D >= 16 and D % 16 == 0 and F >= 16 and F % 16 == 0]
        assert (lib.grouped_workspace_bytes(4, 2, 8, D, F) > 0) == any(ok), (D, F, a, b)
        taken.append(any(ok))
    assert any(taken) and not all(taken)


def test_plan_refusals(lib):
    c = Call(lib.grouped_plan, idx=P, T=4, k=2, first=0, G=8, offsets=P, rows=P, pos=P, ws=P, nbytes=1 << 20, s=None)
    for bad in [dict(T=-1), dict(k=0), dict(G=0), dict(first=-1), dict(idx=None), dict(offsets=None), dict(rows=None),
                dict(pos=None), dict(idx=off(2)), dict(offsets=off(1)), dict(rows=off(2)), dict(pos=off(2)),
                dict(T=4096, ws=None), dict(T=4096, nbytes=4096), dict(T=4096, ws=off(64))]:
        assert c(**bad) == EINVAL, bad
    for bad in [dict(k=33), dict(G=513), dict(T=1 << 30)]:
        assert c(**bad) == EUNSUPPORTED, bad


def test_swiglu_refusals(lib):
    c = Call(lib.grouped_swiglu, xc=P, xs=P, gsa=P, wc=P, ws=P, gsw=P, bias=None, offsets=P, rows=P, T=4, k=2, G=8,
             F=64, D=256, out=P, s=None)
    for bad in [dict(T=-1), dict(k=0), dict(G=0), dict(F=0), dict(F=24), dict(D=0), dict(D=40), dict(xc=None),
                dict(xs=None), dict(gsa=None), dict(wc=None), dict(ws=None), dict(gsw=None), dict(offsets=None),
                dict(rows=None), dict(out=None), dict(xc=off(8)), dict(wc=off(8)), dict(xs=off(1)), dict(ws=off(2)),
                dict(gsa=off(2)), dict(gsw=off(2)), dict(bias=off(2)), dict(offsets=off(2)), dict(rows=off(2)),
                dict(out=off(8))]:
        assert c(**bad) == EINVAL, bad
    for bad in [dict(D=48), dict(k=33), dict(G=513), dict(D=(1 << 22) + 32), dict(F=1 << 22), dict(T=1 << 29, k=4),
                dict(T=1 << 24, k=1), dict(F=1 << 16, D=1 << 16)]:
        assert c(**bad) == EUNSUPPORTED, bad
    assert c(T=0) == 0
    assert c(T=0, xc=None, xs=None, rows=None, out=None) == 0


def test_combine_refusals(lib):
    c = Call(lib.grouped_combine, hc=P, hs=P, gsh=P, wc=P, ws=P, gsw=P, bias=None, offsets=P, pos=P, w=P,
             residual=None, T=4, k=2, G=8, D=64, F=256, out=P, work=P, nbytes=1 << 20, s=None)
    for bad in [dict(T=-1), dict(k=0), dict(G=0), dict(D=0), dict(D=24), dict(F=0), dict(F=40), dict(hc=None),
                dict(hs=None), dict(gsh=None), dict(wc=None), dict(ws=None), dict(gsw=None), dict(offsets=None),
                dict(pos=None), dict(w=None), dict(out=None), dict(work=None), dict(nbytes=STATE), dict(work=off(128)),
                dict(hc=off(8)), dict(wc=off(8)), dict(hs=off(1)), dict(ws=off(2)), dict(gsh=off(2)), dict(gsw=off(2)),
                dict(bias=off(2)), dict(offsets=off(2)), dict(pos=off(2)), dict(w=off(2)), dict(residual=off(8)),
                dict(out=off(8))]:
        assert c(**bad) == EINVAL, bad
    for bad in [dict(F=48), dict(k=33), dict(G=513), dict(F=(1 << 22) + 32), dict(D=(1 << 22) + 16),
                dict(T=1 << 29, k=4), dict(D=1 << 16, F=1 << 17)]:
        assert c(**bad) == EUNSUPPORTED, bad
    assert c(T=0) == 0
    assert c(T=0, hc=None, hs=None, pos=None, w=None, out=None, work=None, nbytes=0) == 0


def test_penalize_refusals(lib):
    c = Call(lib.lmhead_penalize, logits=P, dtype=0, T=2, N=5000, ld=5000, history=P, L=16, ldh=16, lengths=P,
             prompt=P, rep=P, freq=P, pres=P, bstart=P, btok=P, bval=P, nbias=4, mask=P, ldm=157, out=off(1 << 20), ldo=5000,
             idx=P, logit=P, work=P, nbytes=1 << 20, s=None)
    for bad in [dict(dtype=2), dict(T=-1), dict(N=0), dict(ld=4999), dict(ldo=4999), dict(out=P, ldo=5001), dict(logits=None), dict(out=None), dict(idx=None),
                dict(logit=None), dict(L=-1), dict(ldh=15), dict(history=None), dict(btok=None), dict(bval=None),
                dict(nbias=-1), dict(ldm=156), dict(work=None), dict(nbytes=STATE), dict(work=off(64)),
                dict(logits=off(2)), dict(out=off(2)), dict(dtype=1, logits=off(1)), dict(history=off(2)),
                dict(lengths=off(2)), dict(prompt=off(2)), dict(rep=off(2)), dict(freq=off(2)), dict(pres=off(2)),
                dict(bstart=off(2)), dict(btok=off(2)), dict(bval=off(2)), dict(mask=off(2)), dict(idx=off(2)),
                dict(logit=off(2))]:
        assert c(**bad) == EINVAL, bad
    assert c(T=0) == 0


def test_binding_refuses_cpu_tensors():
    idx = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(rt.RouterError):
        rt.grouped_plan(idx, 8, None)
    with pytest.raises(rt.RouterError):
        rt.lmhead_penalize(torch.zeros((2, 8)), None)
    x = rt.empty_nvfp4(4, 32, "cpu")
    w = rt.GroupedWeights(torch.zeros((2, 32, 16), dtype=torch.uint8), torch.zeros((2, 32, 2), dtype=torch.uint8),
                          torch.zeros(2))
    plan = rt.empty_plan(4, 2, 2, "cpu")
    with pytest.raises(rt.RouterError):
        rt.grouped_swiglu(x, w, plan)
    with pytest.raises(rt.RouterError):
        rt.grouped_combine(x, w, plan, torch.zeros((4, 2)), None)
