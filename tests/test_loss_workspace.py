"""CPU checks of the workspace size of the lm_head's losses over their row counts. No call here reaches a launch."""

import os

import pytest

from nvfp4_block_scaled_06_amd import router as rt


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(rt.LIB_PATH):
        from nvfp4_block_scaled_06_amd import build

        build.build()
    return rt.load_library()


@pytest.mark.parametrize("D,N", [(7168, 129280), (2080, 32003), (1056, 50021), (32, 1), (96, 13000), (512, 4000), (4096, 200000)])
def test_size_never_falls_with_more_rows(lib, D, N):
    """A workspace made for the most rows takes every call with fewer; one made for the gradient takes calls without."""
    f = lib.lmhead_loss_workspace_bytes
    steps = list(range(0, 300)) + list(range(300, 4200, 31)) + [2048, 2049, 2073, 5000, 8192, 8193, 16384, 40000, 65536, 65537, 1 << 17, 1 << 18]
    steps.sort()
    for grad in (0, 1):
        sizes = [f(T, D, N, grad) for T in steps]
        falls = [(T, a, b) for T, a, b in zip(steps[1:], sizes, sizes[1:]) if b < a]
        assert not falls, (grad, len(falls), falls[:3])
    assert all(f(T, D, N, 1) >= f(T, D, N, 0) for T in steps)
