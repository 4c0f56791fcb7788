"""What a call leaves behind when its bounded waits run out: never another call's data.  In the
checked build a limit of 0 makes every wait give up at once; these tests run in that build
(test_gpu_checked_build.py runs the whole suite in it)."""
import contextlib
import ctypes

import pytest
import torch

from gqa_attention_flash_b200 import binding

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not binding.CHECKED, reason="checked build only")]

BF = torch.bfloat16


@contextlib.contextmanager
def no_waiting():
    f = binding.lib.attn_debug_wait_limit
    f.restype, f.argtypes = None, [ctypes.c_longlong]
    f(0)
    try:
        yield
    finally:
        f(-1)


def status():
    return binding.STATUS[binding.last_device_status()]


def rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()


@pytest.mark.parametrize("c", [(2, 8, 2, 1000, 64, 200, 5), (1, 32, 1, 1300, 128, 64, 4)], ids=str)
def test_backward_of_split_key_tiles(c):
    """One stream and two; the first call leaves large partials in the workspace that the second
    gets."""
    B, Hq, Hkv, S, D, window, sinks = c
    Q, K, V = rand(0, B, Hq, S, D), rand(1, B, Hkv, S, D), rand(2, B, Hkv, S, D)
    O, L, dQ = torch.empty_like(Q), torch.empty((B, Hq, S), device="cuda"), torch.empty_like(Q)
    binding.attn_fwd_sinks(O, Q, K, V, L, 0.1, window, sinks)
    dO = rand(3, B, Hq, S, D)

    def run(dO):
        dK, dV = torch.zeros_like(K), torch.zeros_like(V)
        binding.attn_bwd_sinks(dQ, dK, dV, dO, Q, K, V, O, L, 0.1, window, sinks)
        return dK, dV

    want = run(dO)
    large = run(dO * 256)
    assert status() == "ATTN_OK"
    assert all(float(x.float().abs().max()) > 100 for x in large)
    with no_waiting():
        given_up = run(dO)
        assert status() == "ATTN_ERR_TIMEOUT"
    for x in given_up:
        assert float(x.float().abs().max()) == 0
    again = run(dO)
    assert status() == "ATTN_OK"
    assert all(torch.equal(x, y) for x, y in zip(again, want))
