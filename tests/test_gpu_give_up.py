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


@pytest.mark.parametrize("n_splits", [1, 2, 5, 8, 9, 24])
@pytest.mark.parametrize("window", [2000, None])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_decode(D, paged, window, n_splits):
    """No slice has a result: the output is 0, whatever lands in shared memory meanwhile."""
    B, Hq, Hkv, S, block = 3, 16, 2, 2048, 16
    Q, K, V = rand(0, B, Hq, D), rand(1, B, Hkv, S, D), rand(2, B, Hkv, S, D)
    lens = torch.tensor([2048, 1500, 1999], dtype=torch.int32, device="cuda")
    if paged:
        K, V = (x.transpose(1, 2).reshape(B * S // block, block, Hkv, D).contiguous() for x in (K, V))
        t = torch.arange(B * S // block, dtype=torch.int32, device="cuda").view(B, -1)
    name = "attn_decode" + ("_paged" if paged else "") + ("_sinks" if window else "")

    def run():
        O = torch.full_like(Q, 7.0)
        getattr(binding, name)(O, Q, K, V, *((t,) if paged else ()), lens, *((window, 4) if window else ()),
                               n_splits)
        return O

    want = run()
    assert status() == "ATTN_OK"
    for _ in range(5):
        with no_waiting():
            got = run()
            assert status() == "ATTN_ERR_TIMEOUT"
        assert int((got != 0).sum()) == 0
    assert torch.equal(run(), want)
    assert status() == "ATTN_OK"


@pytest.mark.parametrize("B,T,ctx", [(1, 8, 3000), (1, 70, 3000), (3, 8, 700)])
def test_tree(B, T, ctx):
    """Segments that several CTAs share come out 0; a CTA's own are not written."""
    Hq, Hkv, D, block = 8, 2, 128, 16
    n = (ctx + T + block - 1) // block
    K, V = rand(1, B * n, block, Hkv, D), rand(2, B * n, block, Hkv, D)
    t = torch.arange(B * n, dtype=torch.int32, device="cuda").view(B, n)
    Q, parents = rand(0, B, Hq, T, D), torch.arange(-1, T - 1, dtype=torch.int32, device="cuda").repeat(B, 1)
    ctx = torch.full((B,), ctx, dtype=torch.int32, device="cuda")

    def run():
        O = torch.full_like(Q, 7.0)
        binding.attn_tree_paged(O, Q, K, V, t, ctx, parents)
        return O

    want = run()
    assert status() == "ATTN_OK"
    with no_waiting():
        got = run()
        assert status() == "ATTN_ERR_TIMEOUT"
    assert int(((got != 0) & (got != 7)).sum()) == 0
    assert torch.equal(run(), want)
    assert status() == "ATTN_OK"
