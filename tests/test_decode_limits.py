"""Decode at the limits of a launch's grid: more sequences than its z dimension holds, and more
KV heads than its y dimension does, which are refused."""
import ctypes

import pytest
import torch


def test_more_kv_heads_than_a_grid_holds_are_refused():
    from gqa_attention_flash_b200 import build
    build.build()
    from gqa_attention_flash_b200 import binding
    L, P = binding.lib, ctypes.c_void_p(16)
    # (O = None: a size that is let through answers NULL, and nothing is launched)
    for H, want in ((65535, 1), (65536, 2)):
        assert L.attn_decode(None, P, P, P, P, 4, None, 1, H, H, 64, 64) == want
        assert L.attn_decode_noalloc(None, P, P, P, P, 1, None, 1, H, H, 64, 64) == want
        assert L.attn_decode_sinks(None, P, P, P, P, 8, 2, 0, None, 1, H, H, 64, 64) == want
        assert L.attn_decode_paged(None, P, P, P, P, P, 4, None, 1, H, H, 9, 8, 4, 64) == want
        assert L.attn_decode_paged_sinks(None, P, P, P, P, P, 8, 2, 0, None, 1, H, H, 9, 8, 4, 64) == want


@pytest.mark.gpu
@pytest.mark.parametrize("n_splits", [1, 2, 9])
@pytest.mark.parametrize("window", [None, 5])
@pytest.mark.parametrize("paged", [False, True])
def test_more_sequences_than_a_grid_holds(paged, window, n_splits):
    """The same, bit for bit, as the two halves in calls of their own."""
    from gqa_attention_flash_b200 import binding
    B, Hq, Hkv, D, cap, cut = 65535 + 70, 2, 1, 64, 16, 40000
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    Q = rand(B, Hq, D)
    lens = torch.randint(0, cap + 1, (B,), generator=g, device="cuda").to(torch.int32)
    if paged:
        K, V = rand(64, 8, Hkv, D), rand(64, 8, Hkv, D)
        t = torch.randint(0, 64, (B, cap // 8), generator=g, device="cuda").to(torch.int32)
    else:
        K, V = rand(B, Hkv, cap, D), rand(B, Hkv, cap, D)

    def run(part):
        q, n = Q[part].contiguous(), lens[part].contiguous()
        O = torch.full_like(q, 7.0)
        args = (O, q, K, V, t[part].contiguous(), n) if paged else (O, q, K[part], V[part], n)
        name = "attn_decode" + ("_paged" if paged else "") + ("_sinks" if window else "")
        getattr(binding, name)(*args, *((window, 2) if window else ()), n_splits)
        assert binding.last_device_status() == 0
        return O

    whole, halves = run(slice(0, B)), [run(slice(0, cut)), run(slice(cut, B))]
    assert torch.equal(whole, torch.cat(halves))
    assert torch.equal((whole == 0).all(-1).all(-1), lens == 0)
