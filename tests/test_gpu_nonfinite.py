"""A NaN in what a query really sees reaches that query's output, whatever the way the call is
split, and no other row of it."""
import pytest
import torch

from gqa_attention_flash_b200 import binding

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
NAN = float("nan")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()


def every(x):
    """All NaN; a plain number, so that a failure prints no tensors."""
    return int(x.isnan().sum()) == x.numel()


@pytest.mark.parametrize("n_splits", [1, 2, 7, 8, 9, 16, 40])
@pytest.mark.parametrize("window", [600, None])
@pytest.mark.parametrize("paged", [False, True])
def test_decode(n_splits, window, paged):
    B, Hq, Hkv, D, S, block = 2, 8, 2, 128, 1024, 16
    Q, lens = rand(0, B, Hq, D), i32([1000, 700])

    def run(Q, K, V):
        O = torch.empty_like(Q)
        if paged:
            cut = lambda x: x.transpose(1, 2).reshape(B * S // block, block, Hkv, D).contiguous()  # noqa: E731
            t = torch.arange(B * S // block, dtype=torch.int32, device="cuda").view(B, -1)
            if window:
                binding.attn_decode_paged_sinks(O, Q, cut(K), cut(V), t, lens, window, 4, n_splits)
            else:
                binding.attn_decode_paged(O, Q, cut(K), cut(V), t, lens, n_splits)
        elif window:
            binding.attn_decode_sinks(O, Q, K, V, lens, window, 4, n_splits)
        else:
            binding.attn_decode(O, Q, K, V, lens, n_splits)
        assert binding.last_device_status() == 0
        return O

    K, V = rand(1, B, Hkv, S, D), rand(2, B, Hkv, S, D)
    clean = run(Q, K, V)
    assert torch.isfinite(clean.float()).all()
    q = Q.clone()
    q[0, 5, 17] = NAN                    # one head's query
    got = run(q, K, V)
    assert every(got[0, 5])
    got[0, 5] = clean[0, 5]
    assert torch.equal(got, clean)
    for j in (2, 650):                   # a sink; a key of the window
        k = K.clone()
        k[0, 1, j, 9] = NAN
        got = run(Q, k, V)
        assert every(got[0, 4:])  # the heads of that KV head
        got[0, 4:] = clean[0, 4:]
        assert torch.equal(got, clean)
    k = K.clone()
    k[0, 1, 300 if window else 1000:400 if window else S] = NAN  # not seen: between, or past the length
    assert torch.equal(run(Q, k, V), clean)
