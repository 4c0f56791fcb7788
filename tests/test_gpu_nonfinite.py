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


@pytest.mark.parametrize("kind", ["plain", "sinks", "document", "blocks"])
def test_forward(kind):
    B, Hq, Hkv, S, D = 2, 4, 2, 700, 128
    Q, K, V = rand(0, B, Hq, S, D), rand(1, B, Hkv, S, D), rand(2, B, Hkv, S, D)

    def run(Q, K):
        O, L = torch.empty_like(Q), torch.empty((B, Hq, S), device="cuda")
        if kind == "plain":
            binding.attn_fwd(O, Q, K, V, L, 0.1, causal=True)
        elif kind == "sinks":
            binding.attn_fwd_sinks(O, Q, K, V, L, 0.1, 200, 4)
        elif kind == "document":
            ids = (torch.arange(S, device="cuda") // 300).to(torch.int32)
            binding.attn_fwd_flex(O, Q, K, V, L, 0.1, causal=True, doc_q=ids, doc_kv=ids)
        else:
            mask = torch.full(binding.block_mask_shape(S, S), 2, dtype=torch.uint8, device="cuda")
            mask[:5, 6:] = 0             # rows below 320 see keys below 384
            binding.attn_fwd_flex(O, Q, K, V, L, 0.1, block_mask=mask)
        assert binding.last_device_status() == 0
        return O, L

    clean = run(Q, K)
    assert all(torch.isfinite(x.float()).all() for x in clean)
    q = Q.clone()
    q[1, 2, 555, 3] = NAN                # one row
    got = run(q, K)
    for x, y in zip(got, clean):
        assert every(x[1, 2, 555])
        x[1, 2, 555] = y[1, 2, 555]
        assert torch.equal(x, y)
    k = K.clone()
    k[0, 0, 690] = NAN                   # a key that the last rows see
    got = run(Q, k)
    assert every(got[0][0, :2, 695:]) and every(got[1][0, :2, 695:])
    for x, y in zip(got, clean):
        assert torch.equal(x[:, 2:], y[:, 2:]) and torch.equal(x[:, :, :300], y[:, :, :300])


@pytest.mark.parametrize("B,Hq,T,ctx", [(1, 8, 8, 1000),      # a segment in many CTAs
                                        (64, 8, 4, 40),       # whole segments
                                        (1, 8, 70, 900), (40, 8, 70, 100)])  # two row tiles
def test_tree(B, Hq, T, ctx):
    Hkv, D, block = 2, 128, 16
    n = (ctx + T + block - 1) // block
    K, V = rand(1, B * n, block, Hkv, D), rand(2, B * n, block, Hkv, D)
    t = torch.arange(B * n, dtype=torch.int32, device="cuda").view(B, n)
    Q, parents = rand(0, B, Hq, T, D), torch.arange(-1, T - 1, dtype=torch.int32, device="cuda").repeat(B, 1)

    def run(Q, K):
        O = torch.empty_like(Q)
        binding.attn_tree_paged(O, Q, K, V, t, i32([ctx] * B), parents)
        assert binding.last_device_status() == 0
        return O

    clean = run(Q, K)
    assert torch.isfinite(clean.float()).all()
    for row in (0, T - 1):
        q = Q.clone()
        q[0, 5, row, 100] = NAN
        got = run(q, K)
        assert every(got[0, 5, row])
        got[0, 5, row] = clean[0, 5, row]
        assert torch.equal(got, clean)
    k = K.clone()
    k[1, 3, 0, 7] = NAN                  # a key of the first sequence's context
    got = run(Q, k)
    assert every(got[0, :4])
    got[0, :4] = clean[0, :4]
    assert torch.equal(got, clean)
