"""Integers that the C ABI's 32 bits do not hold are refused, not cut (2**32 sinks would be
none, a window of 2**32 + 5 one of 5).  No GPU needed: the check comes before the tensors'."""
import pytest
import torch


@pytest.fixture(scope="module")
def b():
    from gqa_attention_flash_b200 import build
    build.build()
    from gqa_attention_flash_b200 import binding
    return binding


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1, 10 ** 30])
def test_wide_integers(b, value):
    bf, i = torch.bfloat16, torch.int32
    z = torch.zeros
    Q, K, L = z(1, 2, 4, 64, dtype=bf), z(1, 1, 4, 64, dtype=bf), z(1, 2, 4)
    q, n, bt, pool = z(1, 2, 64, dtype=bf), z(1, dtype=i), z(1, 4, dtype=i), z(9, 8, 1, 64, dtype=bf)
    refs = z(9, dtype=i)
    calls = {
        "window": [lambda: b.attn_fwd(Q, Q, K, K, L, .1, True, value),
                   lambda: b.attn_fwd_flex(Q, Q, K, K, L, .1, True, value),
                   lambda: b.attn_fwd_sinks(Q, Q, K, K, L, .1, value, 4),
                   lambda: b.attn_bwd(Q, K, K, Q, Q, K, K, Q, L, .1, True, value),
                   lambda: b.attn_bwd_sinks(Q, K, K, Q, Q, K, K, Q, L, .1, value, 4),
                   lambda: b.attn_decode_sinks(q, q, K, K, n, value, 4),
                   lambda: b.attn_decode_paged_sinks(q, q, pool, pool, bt, n, value, 4),
                   lambda: b.block_mask_document(4, 4, n.repeat(4), n.repeat(4), True, value)],
        "sinks": [lambda: b.attn_fwd_sinks(Q, Q, K, K, L, .1, 8, value),
                  lambda: b.attn_bwd_sinks(Q, K, K, Q, Q, K, K, Q, L, .1, 8, value),
                  lambda: b.attn_decode_sinks(q, q, K, K, n, 8, value),
                  lambda: b.attn_decode_paged_sinks(q, q, pool, pool, bt, n, 8, value)],
        "input_pos": [lambda: b.attn_fwd(Q, Q, K, K, L, .1, input_pos=value),
                      lambda: b.attn_fwd_sinks(Q, Q, K, K, L, .1, 8, 2, value),
                      lambda: b.attn_bwd_sinks(Q, K, K, Q, Q, K, K, Q, L, .1, 8, 2, value)],
        "n_splits": [lambda: b.attn_decode(q, q, K, K, n, value),
                     lambda: b.attn_decode_noalloc(q, q, K, K, n, value),
                     lambda: b.attn_decode_paged(q, q, pool, pool, bt, n, value),
                     lambda: b.attn_decode_sinks(q, q, K, K, n, 8, 2, value),
                     lambda: b.attn_decode_paged_sinks(q, q, pool, pool, bt, n, 8, 2, value)],
        "block_size": [lambda: b.cache_fork(bt, refs, n, n, n, n, n, value),
                       lambda: b.cache_extend(bt, refs, n, n, value)],
        "limit_us": [lambda: b.check_bounded_wait(value)],
    }
    for name, fs in calls.items():
        for f in fs:
            with pytest.raises(ValueError, match=f"{name} = .* does not fit in 32 bits"):
                f()
