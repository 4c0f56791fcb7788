"""Refusals of the windowed-with-sinks, tree and cache operators, before any launch: the C
entry points' status codes and the binding's checks.  No GPU needed."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def binding():
    from gqa_attention_flash_b200 import build
    build.build()
    from gqa_attention_flash_b200 import binding as b
    return b


P = ctypes.c_void_p(16)     # non-NULL, 16-byte aligned; never dereferenced on these paths
ODD = ctypes.c_void_p(18)
OK, NULL, INVALID, UNSUPPORTED = 0, 1, 2, 3


def caller(fn, names, **defaults):
    def call(**kw):
        a = dict(defaults, **kw)
        return fn(*[a[n] for n in names.split()])
    return call


def test_forward_and_backward(binding):
    L = binding.lib
    common = dict(B=1, Hq=2, Hkv=1, Sq=4, Sk=4, D=128, scale=0.1, window=8, sinks=2, pos=0, kl=None,
                  ql=None, stream=None)
    fwd = caller(L.attn_fwd_sinks, "O Q K V L B Hq Hkv Sq Sk D scale window sinks pos kl ql stream",
                 O=P, Q=P, K=P, V=P, L=P, **common)
    bwd = caller(L.attn_bwd_sinks, "dQ dK dV dO Q K V O L B Hq Hkv Sq Sk D scale window sinks pos kl "
                 "ql stream", dQ=P, dK=P, dV=P, dO=P, Q=P, K=P, V=P, O=P, L=P, **common)
    for f in (fwd, bwd):
        assert f(window=0) == INVALID
        assert f(window=-3) == INVALID
        assert f(sinks=-1) == INVALID
        assert f(Hq=3, Hkv=2) == INVALID
        assert f(scale=0.0) == INVALID
        assert f(pos=-1) == INVALID
        assert f(D=96) == UNSUPPORTED
        assert f(K=None) == NULL
        assert f(Q=ODD) == INVALID
        assert f(B=0) == OK
    assert fwd(Sq=0) == OK
    assert bwd(L=None) == NULL and bwd(dV=None) == NULL


def test_decode(binding):
    L = binding.lib
    con = caller(L.attn_decode_sinks, "O Q K V lens window sinks n stream B Hq Hkv cap D", O=P, Q=P,
                 K=P, V=P, lens=P, window=8, sinks=2, n=0, stream=None, B=1, Hq=8, Hkv=2, cap=64, D=128)
    pag = caller(L.attn_decode_paged_sinks, "O Q K V bt lens window sinks n stream B Hq Hkv nb bs mb D",
                 O=P, Q=P, K=P, V=P, bt=P, lens=P, window=8, sinks=2, n=0, stream=None, B=1, Hq=8,
                 Hkv=2, nb=10, bs=16, mb=4, D=128)
    for f in (con, pag):
        assert f(window=0) == INVALID and f(sinks=-1) == INVALID
        assert f(n=65) == INVALID and f(n=-1) == INVALID
        assert f(Hq=9) == INVALID and f(Hq=34, Hkv=2) == INVALID
        assert f(D=32) == UNSUPPORTED
        assert f(O=None) == NULL and f(lens=None) == NULL
        assert f(V=ODD) == INVALID
        assert f(B=-1) == INVALID and f(B=0) == OK
    assert con(cap=-1) == INVALID
    assert pag(bs=12) == INVALID and pag(bs=0) == INVALID and pag(nb=0) == INVALID
    assert pag(bt=None) == NULL


def test_tree(binding):
    f = caller(binding.lib.attn_tree_paged, "O Q K V bt ctx par dl stream B Hq Hkv T nb bs mb D", O=P,
               Q=P, K=P, V=P, bt=P, ctx=P, par=P, dl=None, stream=None, B=1, Hq=8, Hkv=2, T=4, nb=10,
               bs=16, mb=4, D=128)
    assert f(T=257) == INVALID and f(T=-1) == INVALID
    assert f(Hq=9) == INVALID and f(Hq=34, Hkv=2) == INVALID
    assert f(bs=4) == INVALID and f(bs=24) == INVALID and f(mb=0) == INVALID and f(nb=0) == INVALID
    assert f(nb=2 ** 30, bs=16) == INVALID and f(mb=2 ** 30, bs=16) == INVALID
    assert f(D=80) == UNSUPPORTED
    for name in ("O", "Q", "K", "V", "bt", "ctx", "par"):
        assert f(**{name: None}) == NULL, name
        assert f(**{name: ODD}) == INVALID, name
    assert f(dl=ODD) == INVALID
    assert f(B=0) == OK and f(T=0) == OK


def test_cache_rows(binding):
    L = binding.lib
    app = caller(L.attn_cache_append, "K V Kn Vn bt start n stream B Hkv T nb bs mb D", K=P, V=P, Kn=P,
                 Vn=P, bt=P, start=P, n=None, stream=None, B=1, Hkv=2, T=4, nb=10, bs=16, mb=4, D=128)
    com = caller(L.attn_cache_compact, "K V bt start keep n stream B Hkv T nb bs mb D", K=P, V=P, bt=P,
                 start=P, keep=P, n=None, stream=None, B=1, Hkv=2, T=4, nb=10, bs=16, mb=4, D=128)
    for f, names in ((app, "K V Kn Vn bt start"), (com, "K V bt start keep")):
        assert f(B=-1) == INVALID and f(Hkv=0) == INVALID and f(T=-1) == INVALID
        assert f(bs=10) == INVALID and f(nb=0) == INVALID and f(mb=0) == INVALID
        assert f(D=100) == UNSUPPORTED
        for name in names.split():
            assert f(**{name: None}) == NULL, name
            assert f(**{name: ODD}) == INVALID, name
        assert f(n=ODD) == INVALID
        assert f(B=0) == OK and f(T=0) == OK
    cop = caller(L.attn_cache_copy_blocks, "K V src dst stream N nb bs Hkv D", K=P, V=P, src=P, dst=P,
                 stream=None, N=2, nb=10, bs=16, Hkv=2, D=128)
    assert cop(N=-1) == INVALID and cop(N=65537) == INVALID and cop(bs=3) == INVALID
    assert cop(Hkv=0) == INVALID and cop(D=1) == UNSUPPORTED
    for name in ("K", "V", "src", "dst"):
        assert cop(**{name: None}) == NULL and cop(**{name: ODD}) == INVALID
    assert cop(N=0) == OK


def test_cache_tables(binding):
    L = binding.lib
    fork = caller(L.attn_cache_fork, "bt rc lens par chi src dst stream N R nb bs mb", bt=P, rc=P,
                  lens=P, par=P, chi=P, src=P, dst=P, stream=None, N=2, R=4, nb=10, bs=16, mb=4)
    ext = caller(L.attn_cache_extend, "bt rc lens to stream N nb bs mb", bt=P, rc=P, lens=P, to=P,
                 stream=None, N=4, nb=10, bs=16, mb=4)
    free = caller(L.attn_cache_free, "bt rc rows first last stream N R nb mb", bt=P, rc=P, rows=P,
                  first=P, last=P, stream=None, N=2, R=4, nb=10, mb=4)
    for f, names in ((fork, "bt rc lens par chi src dst"), (ext, "bt rc lens to"),
                     (free, "bt rc rows first last")):
        assert f(N=-1) == INVALID and f(nb=0) == INVALID and f(mb=0) == INVALID
        for name in names.split():
            assert f(**{name: None}) == NULL, name
            assert f(**{name: ODD}) == INVALID, name
        assert f(N=0) == OK
    assert fork(N=65537) == INVALID and fork(R=-1) == INVALID and free(R=-1) == INVALID
    assert fork(bs=9) == INVALID and ext(bs=9) == INVALID
    assert fork(rc=ctypes.c_void_p(24)) == INVALID  # counts are read 16 bytes at a time
    assert ext(rc=ctypes.c_void_p(24)) == INVALID


def test_caches_past_2_30_positions_are_refused(binding):
    # (O = None: a size that is let through answers NULL, and nothing is launched)
    L = binding.lib
    con = caller(L.attn_decode_sinks, "O Q K V lens window sinks n stream B Hq Hkv cap D", O=None, Q=P,
                 K=P, V=P, lens=P, window=8, sinks=2, n=0, stream=None, B=1, Hq=8, Hkv=2, D=128)
    pag = caller(L.attn_decode_paged_sinks, "O Q K V bt lens window sinks n stream B Hq Hkv nb bs mb D",
                 O=None, Q=P, K=P, V=P, bt=P, lens=P, window=8, sinks=2, n=0, stream=None, B=1, Hq=8,
                 Hkv=2, nb=10, bs=16, D=128)
    tree = caller(L.attn_tree_paged, "O Q K V bt ctx par dl stream B Hq Hkv T nb bs mb D", O=None,
                  Q=P, K=P, V=P, bt=P, ctx=P, par=P, dl=None, stream=None, B=1, Hq=8, Hkv=2, T=4,
                  nb=10, bs=16, D=128)
    assert con(cap=2 ** 30) == NULL and con(cap=2 ** 30 + 1) == INVALID
    for f in (pag, tree):
        assert f(mb=2 ** 26) == NULL
        assert f(mb=2 ** 26 + 1) == INVALID and f(mb=2 ** 27 - 1) == INVALID


def test_extend_refuses_tables_whose_entries_overflow_32_bits(binding):
    # (lens = None: a size that is let through answers NULL, and nothing is launched)
    ext = caller(binding.lib.attn_cache_extend, "bt rc lens to stream N nb bs mb", bt=P, rc=P,
                 lens=None, to=P, stream=None, nb=10, bs=8)
    assert ext(N=1 << 10, mb=1 << 21) == INVALID
    assert ext(N=(1 << 31) - 1, mb=(1 << 28) - 1) == INVALID
    assert ext(N=(1 << 10) - 1, mb=1 << 21) == NULL


def test_binding_refuses_tensors_that_do_not_fit(binding):
    bf, i = torch.bfloat16, torch.int32
    z = torch.zeros
    pool = z(10, 16, 2, 128, dtype=bf)
    bt, n = z(3, 4, dtype=i), z(3, dtype=i)
    Q, q = z(3, 8, 5, 128, dtype=bf), z(3, 8, 128, dtype=bf)
    K = z(3, 2, 5, 128, dtype=bf)
    lse = z(3, 8, 5)
    b = binding
    bad = [
        (ValueError, "V has shape", lambda: b.attn_fwd_sinks(Q, Q, K, K[:, :, :4].contiguous(), lse, .1, 2, 1)),
        (TypeError, "Q must be", lambda: b.attn_fwd_sinks(Q, Q.half(), K, K, lse, .1, 2, 1)),
        (ValueError, "must be a CUDA tensor", lambda: b.attn_fwd_sinks(Q, Q, K, K, lse, .1, 2, 1)),
        (ValueError, "dK has shape", lambda: b.attn_bwd_sinks(Q, Q, K, Q, Q, K, K, Q, lse, .1, 2, 1)),
        (ValueError, "LSE", lambda: b.attn_bwd_sinks(Q, K, K, Q, Q, K, K, Q, None, .1, 2, 1)),
        (ValueError, "O has shape", lambda: b.attn_decode_sinks(Q, q, K, K, n, 2, 1)),
        (TypeError, "lengths must be", lambda: b.attn_decode_sinks(q, q, K, K, n.long(), 2, 1)),
        (ValueError, "V_cache has shape", lambda: b.attn_decode_paged_sinks(q, q, pool, pool[1:], bt, n, 2, 1)),
        (ValueError, "block_tables has shape", lambda: b.attn_decode_paged_sinks(q, q, pool, pool, bt[1:], n, 2, 1)),
        (ValueError, "must be a CUDA tensor", lambda: b.attn_decode_paged_sinks(q, q, pool, pool, bt, n, 2, 1)),
        (ValueError, "parents has shape", lambda: b.attn_tree_paged(Q, Q, pool, pool, bt, n, z(3, 4, dtype=i))),
        (TypeError, "parents must be", lambda: b.attn_tree_paged(Q, Q, pool, pool, bt, n, z(3, 5))),
        (ValueError, "Q must be contiguous", lambda: b.attn_tree_paged(
            Q, z(3, 5, 8, 128, dtype=bf).transpose(1, 2), pool, pool, bt, n, z(3, 5, dtype=i))),
        (ValueError, "draft_lens has shape", lambda: b.attn_tree_paged(Q, Q, pool, pool, bt, n, z(3, 5, dtype=i), n[1:])),
        (ValueError, "KV heads", lambda: b.cache_append(pool, pool, z(3, 4, 5, 128, dtype=bf), z(3, 4, 5, 128, dtype=bf), bt, n)),
        (ValueError, "V_new has shape", lambda: b.cache_append(pool, pool, K, K[:, :, 1:], bt, n)),
        (TypeError, "start must be", lambda: b.cache_append(pool, pool, K, K, bt, n.float())),
        (ValueError, "base has shape", lambda: b.cache_compact(pool, pool, bt, n[1:], z(3, 4, dtype=i))),
        (TypeError, "keep must be", lambda: b.cache_compact(pool, pool, bt, n, z(3, 4))),
        (TypeError, "K_cache must be", lambda: b.cache_compact(None, pool, bt, n, z(3, 4, dtype=i))),
        (ValueError, "dst has shape", lambda: b.cache_copy_blocks(pool, pool, n, n[1:])),
        (ValueError, "seq_lens has shape", lambda: b.cache_fork(bt, z(10, dtype=i), n[1:], n, n, n, n, 16)),
        (ValueError, "children has shape", lambda: b.cache_fork(bt, z(10, dtype=i), n, n, n[1:], n, n, 16)),
        (ValueError, "to_lens has shape", lambda: b.cache_extend(bt, z(10, dtype=i), n, n[1:], 16)),
        (TypeError, "ref_counts must be", lambda: b.cache_free(bt, z(10), n, n, n)),
        (ValueError, "must be a CUDA tensor", lambda: b.cache_free(bt, z(10, dtype=i), n, n, n)),
        (ValueError, "must be contiguous", lambda: b.cache_free(z(4, 3, dtype=i).t(), z(10, dtype=i), n, n, n)),
    ]
    for err, match, f in bad:
        with pytest.raises(err, match=match):
            f()
