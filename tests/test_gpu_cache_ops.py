"""The paged cache's operators (append, compact, copy_blocks, fork, extend, free) against
plain Python on the same tables; every result is exact."""
import pytest
import torch

from gqa_attention_flash_b200 import binding

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
BOUNDS = "ATTN_ERR_DEVICE_BOUNDS"


def status():
    return binding.STATUS[binding.last_device_status()]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pools(seed, n, block, Hkv, D):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(n, block, Hkv, D, generator=g).to(BF).cuda() for _ in range(2)]


def table(seed, R, width, n, lens, block):
    """Distinct pages for each row's length, in a random order."""
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(seed)).tolist()
    t = [[-1] * width for _ in range(R)]
    for r, ln in enumerate(lens):
        for k in range((ln + block - 1) // block):
            t[r][k] = perm.pop()
    return t


# ---------------------------------------------------------------------------------
# rows
# ---------------------------------------------------------------------------------
ROWS = [
    # B, Hkv, T, D, block, start, n
    (1, 1, 1, 64, 8, [0], None),
    (1, 1, 1, 128, 16, [31], None),
    (3, 2, 5, 64, 8, [0, 7, 8], [5, 1, 0]),
    (2, 8, 33, 128, 16, [13, 100], [33, 20]),
    (2, 3, 300, 64, 64, [1, 63], [300, 299]),
    (4, 1, 700, 128, 256, [0, 5, 255, 256], [700, 1, 400, 699]),
]


@pytest.mark.parametrize("c", ROWS, ids=[str(c) for c in ROWS])
def test_append(c):
    B, Hkv, T, D, block, start, n = c
    lens = [s + (n[b] if n else T) for b, s in enumerate(start)]
    width = max(lens) // block + 2
    N = B * width
    t = table(1, B, width, N, lens, block)
    K, V = pools(2, N, block, Hkv, D)
    g = torch.Generator().manual_seed(3)
    Kn, Vn = (torch.randn(B, Hkv, T, D, generator=g).to(BF).cuda() for _ in range(2))
    wk, wv = K.clone(), V.clone()
    for b in range(B):
        for i in range(n[b] if n else T):
            at = t[b][(start[b] + i) // block], (start[b] + i) % block
            wk[at], wv[at] = Kn[b, :, i], Vn[b, :, i]
    binding.cache_append(K, V, Kn, Vn, i32(t), i32(start), i32(n) if n else None)
    assert status() == "ATTN_OK"
    assert torch.equal(K, wk) and torch.equal(V, wv)


def test_append_out_of_range_rows_are_flagged_and_not_written():
    block, width, N = 8, 3, 9
    K, V = pools(4, N, block, 2, 64)
    Kn, Vn = (torch.ones(1, 2, 4, 64, dtype=BF, device="cuda") for _ in range(2))
    for t, start, n, written in (([[5, 6, 7]], 22, 4, 2), ([[5, -1, 7]], 6, 4, 2),
                                 ([[5, N, 7]], 6, 4, 2), ([[5, 6, 7]], -2, 4, 2),
                                 ([[5, 6, 7]], 0, 9, 4), ([[5, 6, 7]], 2 ** 31 - 1, 4, 0),
                                 ([[5, 6, 7]], -(2 ** 31), 4, 0)):
        k, v = K.clone(), V.clone()
        binding.cache_append(k, v, Kn, Vn, i32(t), i32([start]), i32([n]))
        assert status() == BOUNDS, (t, start, n)
        assert int((k != K).any(-1).any(-1).sum()) == written, (t, start, n)
        assert int((v != V).any(-1).any(-1).sum()) == written
    binding.cache_append(k, v, Kn, Vn, i32([[5, 6, 7]]), i32([0]), i32([-3]))
    assert status() == "ATTN_OK"  # a negative count is none


def compact_ref(pool, t, base, keep, block):
    """keep's rows to the front of each sequence, from the pool as it was."""
    out = pool.clone()
    for b, ks in enumerate(keep):
        for k, x in enumerate(ks):
            s, d = base[b] + x, base[b] + k
            out[t[b][d // block], d % block] = pool[t[b][s // block], s % block]
    return out


@pytest.mark.parametrize("B,Hkv,D,block,span,share", [
    (1, 1, 64, 8, 1, 1.0), (1, 8, 128, 16, 8, 0.5), (3, 2, 64, 8, 60, 0.3), (2, 3, 128, 64, 500, 0.9),
    (2, 1, 64, 16, 2000, 0.5), (1, 2, 128, 32, 700, 1.0), (4, 8, 128, 16, 129, 0.02),
    (2, 1, 64, 16, 7000, 0.9), (1, 3, 64, 8, 4097, 0.5001), (1, 1, 128, 4096, 9000, 0.3)])
def test_compact(B, Hkv, D, block, span, share):
    g = torch.Generator().manual_seed(span)
    base = [int(torch.randint(0, 40, (1,), generator=g)) for _ in range(B)]
    width = (max(base) + span) // block + 1
    N = B * width
    t = table(5, B, width, N, [b + span for b in base], block)
    K, V = pools(6, N, block, Hkv, D)
    keep = [torch.nonzero(torch.rand(span, generator=g) <= share).flatten().tolist() for _ in range(B)]
    A = max(1, max(len(k) for k in keep)) + 3
    wide = i32([k + [0] * (A - len(k)) for k in keep])  # entries past n_keep are not looked at
    want = [compact_ref(x.cpu(), t, base, keep, block) for x in (K, V)]
    binding.cache_compact(K, V, i32(t), i32(base), wide, i32([len(k) for k in keep]))
    assert status() == "ATTN_OK"
    assert torch.equal(K.cpu(), want[0]) and torch.equal(V.cpu(), want[1])


def test_compact_without_counts_keeps_every_entry():
    K, V = pools(7, 4, 8, 1, 64)
    t, keep = [[2, 0, 3]], [[1, 2, 9, 20, 23]]
    want = compact_ref(K.cpu(), t, [0], keep, 8)
    binding.cache_compact(K, V, i32(t), i32([0]), i32(keep))
    assert status() == "ATTN_OK" and torch.equal(K.cpu(), want)


@pytest.mark.parametrize("keep,n,base,entry", [
    ([3, 3, 5], 3, 0, None), ([5, 4, 6], 3, 0, None), ([-1, 2, 3], 3, 0, None), ([1, 2, 24], 3, 0, None),
    ([1, 2, 3], 3, -1, None), ([1, 2, 3], 3, 22, None), ([1, 9, 17], 3, 0, -1), ([1, 9, 17], 3, 0, 6),
    ([0, 1, 2], 3, 2 ** 31 - 1, None)])
def test_compact_refuses_bad_lists_whole(keep, n, base, entry):
    """The sequence with the bad list is left as it is, its neighbour is compacted."""
    K, V = pools(8, 6, 8, 2, 64)
    t = [[0, 1, 2], [3, 4, 5]]
    good = [0, 5, 11]
    want = compact_ref(K.cpu(), t, [0, 4], [[], good], 8)
    if entry is not None:
        t[0][1] = entry
    binding.cache_compact(K, V, i32(t), i32([base, 4]), i32([keep, good]), i32([n, 3]))
    assert status() == BOUNDS
    assert torch.equal(K.cpu(), want)


def test_compact_count_above_the_list_is_clamped_and_flagged():
    K, V = pools(9, 3, 8, 1, 64)
    t, keep = [[0, 1, 2]], [[2, 4]]
    want = compact_ref(K.cpu(), t, [0], keep, 8)
    binding.cache_compact(K, V, i32(t), i32([0]), i32(keep), i32([7]))
    assert status() == BOUNDS and torch.equal(K.cpu(), want)


@pytest.mark.parametrize("block,Hkv,D", [(8, 1, 64), (16, 8, 128), (64, 3, 64), (512, 2, 128)])
def test_copy_blocks(block, Hkv, D):
    N = 20
    K, V = pools(10, N, block, Hkv, D)
    src, dst = [3, -1, 3, 7, 8, 2], [4, 5, 0, 11, -1, 2]
    wk, wv = K.clone(), V.clone()
    for s, d in zip(src, dst):
        if s >= 0 and d >= 0:
            wk[d], wv[d] = K[s], V[s]
    binding.cache_copy_blocks(K, V, i32(src), i32(dst))
    assert status() == "ATTN_OK"
    assert torch.equal(K, wk) and torch.equal(V, wv)


def test_copy_blocks_that_meet_are_skipped_and_flagged():
    K, V = pools(11, 10, 8, 2, 64)
    for src, dst, runs in (([1, 2], [2, 3], [0]),         # the second reads what the first writes
                           ([1, 4], [5, 5], [1]),         # the later of two for one page
                           ([1, 10], [5, 6], [0]), ([1, 2], [5, 10], [0]),
                           ([1, 2, 3], [2, 3, 1], [])):   # a ring
        k, v = K.clone(), V.clone()
        wk = K.clone()
        for i in runs:
            wk[dst[i]] = K[src[i]]
        binding.cache_copy_blocks(k, v, i32(src), i32(dst))
        assert status() == BOUNDS and torch.equal(k, wk), (src, dst)


def test_copy_blocks_long_list():
    N = 3000
    K, V = pools(12, 2 * N, 8, 1, 64)
    perm = torch.randperm(2 * N, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    src, dst = perm[:N].contiguous(), perm[N:].contiguous()
    wk, wv = K.clone(), V.clone()
    wk[dst.long()], wv[dst.long()] = K[src.long()], V[src.long()]
    binding.cache_copy_blocks(K, V, src, dst)
    assert status() == "ATTN_OK" and torch.equal(K, wk) and torch.equal(V, wv)


# ---------------------------------------------------------------------------------
# tables
# ---------------------------------------------------------------------------------
class Model:
    """The bookkeeping in plain Python."""

    def __init__(self, t, n, block, lens):
        self.t, self.block, self.lens = [list(r) for r in t], block, list(lens)
        self.refs = [0] * n
        for r in t:
            for p in r:
                if p >= 0:
                    self.refs[p] += 1

    def take(self):
        for p, c in enumerate(self.refs):
            if c == 0:
                self.refs[p] = 1
                return p
        return -1

    def free(self, rows, first, last):
        for r, a, z in zip(rows, first, last):
            if r < 0:
                continue
            for k in range(max(a, 0), min(z, len(self.t[r]))):
                if self.t[r][k] >= 0:
                    self.refs[self.t[r][k]] -= 1
                    self.t[r][k] = -1

    def fork(self, parents, children):
        pairs, need = [], []
        for p, c in zip(parents, children):
            if p < 0 or c < 0:
                pairs.append((-1, -1))
                continue
            full = self.lens[p] // self.block
            row = self.t[p][:full] + [-1] * (len(self.t[p]) - full)
            for x in row:
                if x >= 0:
                    self.refs[x] += 1
            self.t[c], self.lens[c] = row, self.lens[p]
            src = self.t[p][full] if self.lens[p] % self.block else -1
            pairs.append((src, -1))
            if src >= 0:
                need.append((len(pairs) - 1, c, full))
        ok = True
        for i, c, full in need:
            page = self.take()
            ok &= page >= 0
            pairs[i] = (pairs[i][0], page) if page >= 0 else (-1, -1)
            self.t[c][full] = page
        return [s for s, _ in pairs], [d for _, d in pairs], ok

    def extend(self, frm, to):
        ok = True
        for r in range(len(self.t)):
            z = max(0, min((to[r] + self.block - 1) // self.block, len(self.t[r])))
            for k in range(max(frm[r], 0) // self.block, z):
                if self.t[r][k] < 0:
                    self.t[r][k] = self.take()
                    ok &= self.t[r][k] >= 0
        return ok

    def same(self, t, refs, lens=None):
        assert t.tolist() == self.t
        assert refs.tolist() == self.refs
        assert lens is None or lens.tolist() == self.lens


@pytest.mark.parametrize("seed,block,n,width", [(0, 16, 40, 6), (1, 8, 300, 40), (2, 64, 5000, 300),
                                                (3, 16, 70001, 700), (4, 8, 17, 4)])
def test_random_bookkeeping(seed, block, n, width):
    """Twelve rounds of free, fork and extend, every result compared; the smallest pools
    run out of pages now and then."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    R = 9
    most = min(width * block - 1, (n // R) * block)
    lens = [rnd(0, most) for _ in range(R)]
    lens[0] = most // block * block  # no part-filled page
    m = Model(table(seed, R, width, n, lens, block), n, block, lens)
    t, refs, L = i32(m.t), i32(m.refs), i32(m.lens)
    for _ in range(12):
        order = torch.randperm(R, generator=g).tolist()
        children, parents = order[:rnd(0, 4)], order[5:]
        rows = children + [order[4], -1]
        first = [0] * len(children) + [rnd(0, width), 0]
        last = [width + 9] * len(children) + [rnd(0, width), width]
        binding.cache_free(t, refs, i32(rows), i32(first), i32(last))
        m.free(rows, first, last)
        assert status() == "ATTN_OK"
        m.same(t, refs)
        pairs = [(parents[rnd(0, len(parents) - 1)], c) for c in children] + [(-1, 0), (1, -1)]
        par, chi = [p for p, _ in pairs], [c for _, c in pairs]
        src, dst = (torch.full((len(pairs),), 77, dtype=torch.int32, device="cuda") for _ in range(2))
        binding.cache_fork(t, refs, L, i32(par), i32(chi), src, dst, block)
        ws, wd, ok = m.fork(par, chi)
        assert status() == ("ATTN_OK" if ok else "ATTN_ERR_NO_PAGES")
        m.same(t, refs, L)
        assert src.tolist() == ws and dst.tolist() == wd
        to = [min(x + rnd(0, 3 * block), width * block) for x in m.lens]
        binding.cache_extend(t, refs, i32(m.lens), i32(to), block)
        ok = m.extend(m.lens, to)
        assert status() == ("ATTN_OK" if ok else "ATTN_ERR_NO_PAGES")
        m.same(t, refs)


def test_free_flags_what_is_not_held():
    t, refs = i32([[0, 1, 99, -5], [2, 2, 1, -1]]), i32([1, 2, 1])
    binding.cache_free(t, refs, i32([0, 1, 2]), i32([0, 0, 0]), i32([4, 2, 1]))
    assert status() == BOUNDS  # page 99, page 2 given back twice, row 2
    assert t.tolist() == [[-1, -1, -1, -1], [-1, -1, 1, -1]]  # any entry of the range becomes -1
    assert refs.tolist() == [0, 1, 0]
    # a row named twice gives its pages back once
    t, refs = i32([[0, 1]]), i32([1, 1])
    binding.cache_free(t, refs, i32([0, 0]), i32([0, 0]), i32([2, 2]))
    assert status() == "ATTN_OK" and refs.tolist() == [0, 0]
    # ranges outside the row
    t, refs = i32([[0, 1]]), i32([1, 1])
    binding.cache_free(t, refs, i32([0, 0]), i32([-(2 ** 31), 2]), i32([1, 2 ** 31 - 1]))
    assert status() == "ATTN_OK" and t.tolist() == [[-1, 1]] and refs.tolist() == [0, 1]


def test_fork_refuses_pairs_that_meet():
    """A child that is also a parent, or named twice, is skipped; the others go through."""
    lens = [20, 20, 0, 0, 0]
    base = [[0, 1, 2], [3, 4, 5], [-1] * 3, [-1] * 3, [-1] * 3]
    for par, chi, good in (([0, 0], [2, 2], [0]), ([0, 2], [2, 3], [1]), ([1, 0], [1, 3], [1]),
                           ([0, 0], [5, 3], [1]), ([7, 1], [2, 3], [1])):
        m = Model(base, 12, 8, lens)
        t, refs, L = i32(m.t), i32(m.refs), i32(m.lens)
        src, dst = i32([9, 9]), i32([9, 9])
        binding.cache_fork(t, refs, L, i32(par), i32(chi), src, dst, 8)
        assert status() == BOUNDS
        par2 = [p if i in good else -1 for i, p in enumerate(par)]
        ws, wd, _ = m.fork(par2, chi)
        m.same(t, refs, L)
        assert src.tolist() == ws and dst.tolist() == wd


def test_fork_many_pairs_from_few_parents():
    """1500 children of three parents in one call, in an order of their own; the pool runs out
    before the last of them."""
    R, block, n = 1503, 8, 1300
    lens = [21, 16, 5] + [0] * 1500
    m = Model([[0, 1, 2], [3, 4, -1], [5, -1, -1]] + [[-1] * 3] * 1500, n, block, lens)
    t, refs, L = i32(m.t), i32(m.refs), i32(m.lens)
    g = torch.Generator().manual_seed(4)
    par = torch.randint(0, 3, (1500,), generator=g).tolist()
    chi = (3 + torch.randperm(1500, generator=g)).tolist()
    for k in (5, 700, 1499):
        par[k] = 2  # parents with a part-filled page first, in the middle and last
    src, dst = (torch.full((1500,), 9, dtype=torch.int32, device="cuda") for _ in range(2))
    for r in range(3, 1200):  # most of the pool is taken
        m.refs[r + 3] = 1
    refs = i32(m.refs)
    binding.cache_fork(t, refs, L, i32(par), i32(chi), src, dst, block)
    ws, wd, ok = m.fork(par, chi)
    assert not ok and status() == "ATTN_ERR_NO_PAGES"
    m.same(t, refs, L)
    assert src.tolist() == ws and dst.tolist() == wd


def test_extend_keeps_freed_window_pages_empty():
    """Entries before from_lens stay as they are: pages that left a window come not back."""
    t, refs = i32([[4, -1, -1, 5, -1, -1]]), i32([0, 0, 0, 0, 1, 1])
    binding.cache_extend(t, refs, i32([30]), i32([47]), 8)
    assert status() == "ATTN_OK"
    assert t.tolist() == [[4, -1, -1, 5, 0, 1]] and refs.tolist() == [1, 1, 0, 0, 1, 1]
    binding.cache_extend(t, refs, i32([48]), i32([200]), 8)  # past the table
    assert status() == BOUNDS and t.tolist() == [[4, -1, -1, 5, 0, 1]]
    binding.cache_extend(t, refs, i32([-9]), i32([-1]), 8)
    assert status() == "ATTN_OK" and t.tolist() == [[4, -1, -1, 5, 0, 1]]


def test_extend_many_rows():
    R, width, n, block = 1500, 5, 9000, 16
    m = Model([[-1] * width for _ in range(R)], n, block, [0] * R)
    t, refs = i32(m.t), i32(m.refs)
    to = [(7 * r) % (width * block + 1) for r in range(R)]
    binding.cache_extend(t, refs, i32([0] * R), i32(to), block)
    m2 = [0]  # every page is free: they come in order
    for r in range(R):
        for k in range((to[r] + block - 1) // block):
            m.t[r][k] = m2[0]
            m2[0] += 1
    m.refs = [1 if p < m2[0] else 0 for p in range(n)]
    assert status() == "ATTN_OK"
    m.same(t, refs)


def test_large_pool_offsets_pass_32_bits():
    """Rows, pages and moves behind the first 2^31 elements of a pool."""
    block, Hkv, D = 256, 8, 128
    n = 2 ** 31 // (block * Hkv * D) + 4  # the last pages start past 2^31 elements (4.3 GB)
    K = torch.zeros(n, block, Hkv, D, dtype=BF, device="cuda")
    V = torch.zeros(n, block, Hkv, D, dtype=BF, device="cuda")
    t = i32([[n - 1, n - 2]])
    g = torch.Generator().manual_seed(0)
    Kn, Vn = (torch.randn(1, Hkv, 300, D, generator=g).to(BF).cuda() for _ in range(2))
    binding.cache_append(K, V, Kn, Vn, t, i32([100]))
    keep = torch.arange(0, 300, 3, dtype=torch.int32, device="cuda")[None].contiguous()
    binding.cache_compact(K, V, t, i32([100]), keep)
    binding.cache_copy_blocks(K, V, i32([n - 1]), i32([0]))
    assert status() == "ATTN_OK"
    for pool, new in ((K, Kn), (V, Vn)):
        want = new[0, :, keep[0].long()].transpose(0, 1)
        assert torch.equal(pool[n - 1, 100:200], want)
        assert torch.equal(pool[0], pool[n - 1])
    # attention over those pages
    q = torch.randn(1, 16, 4, D, generator=g).to(BF).cuda()
    O, P = torch.empty_like(q), torch.empty_like(q)
    par = i32([[-1, 0, 0, 2]])
    binding.attn_tree_paged(O, q, K, V, t, i32([190]), par)
    small = [x[n - 2:].contiguous() for x in (K, V)]
    binding.attn_tree_paged(P, q, *small, i32([[1, 0]]), i32([190]), par)
    d, e = torch.empty_like(q[:, :, 0]), torch.empty_like(q[:, :, 0])
    one = q[:, :, 0].contiguous()
    binding.attn_decode_paged_sinks(d, one, K, V, t, i32([400]), 150, 4)
    binding.attn_decode_paged_sinks(e, one, *small, i32([[1, 0]]), i32([400]), 150, 4)
    assert status() == "ATTN_OK"
    assert torch.equal(O, P) and torch.equal(d, e)
