"""The cache's operators and the attention that reads it, together, as a serving loop uses
them: prompts forked and extended, drafts appended, checked as a tree and compacted, pages
given back behind a sliding window, every attention result against fp64 on the tokens that
each sequence really holds; and one such step captured in a graph."""
import pytest
import torch

from gqa_attention_flash_b200 import binding
from test_gpu_sinks import BF, F32, U, check, ref_fwd, visible
from test_gpu_tree import ancestors, tree

pytestmark = pytest.mark.gpu

HQ, HKV, D, BLOCK = 8, 2, 128, 16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Stream:
    """Device state of the loop, and beside it the tokens' K and V that each row holds."""

    def __init__(self, rows, width, pages, seed=0):
        self.g = torch.Generator().manual_seed(seed)
        self.K = torch.full((pages, BLOCK, HKV, D), float("nan"), dtype=BF, device="cuda")
        self.V = self.K.clone()
        self.t = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.kv = [(torch.zeros(HKV, 0, D, dtype=BF, device="cuda"),) * 2 for _ in range(rows)]

    def rand(self, *shape):
        return torch.randn(shape, generator=self.g).to(BF).cuda()

    def append(self, rows, Kn, Vn, n):
        """n[b] new tokens of each of the rows: pages, K and V; lens stays."""
        start = self.lens[rows].contiguous()
        to = self.lens.clone()
        to[rows] += n
        binding.cache_extend(self.t, self.refs, self.lens, to, BLOCK)
        binding.cache_append(self.K, self.V, Kn, Vn, self.t[rows].contiguous(), start, n)
        return start

    def hold(self, row, k, v):
        self.kv[row] = tuple(torch.cat([a, b], 1) for a, b in zip(self.kv[row], (k, v)))

    def consistent(self):
        """Every count is the number of table entries that name the page; no page of a
        sequence's last, part-filled slot is shared."""
        used = self.t[self.t >= 0].long()
        assert torch.equal(torch.bincount(used, minlength=self.refs.numel()), self.refs.long())


def test_speculative_steps_with_forks_and_a_window():
    s = Stream(rows=5, width=40, pages=120)
    live = torch.tensor([0, 1])
    # two prompts of their own length, prefilled and written to their pages
    T = 70
    Kn, Vn, Q = s.rand(2, HKV, T, D), s.rand(2, HKV, T, D), s.rand(2, HQ, T, D)
    n = i32([70, 53])
    s.append(live, Kn, Vn, n)
    O, L = torch.empty_like(Q), torch.empty((2, HQ, T), device="cuda")
    binding.attn_fwd_sinks(O, Q, Kn, Vn, L, D ** -0.5, 30, 4, 0, n, n)
    for b in range(2):
        m = int(n[b])
        want, _, _, mag = ref_fwd(Q[b:b + 1, :, :m], Kn[b:b + 1, :, :m], Vn[b:b + 1, :, :m],
                                  visible(m, m, 30, 4, 0)[None, None], D ** -0.5)
        check(O[b:b + 1, :, :m], want, U * (mag + want.abs()) + F32 * mag, "prefill")
        s.hold(b, Kn[b, :, :m], Vn[b, :, :m])
    s.lens[live] += n
    s.consistent()
    # each prompt goes on in another row too; row 4 stays empty
    src, dst = i32([0, 0]), i32([0, 0])
    binding.cache_fork(s.t, s.refs, s.lens, i32([0, 1]), i32([2, 3]), src, dst, BLOCK)
    binding.cache_copy_blocks(s.K, s.V, src, dst)
    assert s.lens.tolist() == [70, 53, 70, 53, 0]
    assert (src >= 0).tolist() == [True, True]
    s.kv[2], s.kv[3] = s.kv[0], s.kv[1]
    s.consistent()
    live = torch.tensor([0, 1, 2, 3])
    for step in range(6):
        T = [7, 1, 16, 5, 12, 3][step]
        drafts = torch.tensor([T, max(T - 2, 0), T, (T + 1) // 2], dtype=torch.int32).cuda()
        Kn, Vn, Q = s.rand(4, HKV, T, D), s.rand(4, HKV, T, D), s.rand(4, HQ, T, D)
        start = s.append(live, Kn, Vn, drafts)
        parents = tree("random", 4, T, step)
        O = torch.empty_like(Q)
        tables = s.t[live].contiguous()
        binding.attn_tree_paged(O, Q, s.K, s.V, tables, start, parents.cuda(), drafts)
        anc = ancestors(parents)
        keep, count = torch.zeros(4, T, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
        for b in range(4):
            d = int(drafts[b])
            k = torch.cat([s.kv[b][0], Kn[b, :, :d]], 1)[None]
            v = torch.cat([s.kv[b][1], Vn[b, :, :d]], 1)[None]
            if d:
                vis = torch.ones(d, k.shape[2], dtype=torch.bool)
                vis[:, k.shape[2] - d:] = anc[b, :d, :d]
                want, _, _, mag = ref_fwd(Q[b:b + 1, :, :d], k, v, vis.cuda()[None, None], D ** -0.5)
                check(O[b:b + 1, :, :d], want, U * (mag + want.abs()) + F32 * mag, f"step {step} row {b}")
                path = torch.nonzero(anc[b, d - 1, :d]).flatten()  # the last draft is accepted
                keep[b, :len(path)], count[b] = path.to(torch.int32), len(path)
        binding.cache_compact(s.K, s.V, tables, start, keep.cuda(), count.cuda())
        for b in range(4):
            p = keep[b, :count[b]].long().cuda()
            s.hold(b, Kn[b][:, p], Vn[b][:, p])
        s.lens[live] += count.cuda()
        # pages behind the accepted tokens go back
        first = (s.lens + BLOCK - 1) // BLOCK
        binding.cache_free(s.t, s.refs, torch.arange(5, dtype=torch.int32, device="cuda"),
                           first.to(torch.int32), torch.full_like(s.lens, 40))
        s.consistent()
        assert [x[0].shape[1] for x in s.kv] == s.lens.tolist()
    # then windowed single tokens, the pages that left the window given back as they go
    W_, S_ = 37, 4
    for step in range(20):
        Kn, Vn, q = s.rand(4, HKV, 1, D), s.rand(4, HKV, 1, D), s.rand(4, HQ, D)
        one = torch.ones(4, dtype=torch.int32, device="cuda")
        s.append(live, Kn, Vn, one)
        s.lens[live] += 1
        for b in range(4):
            s.hold(b, Kn[b], Vn[b])
        gone = torch.clamp((s.lens - W_) // BLOCK, min=0).to(torch.int32)
        binding.cache_free(s.t, s.refs, torch.arange(5, dtype=torch.int32, device="cuda"),
                           torch.full_like(gone, 1), gone)
        s.consistent()
        o = torch.empty_like(q)
        binding.attn_decode_paged_sinks(o, q, s.K, s.V, s.t[live].contiguous(),
                                        s.lens[live].contiguous(), W_, S_)
        for b in range(4):
            k, v = s.kv[b]
            vis = visible(1, k.shape[1], W_, S_, k.shape[1] - 1)
            want, _, _, mag = ref_fwd(q[b:b + 1, :, None], k[None], v[None], vis[None, None], D ** -0.5)
            check(o[b:b + 1], want[:, :, 0], (U * (mag + want.abs()) + F32 * mag)[:, :, 0], f"token {step}")
    assert binding.last_device_status() == 0
    # everything given back leaves an empty pool
    binding.cache_free(s.t, s.refs, torch.arange(5, dtype=torch.int32, device="cuda"),
                       torch.zeros_like(s.lens), torch.full_like(s.lens, 40))
    assert binding.last_device_status() == 0
    assert not s.refs.any() and (s.t == -1).all()


def test_captured_step_advances_the_cache():
    """extend, append, tree, compact and free of one step in a graph: replays go on from the
    state that the replay before left, as the same calls made one by one do."""
    T = 6
    parents = tree("random", 2, T, 2).cuda()
    keep, count = i32([[0, 2, 3, 0, 0, 0], [1, 4, 0, 0, 0, 0]]), i32([3, 2])

    def make():
        s = Stream(rows=2, width=30, pages=64, seed=7)
        s.append(torch.tensor([0, 1]), s.rand(2, HKV, 40, D), s.rand(2, HKV, 40, D), i32([40, 9]))
        s.lens += i32([40, 9])
        s.new = [s.rand(2, HKV, T, D), s.rand(2, HKV, T, D), s.rand(2, HQ, T, D)]
        s.O = torch.zeros_like(s.new[2])
        return s

    def step(s):
        Kn, Vn, Q = s.new
        binding.cache_extend(s.t, s.refs, s.lens, s.lens + T, BLOCK)
        binding.cache_append(s.K, s.V, Kn, Vn, s.t, s.lens)
        binding.attn_tree_paged(s.O, Q, s.K, s.V, s.t, s.lens, parents)
        binding.cache_compact(s.K, s.V, s.t, s.lens, keep, count)
        s.lens += count
        rows = torch.arange(2, dtype=torch.int32, device="cuda")
        first = ((s.lens + BLOCK - 1) // BLOCK).to(torch.int32)
        binding.cache_free(s.t, s.refs, rows, first, torch.full_like(first, 30))
        for x in s.new:
            x.mul_(-0.75)

    a, b = make(), make()
    step(a)
    step(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for i in range(9):
        graph.replay()
        step(b)
        assert torch.equal(a.O, b.O), i
        assert torch.equal(a.t, b.t) and torch.equal(a.refs, b.refs) and torch.equal(a.lens, b.lens)
    assert torch.equal(torch.nan_to_num(a.K), torch.nan_to_num(b.K))
    assert binding.last_device_status() == 0


def test_two_streams_of_calls_at_once():
    """The same calls on two streams at a time, each with its own cache."""
    outs = []
    for parallel in (False, True):
        streams = [torch.cuda.Stream() for _ in range(2)]
        states = []
        for i in range(2):
            s = Stream(rows=3, width=80, pages=300, seed=i)
            s.append(torch.tensor([0, 1, 2]), s.rand(3, HKV, 900, D), s.rand(3, HKV, 900, D),
                     i32([900, 300, 1]))
            s.lens += i32([900, 300, 1])
            s.Q = s.rand(3, HQ, 8, D)
            s.O = torch.empty_like(s.Q)
            s.o = torch.empty((3, HQ, D), dtype=BF, device="cuda")
            states.append(s)
        torch.cuda.synchronize()
        for _ in range(5):
            for s, st in zip(states, streams):
                with torch.cuda.stream(st):
                    binding.attn_tree_paged(s.O, s.Q, s.K, s.V, s.t, torch.clamp(s.lens - 8, min=0),
                                            tree("binary", 3, 8).cuda(), i32([8, 8, 1]))
                    binding.attn_decode_paged_sinks(s.o, s.O[:, :, 0].contiguous(), s.K, s.V, s.t,
                                                    s.lens, 256, 4, 12)
                if not parallel:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        outs.append([x.clone() for s in states for x in (s.O, s.o)])
    assert binding.last_device_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(*outs))
