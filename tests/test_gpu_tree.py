"""Attention of a tree of drafted tokens over a paged cache (attn_tree_paged) against the
definition in fp64: trees of every shape, contexts from none to long, page sizes that end
inside a tile, missing drafts, poisoned cache rows, bad tables.  Bounds as in
test_gpu_sinks.py: u = 2^-8 for each weight's and the result's rounding to bf16."""
import pytest
import torch

from gqa_attention_flash_b200 import binding
from gqa_attention_flash_b200 import workloads as W
from test_gpu_sinks import BF, F32, U, check, ref_fwd

pytestmark = pytest.mark.gpu


def tree(kind, B, T, seed=0):
    g = torch.Generator().manual_seed(seed)
    i = torch.arange(T)
    if kind == "chain":
        p = (i - 1).expand(B, T)
    elif kind == "star":
        p = torch.full((B, T), -1)
    elif kind == "binary":
        p = ((i + 1) // 2 - 1).expand(B, T)
    else:
        p = (torch.rand(B, T, generator=g) * (i + 1)).long() - 1
    return p.to(torch.int32).contiguous()


def ancestors(parents):
    B, T = parents.shape
    m = torch.zeros(B, T, T, dtype=torch.bool)
    for b in range(B):
        p = parents[b].tolist()
        for i in range(T):
            if 0 <= p[i] < i:
                m[b, i] = m[b, p[i]]
            m[b, i, i] = True
    return m


def make(seed, B, Hq, Hkv, D, T, ctx, drafts, block, poison=0.0, spare=3):
    g = torch.Generator().manual_seed(seed)
    lens = [c + d for c, d in zip(ctx, drafts)]
    tables, nblk = W.paged_layout(lens, block, spare, seed)
    Kp = torch.full((nblk, block, Hkv, D), poison, dtype=BF)
    Vp = Kp.clone()
    kv = [(torch.randn(Hkv, n, D, generator=g).to(BF), torch.randn(Hkv, n, D, generator=g).to(BF))
          for n in lens]
    W.fill_paged_cache(Kp, Vp, tables, lambda b: kv[b])
    for b, n in enumerate(lens):
        if n % block:
            Kp[tables[b, n // block], n % block:] = poison
            Vp[tables[b, n // block], n % block:] = poison
    Q = torch.randn(B, Hq, T, D, generator=g).to(BF)
    for b in range(B):
        Q[b, :, drafts[b]:] = poison
    dev = [x.cuda() for x in (Q, Kp, Vp, tables)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return (*dev, i32(ctx), i32(drafts), kv)


def reference(Q, kv, parents, ctx, drafts):
    """O and sum p |v| per sequence in fp64; rows without a draft are 0."""
    anc = ancestors(parents)
    O, M = (torch.zeros(Q.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for b, (k, v) in enumerate(kv):
        c, d = ctx[b], drafts[b]
        if d <= 0:
            continue
        vis = torch.ones(d, c + d, dtype=torch.bool)
        vis[:, c:] = anc[b, :d, :d]
        O[b, :, :d], _, _, M[b, :, :d] = (
            x[0] if x.dim() == 4 else x for x in ref_fwd(Q[b:b + 1, :, :d], k[None].cuda(),
                                                         v[None].cuda(), vis.cuda()[None, None],
                                                         Q.shape[-1] ** -0.5))
    return O, M


def run(Q, Kp, Vp, tables, ctx, parents, drafts):
    O = torch.full_like(Q, float("nan"))
    binding.attn_tree_paged(O, Q, Kp, Vp, tables, ctx, parents.cuda(), drafts)
    return O


CASES = [
    # B, Hq, Hkv, D, T, ctx, drafts, block, tree
    (1, 2, 1, 128, 1, [0], [1], 16, "chain"),               # the first token of all
    (1, 2, 1, 64, 1, [77], [1], 8, "chain"),                # single-token decode
    (3, 8, 2, 128, 8, [0, 1, 300], [8, 8, 8], 16, "random"),
    (4, 8, 2, 128, 7, [120, 121, 127, 128], [7, 7, 7, 7], 16, "binary"),  # around a tile's end
    (3, 4, 4, 64, 33, [500, 95, 31], [33, 1, 0], 32, "star"),
    (2, 32, 8, 128, 16, [1000, 517], [16, 9], 16, "random"),
    (2, 16, 1, 128, 5, [200, 300], [5, 5], 64, "random"),
    (1, 3, 3, 64, 64, [250], [64], 8, "chain"),
    (2, 12, 4, 128, 64, [700, 3], [64, 40], 256, "random"),
    (1, 8, 2, 128, 128, [130], [128], 16, "binary"),
    (1, 4, 2, 64, 256, [300], [256], 16, "random"),
    (1, 16, 1, 128, 100, [90], [99], 128, "random"),        # 1600 rows of one KV head
    (2, 6, 2, 128, 3, [2900, 2048], [3, 2], 512, "star"),
    (1, 10, 2, 128, 26, [60], [26], 16, "random"),          # 130 rows: one past a tile
    (2, 5, 5, 64, 9, [4500, 100], [9, 2], 4096, "random"),  # pages of many tiles
    (1, 64, 64, 64, 2, [300], [2], 8, "star"),              # more KV heads than lanes divide evenly
    (1, 37, 37, 128, 3, [130], [3], 16, "binary"),
    (1, 150, 150, 64, 1, [20], [1], 16, "chain"),
    (8, 4, 1, 64, 4, [0, 5, 64, 128, 129, 700, 1500, 2], [4, 4, 4, 0, 1, 4, 4, 4], 16, "random"),
]


@pytest.mark.parametrize("poison", [0.0, float("nan")])
@pytest.mark.parametrize("c", CASES, ids=[str(c) for c in CASES])
def test_tree(c, poison):
    B, Hq, Hkv, D, T, ctx, drafts, block, kind = c
    Q, Kp, Vp, tables, cl, dl, kv = make(B + T, B, Hq, Hkv, D, T, ctx, drafts, block, poison)
    parents = tree(kind, B, T, T)
    O = run(Q, Kp, Vp, tables, cl, parents, dl)
    assert binding.last_device_status() == 0
    want, mag = reference(torch.nan_to_num(Q, nan=0.0), kv, parents, ctx, drafts)
    check(O, want, U * (mag + want.abs()) + 2 * F32 * mag, "O")  # up to 2^11 keys
    for b in range(B):
        assert torch.all(O[b, :, drafts[b]:] == 0)


def test_draft_lens_default_is_all():
    Q, Kp, Vp, tables, cl, dl, _ = make(1, 2, 4, 2, 128, 6, [50, 9], [6, 6], 16)
    parents = tree("random", 2, 6)
    assert torch.equal(run(Q, Kp, Vp, tables, cl, parents, dl), run(Q, Kp, Vp, tables, cl, parents, None))


def test_a_chain_is_causal_prefill():
    """A chain of drafts is a causal chunk of a prefill on the same keys."""
    B, Hq, Hkv, D, T, c = 1, 8, 2, 128, 40, 333
    Q, Kp, Vp, tables, cl, dl, kv = make(2, B, Hq, Hkv, D, T, [c], [T], 16)
    O = run(Q, Kp, Vp, tables, cl, tree("chain", B, T), dl)
    P, L = torch.empty_like(Q), torch.empty((B, Hq, T), device="cuda")
    K, V = kv[0][0][None].cuda(), kv[0][1][None].cuda()
    binding.attn_fwd(P, Q, K, V, L, D ** -0.5, True, input_pos=c)
    vis = torch.arange(c + T) <= c + torch.arange(T)[:, None]
    want, _, _, mag = ref_fwd(Q, K, V, vis.cuda()[None, None], D ** -0.5)
    bound = U * (mag + want.abs()) + F32 * mag
    check(O, want, bound, "tree")
    check(P, want, bound, "prefill")


def test_bad_parents_tables_and_lengths():
    """Out-of-range parents count as the context, pages outside the pool read as zeros,
    lengths past the table are clamped; each sets the status word."""
    ctx, drafts, T = [40, 100], [6, 6], 6
    Q, Kp, Vp, tables, cl, dl, kv = make(3, 2, 4, 2, 128, T, ctx, drafts, 16)
    good = tree("random", 2, T, 5)
    bad = good.clone()
    bad[0, 2], bad[0, 4], bad[1, 3] = 2, 9, -7
    fixed = good.clone()
    fixed[0, 2] = fixed[0, 4] = fixed[1, 3] = -1
    a = run(Q, Kp, Vp, tables, cl, bad, dl)
    assert binding.STATUS[binding.last_device_status()] == "ATTN_ERR_DEVICE_BOUNDS"
    b = run(Q, Kp, Vp, tables, cl, fixed, dl)
    assert binding.last_device_status() == 0
    assert torch.equal(a, b)
    for page in (-1, -(2 ** 31), Kp.shape[0], 2 ** 31 - 1):
        t = tables.clone()
        t[1, 2] = page
        got = run(Q, Kp, Vp, t, cl, good, dl)
        assert binding.STATUS[binding.last_device_status()] == "ATTN_ERR_DEVICE_BOUNDS"
        kv2 = [kv[0], tuple(x.clone() for x in kv[1])]
        for x in kv2[1]:
            x[:, 32:48] = 0
        want, mag = reference(Q, kv2, good, ctx, drafts)
        check(got, want, U * (mag + want.abs()) + F32 * mag, f"page {page}")
    cap = tables.shape[1] * 16
    for c2, d2 in ((2 ** 31 - 1, 6), (cap - 2, 6), (-5, 6), (40, 7), (40, -3)):
        clx, dlx = cl.clone(), dl.clone()
        clx[0], dlx[0] = c2, d2
        full = tables.clone()
        full[0][full[0] < 0] = 0
        got = run(Q, Kp, Vp, full, clx, good, dlx)
        st = binding.last_device_status()
        assert (st == 0) == (d2 == -3), (c2, d2)  # no drafts is no error
        cx = min(max(c2, 0), cap)
        dx = max(0, min(d2, T, cap - cx))
        clx[0], dlx[0] = cx, dx
        assert torch.equal(got, run(Q, Kp, Vp, full, clx, good, dlx)), (c2, d2)
        assert binding.last_device_status() == 0


def test_unused_entries_are_not_read():
    Q, Kp, Vp, tables, cl, dl, _ = make(4, 2, 4, 2, 64, 4, [30, 200], [4, 4], 8)
    a = run(Q, Kp, Vp, tables, cl, tree("star", 2, 4), dl)
    t = torch.where(tables < 0, 2 ** 30, tables)  # entries past the last page
    b = run(Q, Kp, Vp, t, cl, tree("star", 2, 4), dl)
    assert binding.last_device_status() == 0 and torch.equal(a, b)


def test_large_batch_matches_per_sequence_calls():
    """The whole batch at once is each sequence for itself, within the two results' bounds."""
    B, Hq, Hkv, D, T = 40, 32, 8, 128, 12
    g = torch.Generator().manual_seed(8)
    ctx = torch.randint(0, 2500, (B,), generator=g).tolist()
    drafts = torch.randint(0, T + 1, (B,), generator=g).tolist()
    Q, Kp, Vp, tables, cl, dl, kv = make(6, B, Hq, Hkv, D, T, ctx, drafts, 16)
    parents = tree("random", B, T, 3)
    O = run(Q, Kp, Vp, tables, cl, parents, dl)
    assert binding.last_device_status() == 0
    for b in (0, 1, 7, 20, 39):
        want, mag = reference(Q[b:b + 1], kv[b:b + 1], parents[b:b + 1], ctx[b:b + 1], drafts[b:b + 1])
        bound = U * (mag + want.abs()) + 4 * F32 * mag
        check(O[b:b + 1], want, bound, f"sequence {b} of the batch")
        one = run(Q[b:b + 1].contiguous(), Kp, Vp, tables[b:b + 1].contiguous(), cl[b:b + 1].clone(),
                  parents[b:b + 1].contiguous(), dl[b:b + 1].clone())
        check(one, want, bound, f"sequence {b} alone")


def test_graph_replay_with_new_lengths_and_two_graphs():
    """Two captured calls replayed in turn, on inputs that change between replays."""
    B, Hq, Hkv, D, T = 3, 8, 2, 128, 8
    Q, Kp, Vp, tables, cl, dl, kv = make(9, B, Hq, Hkv, D, T, [900, 40, 300], [8, 8, 8], 16)
    parents = tree("random", B, T).cuda()
    outs = [torch.empty_like(Q) for _ in range(2)]
    graphs = []
    for o in outs:
        binding.attn_tree_paged(o, Q, Kp, Vp, tables, cl, parents, dl)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            binding.attn_tree_paged(o, Q, Kp, Vp, tables, cl, parents, dl)
        graphs.append(graph)
    for new in ([900, 40, 300], [5, 0, 111], [700, 32, 1]):
        cl.copy_(torch.tensor(new, dtype=torch.int32))
        Q.mul_(-0.5)
        want = run(Q, Kp, Vp, tables, cl, parents, dl)
        streams = [torch.cuda.Stream() for _ in graphs]
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):  # both at once, on their own streams
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
    assert binding.last_device_status() == 0
