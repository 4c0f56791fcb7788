"""Cases of the operators that serve and train long streams over a paged cache, with
their plain forms: attention with a sliding window and sinks (prefill, backward,
single-token decode), attention of a tree of drafted tokens over a paged cache, and
the cache's own operators (append, compact, fork, extend, free, copy).

``run`` computes an operator with elementary torch operations in fp32 (``own`` false)
or calls this package's binding (``own`` true); ``exact`` computes it in fp64.
"""
import math

import torch

own = False

DEV = "cuda"
BF = torch.bfloat16
NEG = float("-inf")


# ---------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------
def listed():
    return [
        # one short head pair: what a test or a tiny model calls; latency
        dict(name="sink_fwd_tiny", op="sink_fwd", B=1, Hq=2, Hkv=1, D=64, Sq=128, input_pos=0,
             window=48, sinks=4, ragged=False),
        # ragged long-stream prefill (the sliding-window workload of the benchmark, with sinks)
        dict(name="sink_fwd_stream", op="sink_fwd", B=2, Hq=32, Hkv=8, D=128, Sq=16384, input_pos=0,
             window=4096, sinks=4, ragged=True),
        # a training step of a small model on ragged sequences of odd length
        dict(name="sink_bwd_small", op="sink_bwd", B=2, Hq=8, Hkv=2, D=64, Sq=1000, input_pos=0,
             window=200, sinks=5, ragged=True),
        # the causal training shape of the benchmark, with a window of a quarter
        dict(name="sink_bwd_llm", op="sink_bwd", B=4, Hq=32, Hkv=8, D=128, Sq=4096, input_pos=0,
             window=1024, sinks=4, ragged=False),
        # one stream, one token, contiguous cache: latency of a chat's next token
        dict(name="sink_decode_one", op="sink_decode", B=1, Hq=32, Hkv=8, D=128, cap=8192, lo=8000,
             window=1024, sinks=4, block=0),
        # a full serving batch over 16-token pages, pages outside the window freed
        dict(name="sink_decode_paged", op="sink_decode", B=64, Hq=32, Hkv=8, D=128, cap=32768,
             lo=1024, window=4096, sinks=4, block=16),
        # speculative decoding of one stream: eight drafts over a short context; latency
        dict(name="tree_one", op="tree", B=1, Hq=32, Hkv=8, D=128, T=8, ctx_lo=900, ctx_hi=1100,
             block=16),
        # speculative decoding of the benchmark's paged serving batch, ragged contexts
        dict(name="tree_batch", op="tree", B=64, Hq=32, Hkv=8, D=128, T=16, ctx_lo=1024,
             ctx_hi=32768, block=16),
        # two streams sampled twice each from short prompts
        dict(name="cache_fork_small", op="fork", parents=2, children=2, Hkv=2, D=128, lo=20, hi=90,
             grow=1, block=16),
        # parallel sampling: sixteen long prompts, three more continuations of each
        dict(name="cache_fork_batch", op="fork", parents=16, children=48, Hkv=8, D=128, lo=1024,
             hi=32768, grow=17, block=16),
        # one stream's eight drafts written, the accepted path kept
        dict(name="cache_commit_one", op="commit", B=1, Hkv=8, D=128, T=8, start_lo=900,
             start_hi=1100, keep=0.5, block=16),
        # four prompts written to their pages, then pruned to half of their rows
        dict(name="cache_commit_prune", op="commit", B=4, Hkv=8, D=128, T=4096, start_lo=0,
             start_hi=60, keep=0.5, block=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _heads(rng, most=32):
    while True:
        Hkv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8, 16])
        if Hkv * G <= most:
            return Hkv * G, Hkv


def draw(rng):
    op = rng.choice(["sink_fwd", "sink_bwd", "sink_decode", "tree", "fork", "commit"])
    D = rng.choice([64, 128])
    while True:
        if op in ("sink_fwd", "sink_bwd"):
            Hq, Hkv = _heads(rng)
            c = dict(op=op, B=_log(rng, 1, 4), Hq=Hq, Hkv=Hkv, D=D, Sq=_log(rng, 1, 16384),
                     input_pos=_log(rng, 1, 8192) if rng.random() < 0.35 else 0,
                     window=_log(rng, 1, 4096), sinks=_log(rng, 1, 200) - 1,
                     ragged=rng.random() < 0.5)
            dense = c["B"] * Hq * c["Sq"] * (c["Sq"] + c["input_pos"])
            if dense <= (2 * 32 * 16384 ** 2 if op == "sink_fwd" else 4 * 32 * 4096 ** 2) // 2:
                return c
        elif op == "sink_decode":
            Hq, Hkv = _heads(rng)
            cap = _log(rng, 16, 32768)
            c = dict(op=op, B=_log(rng, 1, 64), Hq=Hq, Hkv=Hkv, D=D, cap=cap,
                     lo=rng.randint(0, cap), window=_log(rng, 1, 4096), sinks=_log(rng, 1, 100) - 1,
                     block=rng.choice([0, 8, 16, 32, 64, 256]))
            if c["B"] * cap * Hkv <= 64 * 32768 * 8:
                return c
        elif op == "tree":
            Hq, Hkv = _heads(rng)
            hi = _log(rng, 1, 32768)
            c = dict(op=op, B=_log(rng, 1, 64), Hq=Hq, Hkv=Hkv, D=D, T=_log(rng, 1, 128),
                     ctx_lo=rng.randint(0, hi), ctx_hi=hi, block=rng.choice([8, 16, 32, 64, 256]))
            if c["B"] * hi * max(Hkv * 128, Hq * c["T"]) <= 64 * 32768 * 1024 // 2:
                return c
        elif op == "fork":
            hi = _log(rng, 2, 32768)
            P = _log(rng, 1, 16)
            c = dict(op=op, parents=P, children=_log(rng, 1, 48), Hkv=rng.choice([1, 2, 4, 8]), D=D,
                     lo=rng.randint(1, hi), hi=hi, grow=_log(rng, 1, 64),
                     block=rng.choice([8, 16, 32, 64]))
            return c
        else:
            B = _log(rng, 1, 64)
            hi = _log(rng, 1, 4096)
            return dict(op=op, B=B, Hkv=rng.choice([1, 2, 4, 8]), D=D,
                        T=_log(rng, 1, 16384 // B), start_lo=rng.randint(0, hi), start_hi=hi,
                        keep=round(rng.uniform(0.05, 1.0), 3), block=rng.choice([8, 16, 32, 64]))


# ---------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV).to(torch.int32)


def _sink_qkv(g, B, Hq, Hkv, Sq, Sk, D, sinks):
    """N(0, 1) tensors whose first keys answer a direction that every query has in
    common, as the first tokens of a trained model do."""
    u = _rand(g, 1, Hkv, 1, D)
    Q = _rand(g, B, Hq, Sq, D) + 0.5 * u.repeat_interleave(Hq // Hkv, 1)
    K = _rand(g, B, Hkv, Sk, D)
    K[:, :, :sinks] += u
    return Q.to(BF), K.to(BF), _rand(g, B, Hkv, Sk, D).to(BF)


def _pages(g, lengths, block, spare, longest=None):
    """Tables (B, max_blocks) of distinct pages in a random order, -1 past the end, and the
    number of pages; with ``longest`` both sizes are those of B sequences of that length."""
    n = [(int(x) + block - 1) // block for x in lengths]
    most, total = max(1, max(n)), sum(n)
    if longest is not None:
        most = (longest + block - 1) // block
        total = most * len(n)
    perm = torch.randperm(total + spare, generator=g, device=DEV).to(torch.int32)
    tables = torch.full((len(n), most), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, k in enumerate(n):
        tables[b, :k] = perm[at:at + k]
        at += k
    return tables, total + spare


def prepare(case, seed):
    g = _gen(seed)
    c, op = case, case["op"]
    s = {"case": c}
    if op in ("sink_fwd", "sink_bwd"):
        B, Hq, Hkv, D, Sq, pos = c["B"], c["Hq"], c["Hkv"], c["D"], c["Sq"], c["input_pos"]
        Sk = Sq + pos
        s["Q"], s["K"], s["V"] = _sink_qkv(g, B, Hq, Hkv, Sq, Sk, D, min(c["sinks"], Sk))
        s["q_len"] = s["k_len"] = None
        if c["ragged"]:
            s["q_len"] = _ints(g, (Sq + 1) // 2, Sq, B)
            s["k_len"] = (s["q_len"] + pos).to(torch.int32)
        s["scale"] = 1.0 / math.sqrt(D)
        s["O"], s["LSE"] = torch.empty_like(s["Q"]), torch.empty(B, Hq, Sq, device=DEV)
        if op == "sink_bwd":
            s["dO"] = _rand(g, B, Hq, Sq, D).to(BF)
            s["dQ"], s["dK"], s["dV"] = (torch.empty_like(s[k]) for k in ("Q", "K", "V"))
            O, LSE = _plain_fwd(s)
            s["O"].copy_(O)
            s["LSE"].copy_(LSE)
    elif op == "sink_decode":
        B, Hq, Hkv, D, cap = c["B"], c["Hq"], c["Hkv"], c["D"], c["cap"]
        s["len"] = _ints(g, c["lo"], cap, B)
        u = _rand(g, Hkv, D)
        s["Q"] = (_rand(g, B, Hq, D) + 0.5 * u.repeat_interleave(Hq // Hkv, 0)).to(BF)
        if c["block"]:
            s["tables"], n = _pages(g, s["len"].tolist(), c["block"], 8)
            s["K"] = _rand(g, n, c["block"], Hkv, D).to(BF)
            s["V"] = _rand(g, n, c["block"], Hkv, D).to(BF)
            first = torch.arange(min(c["sinks"], cap), device=DEV)
            rows = s["tables"].long()[:, (first // c["block"]).clamp(max=s["tables"].shape[1] - 1)]
            rows = (rows * c["block"] + first % c["block"])[rows >= 0]
            s["K"].view(-1, Hkv, D)[rows] += u.to(BF)
            # the pages that no later token of a stream sees have been given back
            k = torch.arange(s["tables"].shape[1], device=DEV)
            gone = (k >= -(-c["sinks"] // c["block"])) & (
                (k + 1) * c["block"] <= (s["len"] - c["window"])[:, None])
            s["tables"] = s["tables"].masked_fill(gone, -1)
        else:
            s["K"] = _rand(g, B, Hkv, cap, D).to(BF)
            s["K"][:, :, :c["sinks"]] += u.to(BF)[None, :, None]
            s["V"] = _rand(g, B, Hkv, cap, D).to(BF)
        s["O"] = torch.empty_like(s["Q"])
    elif op == "tree":
        B, Hq, Hkv, D, T = c["B"], c["Hq"], c["Hkv"], c["D"], c["T"]
        s["ctx"] = _ints(g, c["ctx_lo"], c["ctx_hi"], B)
        s["drafts"] = _ints(g, (T + 1) // 2, T, B)
        s["tables"], n = _pages(g, (s["ctx"] + s["drafts"]).tolist(), c["block"], 8)
        s["K"] = _rand(g, n, c["block"], Hkv, D).to(BF)
        s["V"] = _rand(g, n, c["block"], Hkv, D).to(BF)
        s["Q"] = _rand(g, B, Hq, T, D).to(BF)
        # draft i continues the context (-1) or an earlier draft; late ones more often
        i = torch.arange(T, device=DEV)
        r = torch.rand(B, T, generator=g, device=DEV).sqrt()
        s["parents"] = torch.minimum((r * (i + 1)).long() - 1, i - 1).to(torch.int32).contiguous()
        s["O"] = torch.empty_like(s["Q"])
    elif op == "fork":
        P, C, bs = c["parents"], c["children"], c["block"]
        R = P + C
        lens = torch.zeros(R, dtype=torch.int32, device=DEV)
        lens[:P] = _ints(g, c["lo"], c["hi"], P)
        grow = (c["grow"] + bs - 1) // bs + 1
        held, n = _pages(g, lens[:P].tolist(), bs, R * (grow + 1) + 8, c["hi"])
        s["tables"] = torch.full((R, held.shape[1] + grow), -1, dtype=torch.int32, device=DEV)
        s["tables"][:P, :held.shape[1]] = held
        s["refs"] = torch.zeros(n, dtype=torch.int32, device=DEV)
        s["refs"][held[held >= 0].long()] = 1
        s["lens"] = lens
        s["K"] = _rand(g, n, bs, c["Hkv"], c["D"]).to(BF)
        s["V"] = _rand(g, n, bs, c["Hkv"], c["D"]).to(BF)
        s["parents"] = _ints(g, 0, P - 1, C)
        s["children"] = (P + torch.randperm(C, generator=g, device=DEV)).to(torch.int32)
        s["rows"] = torch.arange(R, dtype=torch.int32, device=DEV)
        s["first"] = ((lens + bs - 1) // bs).to(torch.int32)  # children: 0, their whole rows
        s["last"] = torch.full((R,), s["tables"].shape[1], dtype=torch.int32, device=DEV)
        s["src"] = torch.empty(C, dtype=torch.int32, device=DEV)
        s["dst"] = torch.empty(C, dtype=torch.int32, device=DEV)
    else:
        B, Hkv, D, T, bs = c["B"], c["Hkv"], c["D"], c["T"], c["block"]
        s["start"] = _ints(g, c["start_lo"], c["start_hi"], B)
        s["n_new"] = _ints(g, (T + 1) // 2, T, B)
        s["tables"], n = _pages(g, (s["start"] + s["n_new"]).tolist(), bs, 8,
                                c["start_hi"] + T)
        s["K"] = _rand(g, n, bs, Hkv, D).to(BF)
        s["V"] = _rand(g, n, bs, Hkv, D).to(BF)
        s["Kn"] = _rand(g, B, Hkv, T, D).to(BF)
        s["Vn"] = _rand(g, B, Hkv, T, D).to(BF)
        # rows kept: a random ascending choice among the rows written
        r = torch.rand(B, T, generator=g, device=DEV)
        t = torch.arange(T, device=DEV)
        r = torch.where(t < s["n_new"][:, None], r, torch.full_like(r, 2.0))
        s["n_keep"] = (s["n_new"] * c["keep"]).ceil().to(torch.int32)
        order = r.argsort(1)
        chosen = torch.where(t < s["n_keep"][:, None], order, torch.full_like(order, T))
        s["keep"] = chosen.sort(1).values.to(torch.int32).contiguous()
    return s


# ---------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------
def _visible(s, Sq, Sk):
    c = s["case"]
    p = c["input_pos"] + torch.arange(Sq, device=DEV)[:, None]
    j = torch.arange(Sk, device=DEV)[None, :]
    return (j <= p) & ((j > p - c["window"]) | (j < c["sinks"]))


def _chunks(s, f):
    """f(batch entry indices, KV head indices) over (batch entry, KV head) pairs, as many
    at once as keep the scores below 2^31 values."""
    c = s["case"]
    Sq, Sk = s["Q"].shape[2], s["K"].shape[2]
    at_once = max(1, 2 ** 31 // max(1, c["Hq"] // c["Hkv"] * Sq * Sk))
    pairs = torch.arange(c["B"] * c["Hkv"], device=DEV).split(at_once)
    outs = [f(p // c["Hkv"], p % c["Hkv"]) for p in pairs]
    return [torch.cat(x) for x in zip(*outs)]


def _scores(s, b, h):
    """(pairs, G, Sq, Sk) scaled scores, -inf where masked, with Q and K in fp32."""
    B, Hq, Sq, D = s["Q"].shape
    Hkv, Sk = s["K"].shape[1:3]
    q = s["Q"].view(B, Hkv, Hq // Hkv, Sq, D)[b, h].float()
    k = s["K"][b, h].float()[:, None]
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"])
    vis = _visible(s, Sq, Sk)[None, None]
    if s["q_len"] is not None:
        vis = vis & (torch.arange(Sk, device=DEV) < s["k_len"][b, None, None, None])
        vis = vis & (torch.arange(Sq, device=DEV)[:, None] < s["q_len"][b, None, None, None])
    return x.masked_fill_(~vis, NEG), q, k


def _plain_fwd(s):
    B, Hq, Sq, D = s["Q"].shape

    def f(b, h):
        x, _, _ = _scores(s, b, h)
        m = x.amax(-1, keepdim=True)
        m = torch.where(m == NEG, torch.zeros_like(m), m)
        p = x.sub_(m).exp_()
        l = p.sum(-1, keepdim=True)
        o = (p @ s["V"][b, h].float()[:, None]) / l.clamp_min(1e-30)
        return o.to(BF), (m + l.log()).squeeze(-1)

    O, L = _chunks(s, f)
    return O.reshape(B, Hq, Sq, D), L.reshape(B, Hq, Sq)


def _plain_bwd(s):
    B, Hq, Sq, D = s["Q"].shape
    Hkv, Sk = s["K"].shape[1:3]
    G = Hq // Hkv

    def f(b, h):
        x, q, k = _scores(s, b, h)
        lse = s["LSE"].view(B, Hkv, G, Sq)[b, h]
        p = x.sub_(torch.where(lse == NEG, torch.zeros_like(lse), lse)[..., None]).exp_()
        do = s["dO"].view(B, Hkv, G, Sq, D)[b, h].float()
        delta = (do * s["O"].view(B, Hkv, G, Sq, D)[b, h].float()).sum(-1, keepdim=True)
        dv = (p.transpose(-1, -2) @ do).sum(1)
        ds = (do @ s["V"][b, h].float()[:, None].transpose(-1, -2)).sub_(delta).mul_(p)
        dq = (ds @ k).mul_(s["scale"])
        dk = (ds.transpose(-1, -2) @ q).sum(1).mul_(s["scale"])
        return dq.to(BF), dk.to(BF), dv.to(BF)

    dQ, dK, dV = _chunks(s, f)
    return dQ.reshape(B, Hq, Sq, D), dK.reshape(B, Hkv, Sk, D), dV.reshape(B, Hkv, Sk, D)


def _rows_of(tables, pos, block):
    """Cache row of position pos (B, n) of each sequence; -1 where it has no page."""
    page = tables.long().gather(1, (pos // block).clamp(0, tables.shape[1] - 1))
    ok = (page >= 0) & (pos >= 0) & (pos // block < tables.shape[1])
    return torch.where(ok, page * block + pos % block, torch.full_like(page, -1))


def _plain_sink_decode(s):
    c = s["case"]
    B, Hq, D = s["Q"].shape
    Hkv = c["Hkv"]
    n = s["len"].long()[:, None]
    first = torch.arange(c["sinks"], device=DEV).expand(B, -1)
    last = n - min(c["window"], c["cap"]) + torch.arange(min(c["window"], c["cap"]), device=DEV)
    pos = torch.cat([first, last], 1)
    vis = torch.cat([first < n, last >= c["sinks"]], 1) & (pos >= 0)
    if c["block"]:
        rows = _rows_of(s["tables"], pos, c["block"]).clamp_min(0)
        K = s["K"].view(-1, Hkv, D)[rows].float().transpose(1, 2)
        V = s["V"].view(-1, Hkv, D)[rows].float().transpose(1, 2)
    else:
        at = pos.clamp(0, c["cap"] - 1)[:, None, :, None].expand(B, Hkv, -1, D)
        K, V = s["K"].gather(2, at).float(), s["V"].gather(2, at).float()
    x = s["Q"].view(B, Hkv, Hq // Hkv, D).float() @ K.transpose(-1, -2) / math.sqrt(D)
    x = x.masked_fill(~vis[:, None, None], NEG)
    m = x.amax(-1, keepdim=True)
    p = (x - torch.where(m == NEG, torch.zeros_like(m), m)).exp()
    return ((p @ V) / p.sum(-1, keepdim=True).clamp_min(1e-30)).reshape(B, Hq, D).to(BF)


def _ancestors(parents):
    """(B, T, T) truth: draft j is draft i or one of its ancestors."""
    T = parents.shape[1]
    j = torch.arange(T, device=DEV)
    m = ((parents[..., None] == j) | (j[:, None] == j)).float()
    for _ in range(max(1, (T - 1).bit_length())):  # paths of length 1, 2, 4, ...
        m = ((m @ m) > 0).float()
    return m > 0


def _plain_tree(s):
    c = s["case"]
    B, Hq, T, D = s["Q"].shape
    Hkv = c["Hkv"]
    n = s["tables"].shape[1] * c["block"]
    pos = torch.arange(n, device=DEV).expand(B, -1)
    rows = _rows_of(s["tables"], pos, c["block"]).clamp_min(0)
    ctx, drafts = s["ctx"].long()[:, None], s["drafts"].long()[:, None]
    d = pos - ctx  # draft of each key, negative in the context
    anc = _ancestors(s["parents"]).gather(2, d.clamp(0, T - 1)[:, None].expand(B, T, n))
    vis = (d < 0)[:, None] | (anc & (d < drafts)[:, None])
    vis = vis & (torch.arange(T, device=DEV) < drafts)[..., None]
    q = s["Q"].view(B, Hkv, Hq // Hkv, T, D).float().flatten(2, 3)
    K = s["K"].view(-1, Hkv, D)[rows].float().transpose(1, 2)
    x = (q @ K.transpose(-1, -2)).div_(math.sqrt(D)).view(B, Hkv, Hq // Hkv, T, n)
    del K
    x.masked_fill_(~vis[:, None, None], NEG)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(m == NEG, torch.zeros_like(m), m)).exp_()
    l = p.sum(-1, keepdim=True).clamp_min(1e-30)
    V = s["V"].view(-1, Hkv, D)[rows].float().transpose(1, 2)
    o = (p.flatten(2, 3) @ V).view(B, Hkv, Hq // Hkv, T, D) / l
    return o.reshape(B, Hq, T, D).to(BF)


def _next_free(refs, k):
    """Number of the k-th free page (k counts from 0), in increasing order."""
    seen = (refs == 0).int().cumsum(0, dtype=torch.int32)
    return torch.searchsorted(seen, (k + 1).to(torch.int32)).to(torch.int32)


def _plain_fork(s):
    bs = s["case"]["block"]
    tables, refs, lens = s["tables"], s["refs"], s["lens"]
    R, width = tables.shape
    k = torch.arange(width, device=DEV)
    ones = torch.ones((), dtype=torch.int32, device=DEV)
    trash = refs.shape[0]  # pages counted nowhere
    count = torch.cat([refs, refs.new_zeros(1)])
    # give back entries [first, last) of every row
    out = (k >= s["first"][:, None]) & (k < s["last"][:, None])
    gone = torch.where(out & (tables >= 0), tables, trash).long().flatten()
    count.index_add_(0, gone, (-ones).expand(gone.shape[0]))
    tables.masked_fill_(out, -1)
    # fork: whole pages shared, the part-filled one copied to a fresh page
    par, chi = s["parents"].long(), s["children"].long()
    lens[chi] = lens[par]
    full = (lens[par] // bs)[:, None]
    row = torch.where(k < full, tables[par], -1)
    shared = torch.where(row >= 0, row, trash).long().flatten()
    count.index_add_(0, shared, ones.expand(shared.shape[0]))
    part = lens[par] % bs > 0
    fresh = _next_free(count[:trash], part.int().cumsum(0) - 1)
    src = torch.where(part, tables[par].gather(1, full.long()).squeeze(1), -1)
    dst = torch.where(part, fresh, -1)
    row = torch.where((k == full) & part[:, None], dst[:, None], row)
    tables[chi] = row
    count.index_add_(0, torch.where(part, dst, trash).long(), ones.expand(dst.shape[0]))
    # extend every row to its length and `grow` more tokens
    to = (lens + s["case"]["grow"] + bs - 1) // bs
    need = (k >= (lens // bs)[:, None]) & (k < to[:, None]) & (tables < 0)
    rank = need.flatten().int().cumsum(0).view(R, width) - 1
    new = _next_free(count[:trash], rank.clamp_min(0).flatten()).view(R, width)
    tables.copy_(torch.where(need, new, tables))
    count.index_add_(0, torch.where(need, new, trash).long().flatten(), ones.expand(R * width))
    refs.copy_(count[:trash])
    # copy the part-filled pages
    s["src"].copy_(src)
    s["dst"].copy_(dst)
    one = part.int().argmax()  # a child without such a page repeats another's copy
    at = torch.where(part, src, src[one]).clamp_min(0).long()
    to_ = torch.where(part, dst, dst[one]).clamp_min(0).long()
    for pool in (s["K"], s["V"]):
        pool[to_] = pool[at]
    return tables, refs, lens, s["src"], s["dst"], s["K"], s["V"]


def _plain_commit(s):
    c = s["case"]
    B, T, D, Hkv, bs = c["B"], c["T"], c["D"], c["Hkv"], c["block"]
    t = torch.arange(T, device=DEV).expand(B, -1)
    start = s["start"].long()[:, None]
    rows = _rows_of(s["tables"], start + t, bs)
    ok = (t < s["n_new"][:, None]) & (rows >= 0)
    src = _rows_of(s["tables"], start + s["keep"].long(), bs).clamp_min(0)
    moved = t < s["n_keep"][:, None]
    n = s["K"].shape[0] * bs  # a row that is never read takes what is not written
    for pool, new in ((s["K"], s["Kn"]), (s["V"], s["Vn"])):
        flat = pool.view(n, Hkv, D)
        wide = torch.cat([flat, flat.new_zeros(1, Hkv, D)])
        wide[torch.where(ok, rows, n)] = new.transpose(1, 2)
        kept = wide[src]
        wide[torch.where(moved, rows, n)] = kept
        flat.copy_(wide[:n])
    return s["K"], s["V"]


# ---------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------
def run(s):
    c, op = s["case"], s["case"]["op"]
    if not own:
        if op == "sink_fwd":
            return _plain_fwd(s)
        if op == "sink_bwd":
            return _plain_bwd(s)
        if op == "sink_decode":
            return _plain_sink_decode(s)
        return {"tree": _plain_tree, "fork": _plain_fork, "commit": _plain_commit}[op](s)
    from gqa_attention_flash_b200 import binding
    if op == "sink_fwd":
        binding.attn_fwd_sinks(s["O"], s["Q"], s["K"], s["V"], s["LSE"], s["scale"], c["window"],
                               c["sinks"], c["input_pos"], s["k_len"], s["q_len"])
        return s["O"], s["LSE"]
    if op == "sink_bwd":
        binding.attn_bwd_sinks(s["dQ"], s["dK"], s["dV"], s["dO"], s["Q"], s["K"], s["V"], s["O"],
                               s["LSE"], s["scale"], c["window"], c["sinks"], c["input_pos"],
                               s["k_len"], s["q_len"])
        return s["dQ"], s["dK"], s["dV"]
    if op == "sink_decode":
        if c["block"]:
            binding.attn_decode_paged_sinks(s["O"], s["Q"], s["K"], s["V"], s["tables"], s["len"],
                                            c["window"], c["sinks"])
        else:
            binding.attn_decode_sinks(s["O"], s["Q"], s["K"], s["V"], s["len"], c["window"],
                                      c["sinks"])
        return s["O"]
    if op == "tree":
        binding.attn_tree_paged(s["O"], s["Q"], s["K"], s["V"], s["tables"], s["ctx"],
                                s["parents"], s["drafts"])
        return s["O"]
    if op == "fork":
        bs = c["block"]
        binding.cache_free(s["tables"], s["refs"], s["rows"], s["first"], s["last"])
        binding.cache_fork(s["tables"], s["refs"], s["lens"], s["parents"], s["children"],
                           s["src"], s["dst"], bs)
        binding.cache_extend(s["tables"], s["refs"], s["lens"], s["lens"] + c["grow"], bs)
        binding.cache_copy_blocks(s["K"], s["V"], s["src"], s["dst"])
        return s["tables"], s["refs"], s["lens"], s["src"], s["dst"], s["K"], s["V"]
    binding.cache_append(s["K"], s["V"], s["Kn"], s["Vn"], s["tables"], s["start"], s["n_new"])
    binding.cache_compact(s["K"], s["V"], s["tables"], s["start"], s["keep"], s["n_keep"])
    return s["K"], s["V"]


# ---------------------------------------------------------------------------------
# bytes and operations that a pass cannot do without
# ---------------------------------------------------------------------------------
def _pairs(Sq, pos, window, sinks):
    """Visible (query, key) pairs of one head without lengths."""
    p = torch.arange(Sq, dtype=torch.int64) + pos
    lo = (p - window + 1).clamp_min(0)
    return int((p + 1 - lo).sum() + torch.minimum(lo, torch.full_like(lo, sinks)).sum())


def work(case):
    """Ragged lengths count at the middle of their range."""
    c, op = case, case["op"]
    if op in ("sink_fwd", "sink_bwd"):
        Sq = int(c["Sq"] * 0.75) if c["ragged"] else c["Sq"]
        Sq = max(1, Sq)
        pairs = c["B"] * c["Hq"] * _pairs(Sq, c["input_pos"], c["window"], c["sinks"])
        q = 2 * c["B"] * c["Hq"] * Sq * c["D"]
        k = 2 * c["B"] * c["Hkv"] * (Sq + c["input_pos"]) * c["D"]
        lse = 4 * c["B"] * c["Hq"] * Sq
        if op == "sink_fwd":
            return {"bytes": 2 * q + 2 * k + lse, "flops": 4 * c["D"] * pairs}
        return {"bytes": 4 * q + 4 * k + lse, "flops": 10 * c["D"] * pairs}
    if op == "sink_decode":
        keys = min((c["lo"] + c["cap"]) // 2, c["window"] + c["sinks"])
        return {"bytes": 4 * c["B"] * c["Hkv"] * keys * c["D"] + 4 * c["B"] * c["Hq"] * c["D"],
                "flops": 4 * c["B"] * c["Hq"] * keys * c["D"]}
    if op == "tree":
        T = max(1, int(0.75 * c["T"]))
        keys = (c["ctx_lo"] + c["ctx_hi"]) // 2 + T
        return {"bytes": 4 * c["B"] * c["Hkv"] * keys * c["D"] + 4 * c["B"] * c["Hq"] * T * c["D"],
                "flops": 4 * c["B"] * c["Hq"] * T * keys * c["D"]}
    if op == "fork":
        bs, mid = c["block"], (c["lo"] + c["hi"]) // 2
        page = 4 * bs * c["Hkv"] * c["D"]  # K and V of one page
        entries = c["children"] * (mid // bs)
        new = c["children"] + (c["parents"] + c["children"]) * (c["grow"] // bs)
        # a shared entry: read, written, its count read and written; a page copied
        return {"bytes": 16 * entries + 12 * new + 2 * c["children"] * page, "flops": 0}
    row = 4 * c["Hkv"] * c["D"]  # K and V of one token
    n = c["B"] * max(1, int(0.75 * c["T"]))
    return {"bytes": 2 * n * row + 2 * int(n * c["keep"]) * row, "flops": 0}


# ---------------------------------------------------------------------------------
# the definitions in fp64
# ---------------------------------------------------------------------------------
def _exact_rows(q, k, v, vis):
    """softmax(q k^T / sqrt(D)) v and its log-sum-exp on the visible pairs (fp64)."""
    x = torch.where(vis, q @ k.mT / math.sqrt(q.shape[-1]), NEG)
    lse = x.logsumexp(-1)
    p = torch.where(vis, (x - lse[..., None]).exp(), 0.0)
    return p @ v, lse, p


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op in ("sink_fwd", "sink_bwd"):
        B, Hq, Sq, D = s["Q"].shape
        Hkv, Sk = s["K"].shape[1:3]
        O = torch.zeros(B, Hq, Sq, D, dtype=torch.float64, device=DEV)
        L = torch.full((B, Hq, Sq), NEG, dtype=torch.float64, device=DEV)
        dQ, dK, dV = torch.zeros_like(O), *(torch.zeros(B, Hkv, Sk, D, dtype=torch.float64,
                                                       device=DEV) for _ in range(2))
        for b in range(B):
            nq = int(s["q_len"][b]) if s["q_len"] is not None else Sq
            nk = int(s["k_len"][b]) if s["k_len"] is not None else Sk
            i = torch.arange(c["input_pos"], c["input_pos"] + nq, device=DEV)[:, None]
            j = torch.arange(nk, device=DEV)[None]
            vis = (i >= j) & ~((i - j >= c["window"]) & (j >= c["sinks"]))
            for h in range(Hq):
                kv = h // (Hq // Hkv)
                q, k, v = s["Q"][b, h, :nq].double(), s["K"][b, kv, :nk].double(), \
                    s["V"][b, kv, :nk].double()
                if op == "sink_fwd":
                    O[b, h, :nq], L[b, h, :nq], _ = _exact_rows(q, k, v, vis)
                    continue
                do, o = s["dO"][b, h, :nq].double(), s["O"][b, h, :nq].double()
                x = q @ k.mT / math.sqrt(D) - s["LSE"][b, h, :nq, None].double()
                p = torch.where(vis, x, NEG).exp()
                ds = p * (do @ v.mT - (do * o).sum(-1, keepdim=True)) / math.sqrt(D)
                dQ[b, h, :nq] = ds @ k
                dK[b, kv, :nk] += ds.mT @ q
                dV[b, kv, :nk] += p.mT @ do
        return (O, L) if op == "sink_fwd" else (dQ, dK, dV)
    if op in ("sink_decode", "tree"):
        O = torch.zeros(s["Q"].shape, dtype=torch.float64, device=DEV)
        Hq, Hkv = c["Hq"], c["Hkv"]
        for b in range(c["B"]):
            n = int(s["len"][b]) if op == "sink_decode" else int(s["ctx"][b] + s["drafts"][b])
            at = torch.arange(n, device=DEV)
            if op == "sink_decode":
                at = at[(at >= n - c["window"]) | (at < c["sinks"])]
            if at.numel() == 0:
                continue
            if c["block"]:
                row = s["tables"][b].long()[at // c["block"]], at % c["block"]
                k, v = s["K"][row].double().transpose(0, 1), s["V"][row].double().transpose(0, 1)
            else:
                k, v = s["K"][b][:, at].double(), s["V"][b][:, at].double()
            if op == "sink_decode":
                q = s["Q"][b].double().view(Hkv, Hq // Hkv, -1)
                O[b] = _exact_rows(q, k, v, torch.ones((), dtype=torch.bool,
                                                       device=DEV))[0].flatten(0, 1)
                continue
            ctx, drafts, par = int(s["ctx"][b]), int(s["drafts"][b]), s["parents"][b].tolist()
            vis = torch.zeros(drafts, n, dtype=torch.bool)
            vis[:, :ctx] = True
            for i in range(drafts):
                a = i
                while a >= 0:
                    vis[i, ctx + a] = True
                    a = par[a]
            q = s["Q"][b, :, :drafts].double().view(Hkv, -1, c["D"])
            o = _exact_rows(q, k, v, vis.to(DEV).repeat(Hq // Hkv, 1))[0]
            O[b, :, :drafts] = o.view(Hq, drafts, c["D"])
        return O
    if op == "fork":
        # whole numbers are compared as such; the pools are the prepared ones with the
        # part-filled pages copied to the lowest free pages, child by child
        refs, tables, lens = s["refs"].tolist(), s["tables"].tolist(), s["lens"].tolist()
        free = iter([p for p, n in enumerate(refs) if n == 0])
        K, V = s["K"].double(), s["V"].double()
        for p in s["parents"].tolist():
            if lens[p] % c["block"]:
                to, at = next(free), tables[p][lens[p] // c["block"]]
                K[to], V[to] = K[at].clone(), V[at].clone()
        return None, None, None, None, None, K, V
    K, V = s["K"].double(), s["V"].double()
    for b in range(c["B"]):
        n, k, first = int(s["n_new"][b]), int(s["n_keep"][b]), int(s["start"][b])
        at = torch.arange(first, first + n, device=DEV)
        row = s["tables"][b].long()[at // c["block"]], at % c["block"]
        keep = s["keep"][b, :k].long()
        for pool, new in ((K, s["Kn"]), (V, s["Vn"])):
            new = new[b, :, :n].transpose(0, 1).double()
            pool[row] = new
            pool[row[0][:k], row[1][:k]] = new[keep]
    return K, V
