"""Sliding window with sinks on the GPU (attn_fwd_sinks, attn_bwd_sinks, attn_decode_sinks,
attn_decode_paged_sinks) against the definition in fp64.

Tolerances follow from the roundings, u = 2^-8 being half a step of bf16 relative to the
value: the kernels round each weight p (forward, dV) or p (dP - delta) (dQ, dK) to bf16
before its product, and the result once more, so
    |dO| <= u (sum_j p_j |v_j| + |O|),  |d dV| <= u (sum_i p_i |dO_i| + |dV|),
    |d dQ| <= u (scale sum_j |dS_j| |k_j| + |dQ|), and dK likewise.
Everything else is fp32: sums of n <= 2^11 terms lose at most n 2^-24 = 2^-13 of the sum
of their magnitudes, which the bounds add with the magnitudes before any cancellation."""
import math

import pytest
import torch

from gqa_attention_flash_b200 import binding
from gqa_attention_flash_b200 import workloads as W

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
F32 = 2.0 ** -13
NEG = float("-inf")
BF = torch.bfloat16


def visible(Sq, Sk, window, sinks, input_pos, device="cuda"):
    p = input_pos + torch.arange(Sq, device=device)[:, None]
    j = torch.arange(Sk, device=device)[None]
    return (j <= p) & ((j > p - window) | (j < sinks))


def lengths_mask(B, Sq, Sk, k_len, q_len):
    m = torch.ones(B, Sq, Sk, dtype=torch.bool, device="cuda")
    if k_len is not None:
        m &= torch.arange(Sk, device="cuda") < k_len[:, None, None]
    if q_len is not None:
        m &= torch.arange(Sq, device="cuda")[:, None] < q_len[:, None, None]
    return m


def ref_fwd(Q, K, V, vis, scale):
    """O, LSE, P and sum p |v| in fp64; vis (B, 1, Sq, Sk)."""
    G = Q.shape[1] // K.shape[1]
    q, k, v = (x.double() for x in (Q, K.repeat_interleave(G, 1), V.repeat_interleave(G, 1)))
    s = torch.where(vis, q @ k.mT * scale, NEG)
    lse = torch.logsumexp(s, -1)
    p = torch.where(vis, (s - torch.where(lse == NEG, 0.0, lse)[..., None]).exp(), 0.0)
    return p @ v, lse, p, p @ v.abs()


def check(got, want, bound, what):
    bad = (got.double() - want).abs() > bound
    assert torch.isfinite(got.float()).all(), f"{what}: not finite"
    assert not bad.any(), (what, float(((got.double() - want).abs() - bound).max()), int(bad.sum()))


def inputs(seed, B, Hq, Hkv, Sq, Sk, D):
    return [x.cuda() for x in W.random_prefill(seed, B, Hq, Hkv, Sq, Sk, D)]


CASES = [
    # B, Hq, Hkv, Sq, input_pos, D, window, sinks, q_len, k_len
    (1, 2, 1, 1, 0, 64, 1, 0, None, None),             # one token that sees itself
    (1, 2, 1, 1, 300, 128, 5, 3, None, None),          # one token far behind the sinks
    (1, 2, 2, 129, 0, 64, 1, 1, None, None),
    (2, 4, 2, 200, 0, 128, 17, 4, None, None),
    (1, 4, 1, 700, 0, 128, 130, 4, None, None),        # sink tile and window tiles apart
    (1, 2, 1, 700, 0, 64, 100, 129, None, None),       # sinks across two tiles
    (1, 2, 1, 600, 0, 64, 100, 300, None, None),       # sinks beyond the windows' start
    (1, 2, 1, 600, 0, 128, 64, 5000, None, None),      # more sinks than keys: causal
    (1, 2, 1, 500, 0, 128, 5000, 2, None, None),       # window wider than the keys: causal
    (1, 2, 1, 500, 0, 128, 2 ** 31 - 1, 2 ** 31 - 1, None, None),
    (1, 2, 1, 257, 1000, 128, 128, 4, None, None),     # chunk of a longer prompt
    (2, 2, 1, 385, 640, 64, 256, 130, None, None),
    (3, 4, 2, 400, 0, 64, 50, 7, (400, 1, 0), (400, 1, 0)),
    (3, 2, 1, 640, 0, 128, 70, 6, (640, 640, 333), (640, 3, 100)),  # keys end before windows
    (2, 2, 1, 300, 500, 128, 90, 4, (300, 17), (800, 517)),
    (2, 32, 2, 260, 0, 128, 33, 4, None, None),
    (1, 3, 3, 1030, 0, 64, 127, 128, None, None),
    (1, 2, 1, 512, 0, 128, 128, 128, None, None),
    (1, 32, 1, 1300, 0, 64, 64, 4, None, None),        # a sink tile of many items, split
    (4, 16, 8, 900, 0, 128, 250, 4, (900, 899, 1, 450), (900, 899, 1, 450)),
]


def case_inputs(c):
    B, Hq, Hkv, Sq, pos, D, window, sinks, ql, kl = c
    Sk = Sq + pos
    t = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ql, kl = t(ql), t(kl)
    vis = (visible(Sq, Sk, window, sinks, pos) & lengths_mask(B, Sq, Sk, kl, ql))[:, None]
    return inputs(sum(c[:8]) % 1000, B, Hq, Hkv, Sq, Sk, D), ql, kl, vis


@pytest.mark.parametrize("c", CASES, ids=[str(c) for c in CASES])
def test_forward(c):
    B, Hq, Hkv, Sq, pos, D, window, sinks, _, _ = c
    (Q, K, V), ql, kl, vis = case_inputs(c)
    O = torch.full_like(Q, float("nan"))
    L = torch.full((B, Hq, Sq), float("nan"), device="cuda")
    binding.attn_fwd_sinks(O, Q, K, V, L, D ** -0.5, window, sinks, pos, kl, ql)
    assert binding.last_device_status() == 0
    want, lse, _, mag = ref_fwd(Q, K, V, vis, D ** -0.5)
    check(O, want, U * (mag + want.abs()) + F32 * mag, "O")
    empty = lse == NEG
    assert torch.equal(L == NEG, empty) and not L.isnan().any()
    assert torch.all(O[empty] == 0)
    # scores: D products summed in fp32, then the sum of the weights
    assert float((L.double() - lse)[~empty].abs().max() if (~empty).any() else 0) <= 2e-5


@pytest.mark.parametrize("c", CASES, ids=[str(c) for c in CASES])
def test_backward(c):
    B, Hq, Hkv, Sq, pos, D, window, sinks, _, _ = c
    (Q, K, V), ql, kl, vis = case_inputs(c)
    G, scale = Hq // Hkv, D ** -0.5
    dO = inputs(5, B, Hq, Hkv, Sq, 1, D)[0]
    O, L = torch.empty_like(Q), torch.empty((B, Hq, Sq), device="cuda")
    binding.attn_fwd_sinks(O, Q, K, V, L, scale, window, sinks, pos, kl, ql)
    g = [torch.full_like(x, float("nan")) for x in (Q, K, V)]
    binding.attn_bwd_sinks(*g, dO, Q, K, V, O, L, scale, window, sinks, pos, kl, ql)
    assert binding.last_device_status() == 0
    # the gradients' formulas, with the forward's saved O and LSE as they are
    q, do = Q.double(), dO.double()
    k, v = (x.double().repeat_interleave(G, 1) for x in (K, V))
    lse = torch.where(L == NEG, 0.0, L.double())[..., None]
    p = torch.where(vis, (q @ k.mT * scale - lse).exp(), 0.0)
    delta = (do * O.double()).sum(-1, keepdim=True)
    ds = p * (do @ v.mT - delta)
    raw = p * (do.abs() @ v.abs().mT + (do * O.double()).abs().sum(-1, keepdim=True))
    fold = lambda x: x.view(B, Hkv, G, *x.shape[2:]).sum(2)  # noqa: E731
    want = ds @ k * scale, fold(ds.mT @ q) * scale, fold(p.mT @ do)
    mag = ds.abs() @ k.abs() * scale, fold(ds.abs().mT @ q.abs()) * scale, fold(p.mT @ do.abs())
    fp32 = raw @ k.abs() * scale, fold(raw.mT @ q.abs()) * scale, mag[2]
    for name, x, w, m, f in zip(("dQ", "dK", "dV"), g, want, mag, fp32):
        check(x, w, U * (m + w.abs()) + F32 * f, name)
    for b in range(B):  # gradients of padding are zero
        if ql is not None:
            assert torch.all(g[0][b, :, int(ql[b]):] == 0)
        if kl is not None:
            assert torch.all(g[1][b, :, int(kl[b]):] == 0) and torch.all(g[2][b, :, int(kl[b]):] == 0)


def test_backward_against_differences():
    """Directional derivatives of sum(O dO) in fp64 against the kernels' gradients."""
    B, Hq, Hkv, S, D, window, sinks = 1, 2, 1, 300, 64, 40, 5
    Q, K, V = inputs(9, B, Hq, Hkv, S, S, D)
    dO = inputs(10, B, Hq, Hkv, S, 1, D)[0]
    vis = visible(S, S, window, sinks, 0)[None, None]
    O, L = torch.empty_like(Q), torch.empty((B, Hq, S), device="cuda")
    binding.attn_fwd_sinks(O, Q, K, V, L, 0.125, window, sinks)
    g = [torch.empty_like(x) for x in (Q, K, V)]
    binding.attn_bwd_sinks(*g, dO, Q, K, V, O, L, 0.125, window, sinks)
    f = lambda q, k, v: float((ref_fwd(q, k, v, vis, 0.125)[0] * dO.double()).sum())  # noqa: E731
    x = [t.double() for t in (Q, K, V)]
    for i in range(3):
        d = torch.randn(x[i].shape, generator=torch.Generator().manual_seed(i)).double().cuda()
        h = 1e-5
        up, dn = list(x), list(x)
        up[i], dn[i] = x[i] + h * d, x[i] - h * d
        slope = (f(*up) - f(*dn)) / (2 * h)
        got = float((g[i].double() * d).sum())
        # the kernel's roundings, u relative to each weight and each gradient: both sums
        # have random signs, so 4 standard deviations of u |g| |d| bound them
        bound = 4 * 3 * U * float((g[i].double() * d).norm()) + 1e-3
        assert abs(got - slope) <= bound, (i, got, slope, bound)


def test_no_sinks_is_the_window_and_wide_window_is_causal():
    Q, K, V = inputs(3, 2, 4, 2, 500, 500, 128)
    outs = []
    for f in (lambda O, L: binding.attn_fwd(O, Q, K, V, L, 0.1, True, window=77),
              lambda O, L: binding.attn_fwd_sinks(O, Q, K, V, L, 0.1, 77, 0),
              lambda O, L: binding.attn_fwd(O, Q, K, V, L, 0.1, True),
              lambda O, L: binding.attn_fwd_sinks(O, Q, K, V, L, 0.1, 500, 9)):
        O, L = torch.empty_like(Q), torch.empty((2, 4, 500), device="cuda")
        f(O, L)
        outs.append((O, L))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.equal(outs[2][0], outs[3][0]) and torch.equal(outs[2][1], outs[3][1])


def test_padding_rows_hold_anything():
    """Rows of K and V past k_lengths and of Q past q_lengths hold NaN."""
    (Q, K, V), _, _, _ = case_inputs(CASES[12])
    B, Hq, Sq = Q.shape[:3]
    ql = torch.tensor([400, 130, 5], dtype=torch.int32, device="cuda")
    kl = torch.tensor([333, 130, 5], dtype=torch.int32, device="cuda")
    clean = torch.empty_like(Q)
    L = torch.empty((B, Hq, Sq), device="cuda")
    binding.attn_fwd_sinks(clean, Q, K, V, L, 0.125, 50, 7, 0, kl, ql)
    for b in range(B):
        Q[b, :, int(ql[b]):] = float("nan")
        K[b, :, int(kl[b]):] = float("nan")
        V[b, :, int(kl[b]):] = float("inf")
    O = torch.empty_like(Q)
    binding.attn_fwd_sinks(O, Q, K, V, L, 0.125, 50, 7, 0, kl, ql)
    assert torch.equal(O, clean)


# ---------------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------------
DECODE = [
    # B, Hq, Hkv, D, cap, lengths, window, sinks, n_splits, block (0 = contiguous)
    (1, 2, 1, 64, 1, [1], 1, 0, 0, 0),
    (4, 8, 2, 128, 300, [0, 1, 64, 300], 1, 0, 0, 0),
    (4, 8, 2, 128, 300, [0, 3, 65, 300], 10, 4, 3, 0),
    (3, 16, 1, 64, 2000, [2000, 1999, 130], 500, 70, 0, 0),
    (3, 4, 4, 128, 2000, [2000, 700, 64], 64, 64, 64, 0),
    (2, 8, 8, 128, 1000, [1000, 900], 5000, 3, 0, 0),
    (2, 8, 8, 128, 1000, [1000, 900], 100, 5000, 7, 0),
    (1, 32, 8, 128, 8192, [8100], 1024, 4, 0, 0),
    (5, 8, 2, 128, 0, [0, 1, 15, 16, 17], 4, 2, 0, 16),
    (4, 32, 8, 128, 0, [3000, 517, 1025, 64], 300, 5, 0, 16),
    (3, 6, 2, 64, 0, [700, 65, 129], 63, 9, 5, 8),
    (2, 4, 4, 64, 0, [1000, 640], 100, 1, 0, 64),
    (2, 8, 1, 128, 0, [2048, 257], 130, 33, 0, 256),
    (2, 10, 2, 128, 0, [900, 333], 2 ** 31 - 1, 2 ** 31 - 1, 0, 32),
    (2, 16, 1, 128, 1500, [1500, 40], 700, 9, 8, 0),
    (3, 32, 2, 128, 0, [1500, 64, 700], 640, 65, 6, 16),
    (1, 4, 2, 64, 0, [5000], 300, 4, 9, 4096),
    (40, 8, 8, 64, 0, [17 * k for k in range(40)], 100, 4, 0, 8),
]


def decode_case(c, poison):
    """Inputs of a decode case; rows without a visible key hold ``poison``, pages without
    one are not in the table."""
    B, Hq, Hkv, D, cap, lens, window, sinks, n_splits, block = c
    g = torch.Generator().manual_seed(B + D + window % 1000)
    Q = torch.randn(B, Hq, D, generator=g).to(BF).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    most = max(cap, max(lens))
    K = torch.randn(B, Hkv, most, D, generator=g).to(BF).cuda()
    V = torch.randn(B, Hkv, most, D, generator=g).to(BF).cuda()
    j = torch.arange(most, device="cuda")
    vis = (j < n[:, None]) & ((j >= n[:, None].long() - window) | (j < sinks))
    hide = ~vis[:, None, :, None]
    K, V = K.masked_fill(hide, poison), V.masked_fill(hide, poison)
    if not block:
        return Q, K, V, n, vis, None, K, V
    tables, nblk = W.paged_layout(lens, block, 3, 1)
    Kp = torch.full((nblk, block, Hkv, D), poison, dtype=BF, device="cuda")
    Vp = Kp.clone()
    W.fill_paged_cache(Kp, Vp, tables, lambda b: (K[b, :, :lens[b]], V[b, :, :lens[b]]))
    for b in range(B):
        for k in range(tables.shape[1]):
            if not vis[b, k * block:(k + 1) * block].any():
                tables[b, k] = -1
    # page slots past the length
    for b, ln in enumerate(lens):
        if ln % block:
            page = int(tables[b, ln // block])
            Kp[page, ln % block:] = poison
            Vp[page, ln % block:] = poison
    return Q, K, V, n, vis, tables.cuda(), Kp, Vp


@pytest.mark.parametrize("poison", [0.0, float("nan"), float("inf")])
@pytest.mark.parametrize("c", DECODE, ids=[str(c) for c in DECODE])
def test_decode(c, poison):
    B, Hq, Hkv, D, cap, lens, window, sinks, n_splits, block = c
    Q, K, V, n, vis, tables, Kc, Vc = decode_case(c, poison)
    O = torch.full_like(Q, float("nan"))
    if block:
        binding.attn_decode_paged_sinks(O, Q, Kc, Vc, tables, n, window, sinks, n_splits)
    else:
        binding.attn_decode_sinks(O, Q, Kc, Vc, n, window, sinks, n_splits)
    assert binding.last_device_status() == 0
    hide = ~vis[:, None, :, None]
    K, V = K.masked_fill(hide, 0.0), V.masked_fill(hide, 0.0)
    want, lse, _, mag = ref_fwd(Q[:, :, None], K, V, vis[:, None, None], D ** -0.5)
    check(O, want[:, :, 0], (U * (mag + want.abs()) + F32 * mag)[:, :, 0], "O")
    assert torch.all(O[(lse == NEG)[..., 0]] == 0)


def test_decode_is_the_last_row_of_the_forward():
    B, Hq, Hkv, S, D = 2, 8, 2, 900, 128
    Q, K, V = inputs(21, B, Hq, Hkv, S, S, D)
    O, L = torch.empty_like(Q), torch.empty((B, Hq, S), device="cuda")
    binding.attn_fwd_sinks(O, Q, K, V, L, D ** -0.5, 200, 4)
    last = torch.empty((B, Hq, D), dtype=BF, device="cuda")
    n = torch.full((B,), S, dtype=torch.int32, device="cuda")
    binding.attn_decode_sinks(last, Q[:, :, -1].contiguous(), K, V, n, 200, 4)
    _, _, _, mag = ref_fwd(Q[:, :, -1:], K, V, visible(S, S, 200, 4, 0)[-1:][None, None], D ** -0.5)
    # each of the two within the forward's bound of the same exact value
    bound = 2 * (U * (mag[:, :, 0] + last.double().abs() * 1.01) + F32 * mag[:, :, 0])
    check(last, O[:, :, -1].double(), bound, "last row")


def test_lengths_out_of_range_are_flagged_and_clamped():
    Q, K, V = inputs(4, 2, 4, 2, 100, 100, 64)
    n = torch.tensor([100, 150], dtype=torch.int32, device="cuda")
    q = Q[:, :, 0].contiguous()
    O, P = torch.empty_like(q), torch.empty_like(q)
    binding.attn_decode_sinks(O, q, K, V, n, 30, 4)
    assert binding.STATUS[binding.last_device_status()] == "ATTN_ERR_DEVICE_BOUNDS"
    binding.attn_decode_sinks(P, q, K, V, n.clamp(max=100), 30, 4)
    assert binding.last_device_status() == 0 and torch.equal(O, P)


@pytest.mark.parametrize("where", ["stream", "graph"])
def test_other_stream_and_graph(where):
    """Forward, backward and decode on a stream of their own, and replayed from a graph on
    new inputs, give what the plain calls give."""
    B, Hq, Hkv, S, D, w, sk = 2, 4, 2, 333, 128, 60, 4
    Q, K, V = inputs(31, B, Hq, Hkv, S, S, D)
    dO = inputs(32, B, Hq, Hkv, S, 1, D)[0]
    n = torch.tensor([333, 200], dtype=torch.int32, device="cuda")

    def step(o):
        binding.attn_fwd_sinks(o["O"], Q, K, V, o["L"], D ** -0.5, w, sk)
        binding.attn_bwd_sinks(o["dQ"], o["dK"], o["dV"], dO, Q, K, V, o["O"], o["L"], D ** -0.5, w, sk)
        binding.attn_decode_sinks(o["d"], o["O"][:, :, 7].contiguous(), K, V, n, w, sk)

    def outs():
        e = torch.empty_like
        return dict(O=e(Q), L=torch.empty((B, Hq, S), device="cuda"), dQ=e(Q), dK=e(K), dV=e(V),
                    d=torch.empty((B, Hq, D), dtype=BF, device="cuda"))

    got, want = outs(), outs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    if where == "stream":
        with torch.cuda.stream(s):
            step(got)
        torch.cuda.current_stream().wait_stream(s)
    else:
        with torch.cuda.stream(s):
            step(got)
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(got)
        for x in (Q, K, V, dO):
            x.mul_(0.5)
        n.fill_(77)
        for _ in range(3):
            graph.replay()
    step(want)
    assert binding.last_device_status() == 0
    for k in want:
        assert torch.equal(got[k], want[k]), k


def test_repeated_calls_are_bitwise_equal():
    Q, K, V = inputs(41, 1, 8, 2, 700, 700, 128)
    dO = inputs(42, 1, 8, 2, 700, 1, 128)[0]
    first = None
    for _ in range(3):
        O, L = torch.empty_like(Q), torch.empty((1, 8, 700), device="cuda")
        binding.attn_fwd_sinks(O, Q, K, V, L, 0.09, 100, 4)
        g = [torch.empty_like(x) for x in (Q, K, V)]
        binding.attn_bwd_sinks(*g, dO, Q, K, V, O, L, 0.09, 100, 4)
        now = [O, L, *g]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_window_workload_rows():
    """The ragged sliding-window workload at full size with sinks: sampled rows in fp64."""
    w = W.WINDOW
    x = W.make_prefill(w)
    Q, K, V = x.Q.cuda(), x.K.cuda(), x.V.cuda()
    kl = x.k_lengths.cuda()
    O = torch.empty_like(Q)
    L = torch.empty(Q.shape[:3], device="cuda")
    binding.attn_fwd_sinks(O, Q, K, V, L, w.scale, w.window, 4, 0, kl, kl)
    assert binding.last_device_status() == 0
    for b in range(w.B):
        n = int(kl[b])
        rows = torch.tensor([0, 4, 127, 4095, 4096, 4100, 5000, n - 1], device="cuda")
        vis = visible(w.Sq, n, w.window, 4, 0)[rows][None, None]
        want, lse, _, mag = ref_fwd(Q[b:b + 1, :, rows], K[b:b + 1, :, :n], V[b:b + 1, :, :n], vis,
                                    w.scale)
        # 4100 weights summed in fp32
        check(O[b:b + 1, :, rows], want, U * (mag + want.abs()) + 4 * F32 * mag, f"sequence {b}")
        assert float((L[b:b + 1, :, rows].double() - lse).abs().max()) <= 2e-5
        assert torch.all(O[b, :, n:] == 0)
    assert math.isfinite(float(O.float().abs().max()))


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("block", [8, 16, 256])
def test_pages_outside_the_pool_read_as_zeros(block, sinks):
    """Whatever the page number, also one whose row number does not fit 32 bits."""
    lens = [600, 300]
    c = (2, 8, 2, 128, 0, lens, 1000, 4, 2, block)
    Q, _, _, n, _, tables, Kp, Vp = decode_case(c, 0.0)

    def run(t, K, V):
        O = torch.full_like(Q, float("nan"))
        if sinks:
            binding.attn_decode_paged_sinks(O, Q, K, V, t, n, 1000, 4, 2)
        else:
            binding.attn_decode_paged(O, Q, K, V, t, n, 2)
        return O

    page = int(tables[0, 1])
    Kz, Vz = Kp.clone(), Vp.clone()
    Kz[page] = 0
    Vz[page] = 0
    want = run(tables, Kz, Vz)
    assert binding.last_device_status() == 0
    for bad in (-1, -(2 ** 31), Kp.shape[0], 2 ** 32 // block, 2 ** 31 - 1):
        t = tables.clone()
        t[0, 1] = bad
        got = run(t, Kp, Vp)
        assert binding.STATUS[binding.last_device_status()] == "ATTN_ERR_DEVICE_BOUNDS"
        assert torch.equal(got, want), bad
