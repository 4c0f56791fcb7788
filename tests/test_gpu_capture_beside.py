"""A backward that is captured into a graph while other streams run, or capture, backwards of
their own: each call's second stream belongs to its own capture or to none."""
import ctypes

import pytest
import torch

from gqa_attention_flash_b200 import binding

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
B, HQ, HKV, S, D = 1, 32, 8, 1024, 64  # enough tiles for two streams


def rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()


class Backward:
    def __init__(self, seed, sinks):
        self.sinks = sinks
        self.Q, self.dO = rand(seed, B, HQ, S, D), rand(seed + 1, B, HQ, S, D)
        self.K, self.V = rand(seed + 2, B, HKV, S, D), rand(seed + 3, B, HKV, S, D)
        self.O, self.L = torch.empty_like(self.Q), torch.empty((B, HQ, S), device="cuda")
        if sinks:
            binding.attn_fwd_sinks(self.O, self.Q, self.K, self.V, self.L, 0.1, 300, 4)
        else:
            binding.attn_fwd(self.O, self.Q, self.K, self.V, self.L, 0.1, causal=True)
        self.grads = [torch.empty_like(x) for x in (self.Q, self.K, self.V)]
        self(None)
        torch.cuda.synchronize()
        self.want = [x.clone() for x in self.grads]

    def __call__(self, stream):
        args = (*self.grads, self.dO, self.Q, self.K, self.V, self.O, self.L, 0.1)
        if self.sinks:
            binding.attn_bwd_sinks(*args, 300, 4, stream=stream)
        else:
            binding.attn_bwd(*args, causal=True, stream=stream)

    def clear(self):
        for x in self.grads:
            x.zero_()
        torch.cuda.synchronize()

    def check(self):
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(self.grads, self.want))


class Graph:
    """Stream capture of the CUDA runtime (one that may lie beside another one)."""
    rt = None

    def __init__(self, stream, mode):
        if Graph.rt is None:
            Graph.rt = ctypes.CDLL("libcudart.so.12")
        self.s, self.graph, self.exec = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p(), ctypes.c_void_p()
        assert self.rt.cudaStreamBeginCapture(self.s, mode) == 0

    def end(self):
        assert self.rt.cudaStreamEndCapture(self.s, ctypes.byref(self.graph)) == 0
        assert self.rt.cudaGraphInstantiate(ctypes.byref(self.exec), self.graph, ctypes.c_ulonglong(0)) == 0

    def launch(self):
        assert self.rt.cudaGraphLaunch(self.exec, self.s) == 0

    def free(self):
        torch.cuda.synchronize()
        assert self.rt.cudaGraphExecDestroy(self.exec) == 0
        assert self.rt.cudaGraphDestroy(self.graph) == 0


@pytest.mark.parametrize("mode", [0, 1, 2])  # global, thread-local, relaxed
@pytest.mark.parametrize("sinks", [False, True])
def test_eager_beside_a_capture(sinks, mode):
    a, b = Backward(0, sinks), Backward(10, sinks)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    b.clear()
    g = Graph(sa, mode)
    try:
        a(sa)
        b(sb)   # runs now
        a(sa)   # the capture's own side stream again
        b(sb)
    finally:
        g.end()
    b.check()
    a.clear()
    for _ in range(3):
        g.launch()
        b(sb)
    a.check()
    b.check()
    g.free()


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_workspaces_beside_a_capture(mode):
    """Calls on another stream that allocate: decode in slices, a tree, fork and extend."""
    q, k = rand(0, 2, 8, D), rand(1, 40, 16, 2, D)
    o, O = torch.empty_like(q), torch.empty((2, 8, 3, D), dtype=BF, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, par = i32([100, 37]), i32([[-1, 0, 1]] * 2)
    t0, refs0 = torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10), torch.zeros(40, dtype=torch.int32, device="cuda")
    t, refs, L, p, c, src, dst = t0.clone(), refs0.clone(), lens.clone(), i32([0]), i32([1]), i32([0]), i32([0])
    to, Q3 = L + 60, rand(2, 2, 8, 3, D)

    def calls(s):
        binding.attn_decode_paged(o, q, k, k, t0, lens, 8, stream=s)
        binding.attn_tree_paged(O, Q3, k, k, t0, lens, par, stream=s)
        binding.cache_fork(t, refs, L, p, c, src, dst, 16, stream=s)
        binding.cache_extend(t, refs, L, to, 16, stream=s)

    def result():
        torch.cuda.synchronize()
        assert binding.last_device_status() == 0
        got = [x.clone() for x in (o, O, t, refs, L, src, dst)]
        for x, y in ((t, t0), (refs, refs0), (L, lens)):
            x.copy_(y)
        o.zero_(), O.zero_()
        torch.cuda.synchronize()
        return got

    calls(None)
    want = result()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    g = Graph(sa, mode)
    try:
        calls(sa)
        calls(sb)
    finally:
        g.end()
    assert all(torch.equal(x, y) for x, y in zip(result(), want))
    g.launch()
    assert all(torch.equal(x, y) for x, y in zip(result(), want))
    g.free()


@pytest.mark.parametrize("sinks", [False, True])
def test_two_captures_at_once(sinks):
    a, b, c = Backward(0, sinks), Backward(10, sinks), Backward(20, sinks)
    sa, sb, sc = (torch.cuda.Stream() for _ in range(3))
    c.clear()
    ga = Graph(sa, 2)
    gb = Graph(sb, 2)
    try:
        for _ in range(2):
            a(sa)
            b(sb)
            c(sc)
    finally:
        ga.end()
        gb.end()
    c.check()
    a.clear()
    b.clear()
    for _ in range(3):
        ga.launch()
        gb.launch()
        c(sc)
    for x in (a, b, c):
        x.check()
    ga.free()
    gb.free()
