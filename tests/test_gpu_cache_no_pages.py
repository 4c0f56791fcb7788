"""A pool that runs out of pages: the status says so whatever was flagged before, the children
that lack their last page can be told from the table, and freeing and forking them again gives
them their tokens."""
import torch
import pytest

from gqa_attention_flash_b200 import binding

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
BLOCK, HKV, D = 8, 2, 64


def status():
    return binding.STATUS[binding.last_device_status()]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_missing_pages_are_not_hidden_by_a_clamped_length():
    t, refs = i32([[-1, -1], [-1, -1]]), i32([1, 1])
    # one call: row 0's length is past the table, and no page is left for any entry
    binding.cache_extend(t, refs, i32([0, 0]), i32([99, 8]), BLOCK)
    assert status() == "ATTN_ERR_NO_PAGES"
    # two calls: the first only clamps
    full, refs = i32([[0, 1], [-1, -1], [-1, -1]]), i32([1, 1])
    binding.cache_extend(full, refs, i32([0] * 3), i32([99, 0, 0]), BLOCK)
    src, dst = i32([0]), i32([0])
    binding.cache_fork(full, refs, i32([12, 0, 0]), i32([0]), i32([1]), src, dst, BLOCK)
    assert status() == "ATTN_ERR_NO_PAGES"
    # and it stays until it is read
    binding.cache_fork(full, refs, i32([12, 0, 0]), i32([0]), i32([1]), src, dst, BLOCK)
    binding.cache_extend(full, refs, i32([0] * 3), i32([99, 0, 0]), BLOCK)
    assert status() == "ATTN_ERR_NO_PAGES" and status() == "ATTN_OK"


def test_children_without_their_last_page_are_told_and_mended():
    R, width, n = 6, 4, 8
    g = torch.Generator().manual_seed(0)
    K, V = (torch.randn(n, BLOCK, HKV, D, generator=g).to(BF).cuda() for _ in range(2))
    # rows 0 (20 tokens: pages 0, 1, 2) and 1 (16 tokens, two whole pages); row 5 holds page 6
    t = i32([[0, 1, 2, -1], [3, 4, -1, -1]] + [[-1] * 4] * 3 + [[6, -1, -1, -1]])
    lens, refs = i32([20, 16, 0, 0, 0, 8]), i32([1, 1, 1, 1, 1, 0, 1, 1])  # only page 5 is free
    src, dst = i32([7] * 3), i32([7] * 3)
    pairs = i32([0, 0, 1]), i32([2, 3, 4])
    binding.cache_fork(t, refs, lens, *pairs, src, dst, BLOCK)
    assert status() == "ATTN_ERR_NO_PAGES"
    binding.cache_copy_blocks(K, V, src, dst)
    assert lens.tolist() == [20, 16, 20, 20, 16, 8]

    def missing():
        last = t.gather(1, (lens // BLOCK).clamp(max=width - 1).long()[:, None])[:, 0]
        return torch.nonzero((lens % BLOCK != 0) & (last < 0)).flatten().tolist()

    assert missing() == [3]              # row 2 got page 5, row 4 needed none
    assert (src.tolist(), dst.tolist()) == ([2, -1, -1], [5, -1, -1])
    # attention of such a row is flagged: its last tokens' page reads as zeros
    q = torch.randn(1, 4, D, generator=g).to(BF).cuda()
    o = torch.empty_like(q)
    binding.attn_decode_paged_sinks(o, q, K, V, t[3:4].contiguous(), lens[3:4].contiguous(), 100, 4)
    assert status() == "ATTN_ERR_DEVICE_BOUNDS"
    # row 5 ends; row 3 is given back and forked again
    binding.cache_free(t, refs, i32([5, 3]), i32([0, 0]), i32([width, width]))
    lens[5] = 0
    src, dst = i32([7]), i32([7])
    binding.cache_fork(t, refs, lens, i32([0]), i32([3]), src, dst, BLOCK)
    binding.cache_copy_blocks(K, V, src, dst)
    assert status() == "ATTN_OK" and missing() == []
    assert t.tolist() == [[0, 1, 2, -1], [3, 4, -1, -1], [0, 1, 5, -1], [0, 1, 6, -1], [3, 4, -1, -1], [-1] * 4]
    assert refs.tolist() == [3, 3, 1, 2, 2, 1, 1, 1]
    outs = []
    for r in (0, 2, 3):                  # the same tokens, through each row's own pages
        binding.attn_decode_paged_sinks(o, q, K, V, t[r:r + 1].contiguous(), lens[r:r + 1].contiguous(), 100, 4)
        outs.append(o.clone())
    assert status() == "ATTN_OK"
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
