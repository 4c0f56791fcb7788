"""The range-checked build's coverage, read from the sources: every kernel checks the TMA
coordinates, workspace slots, table entries and pool rows that it uses, except those whose
indices are their own grid and the sizes of the call."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gqa_attention_flash_b200",
                    "csrc")

# no index that comes from data, a list of work or a split: blocks and threads over whole tensors
UNCHECKED = {"wait_probe_kernel", "bwd_delta_kernel", "decode_combine_kernel", "rbs_centroid_kernel",
             "rbs_beta_kernel", "rbs_scores_kernel"}


def bodies(text, start):
    """The text between the first brace behind `start` and the one that closes it."""
    i = text.index("{", start)
    depth, j = 0, i
    while True:
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        j += 1
        if depth == 0:
            return text[i:j]


def kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__", text):
            name = re.search(r"(\w+_kernel)\s*\(", text[m.end():]).group(1)
            yield name, bodies(text, m.end())


def test_every_kernel_checks_its_indices():
    found = dict(kernels())
    assert len(found) > 15
    unchecked = {name for name, body in found.items() if "in_range(" not in body}
    assert unchecked == UNCHECKED


def test_the_rows_of_the_cache_are_checked_where_they_are_looked_up():
    text = open(os.path.join(CSRC, "cache_ops.cu")).read()
    body = bodies(text, text.index("long long pool_row("))
    assert body.index("in_range(") < body.index("bt[pos")
    body = bodies(text, text.index("__device__ int free_pages("))
    assert body.index("in_range(") < body.index("list[rank")
