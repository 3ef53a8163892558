"""No kernel that may start before the one in front of it has ended can itself end first.

A launch on a stream waits for the launch before it only. Where that one was started early by
the launch before *it* (griddepcontrol.launch_dependents), it has to hold the order: at least one
of its threads executes griddepcontrol.wait before its grid ends. Read off the sources (CPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_77_gb300", "csrc")
# Returns in front of a wait: warps of a block whose first warp goes on.
PART_OF_A_BLOCK = {"decode_merge_kernel": ["if (h >= n_rep) return;"]}


def _kernels():
    for file in sorted(os.listdir(CSRC)):
        if not file.endswith((".cu", ".cuh")):
            continue
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, file)).read())
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\s*\(", text):
            start = at = text.index("{", m.end())
            depth = 0
            while True:
                depth += (text[at] == "{") - (text[at] == "}")
                if depth == 0:
                    break
                at += 1
            yield m.group(1), text[start:at]


KERNELS = dict(_kernels())


def test_the_kernels_are_found():
    for name in ("decode_merge_kernel", "sparse_merge_kernel", "mla_merge_kernel", "prefill_merge_kernel",
                 "decode_tc_kernel", "decode_fp8_kernel", "decode_fp4_kernel", "select_rows_kernel",
                 "attn_weights_runs_kernel", "compact_rows_kernel", "rope_write_kernel"):
        assert "pdl_wait" in KERNELS[name], name


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_no_return_before_the_wait(name):
    body = KERNELS[name]
    if "pdl_wait" not in body:  # launched behind everything that precedes it
        return
    before = body[:body.index("pdl_wait")]
    returns = [line.strip() for line in before.split("\n") if re.search(r"\breturn;", line)]
    assert returns == PART_OF_A_BLOCK.get(name, [])
