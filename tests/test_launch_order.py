"""Kernels that start early (programmatic dependent launch) let the next one start only after their own wait, read from
the sources: when a kernel starts, every kernel two launches back has then completed, and what it wrote is visible to a
kernel that waits."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_verify_04_gb300", "csrc")


def kernels():
    """(file, name, body) of every kernel of the library."""
    for f in sorted(os.listdir(CSRC)):
        if not f.endswith((".cu", ".cuh")):
            continue
        with open(os.path.join(CSRC, f)) as fh:
            text = re.sub(r"//[^\n]*", "", fh.read())
        for m in re.finditer(r"__global__", text):
            head = text[m.end():text.index("{", m.end())]
            name = re.findall(r"(\w+)\s*\(", re.sub(r"__launch_bounds__\s*\((?:[^()]|\((?:[^()]|\([^()]*\))*\))*\)", "", head))[0]
            at = text.index("{", m.end())
            depth, i = 0, at
            while True:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                if depth == 0:
                    break
                i += 1
            yield f, name, text[at:i + 1]


def test_the_kernels_are_found():
    names = {name for _, name, _ in kernels()}
    assert {"plan_kernel", "append_kernel", "attend_rows_kernel", "attend_join_kernel", "attend_tile_kernel",
            "logprobs_kernel", "commit_tree_kernel", "ensure_pages_kernel"} <= names


def test_no_dependant_starts_before_its_own_wait():
    for f, name, body in kernels():
        if "pdl_trigger()" not in body:
            continue
        # a wait that every thread reaches: a statement of its own line, not behind a condition
        before = body[:body.index("pdl_trigger()")]
        assert re.search(r"^\s*pdl_wait\(\);", before, re.M), f"{f}: {name} lets its dependants start before it has waited"
