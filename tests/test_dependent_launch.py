"""Kernels that start before the kernel they depend on has ended (grid_dependency_wait in
csrc/tri_norm.cuh): what the two hold at the same time must not be promised to the compiler as
unchanging.  Read from the sources, no GPU."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "triangle_attention_biomolecular_b200", "csrc")


def closing(text, at):
    """Where the bracket that opens just before ``at`` is closed."""
    pairs = {"(": 1, "{": 1, ")": -1, "}": -1}
    depth = 1
    while depth:
        depth += pairs.get(text[at], 0)
        at += 1
    return at


def kernels():
    """(name, parameters, body) of every __global__ function, comments taken out."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*|/\*.*?\*/", " ", open(path).read(), flags=re.S)
        for m in re.finditer(r"__global__\s+void\s+", text):
            at = m.end()
            if text.startswith("__launch_bounds__", at):
                at = closing(text, text.index("(", at) + 1)
            start = text.index("(", at) + 1
            end = closing(text, start)
            body = text.index("{", end) + 1
            yield text[at:start - 1].strip(), text[start:end - 1], text[body:closing(text, body) - 1]


def test_waiting_kernels_read_nothing_as_read_only():
    """The producer's writes appear while such a kernel runs: a const __restrict__ pointer (or a
    load through the read-only path) would let its loads move ahead of the wait."""
    found = list(kernels())
    assert all(re.fullmatch(r"\w+", k[0]) for k in found)
    assert {"tri_norm_fwd_kernel", "tri_norm_bwd_kernel", "tri_relpos_bwd_kernel", "tri_act8_kernel"} <= {k[0] for k in found}
    waiting = [k for k in found if "grid_dependency_wait(" in k[2]]
    assert [k[0] for k in waiting] == ["tri_ordered_sum_kernel"]
    for name, params, body in waiting:
        assert "__restrict__" not in params, name
        assert not re.search(r"__ldg|\.nc\b", body), name
        # what it does before the wait touches no global memory
        before = body[:body.index("grid_dependency_wait(")]
        assert not re.search(r"\bpart\b|\bout\d\b|device_error_pending", before), name
