"""Kernels that start before the kernel they depend on has ended (grid_dependency_wait in
csrc/tri_norm.cuh): what the two hold at the same time must not be promised to the compiler as
unchanging.  Read from the sources, no GPU."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "triangle_attention_biomolecular_b200", "csrc")


def kernels():
    """(name, parameters, body) of every __global__ function, comments taken out."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*|/\*.*?\*/", " ", open(path).read(), flags=re.S)
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\s*\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\s*\(", text):
            end = m.end()
            depth = 1
            while depth:  # the parameter list
                depth += {"(": 1, ")": -1}.get(text[end], 0)
                end += 1
            start = text.index("{", end)
            stop, depth = start + 1, 1
            while depth:  # the body
                depth += {"{": 1, "}": -1}.get(text[stop], 0)
                stop += 1
            yield m.group(1), text[m.end():end - 1], text[start:stop]


def test_waiting_kernels_read_nothing_as_read_only():
    """The producer's writes appear while such a kernel runs: a const __restrict__ pointer (or a
    load through the read-only path) would let its loads move ahead of the wait."""
    found = list(kernels())
    assert len(found) > 10
    waiting = [k for k in found if "grid_dependency_wait(" in k[2]]
    assert [k[0] for k in waiting] == ["tri_ordered_sum_kernel"]
    for name, params, body in waiting:
        assert "__restrict__" not in params, name
        assert not re.search(r"__ldg|\.nc\b", body), name
        # what it does before the wait touches no global memory
        before = body[:body.index("grid_dependency_wait(")]
        assert not re.search(r"\bpart\b|\bout\d\b|device_error_pending", before), name
