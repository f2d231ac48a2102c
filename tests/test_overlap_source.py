"""Rules of the kernels that may become resident while their predecessor of the
stream still runs, checked in their source: what breaks them shows on a GPU only
by chance, or as a wait that runs out."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mixture_experts_layer_schedule_gb300", "csrc")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def overlapped_files():
    """Files whose kernels wait for their predecessor, and the headers of their device code."""
    cu = [f for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") and "grid_dep_wait()" in source(f)]
    heads = {h for f in cu for h in re.findall(r'#include "([^"/]+\.cuh)"', source(f))}
    return cu, sorted(heads)


def test_the_files_are_found():
    cu, heads = overlapped_files()
    assert cu == ["ffn.cu", "fp4.cu", "fp4_gemm.cu"] and {"dense_common.cuh", "fp4.cuh"} <= set(heads)


def test_no_loads_on_the_read_only_path():
    """Data that the predecessor may still write when the kernel starts is not
    constant for the kernel's lifetime."""
    cu, heads = overlapped_files()
    for f in cu + heads:
        for bad in (r"__ldg\b", r"\.nc\b", r"__restrict__"):
            assert not re.search(bad, source(f)), (f, bad)


def kernels(text):
    """(name, body) of every kernel in a source; bodies by their braces."""
    for m in re.finditer(r"__global__[^;{]*?(\w+)\s*\(const __grid_constant__[^{]*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1), text[m.end():i]


def roles(body):
    """The parts of a kernel's body, at its own level, that different warps run."""
    cuts = [m.start() for m in re.finditer(r"^  (?:if \(warp == 0|\} else )", body, flags=re.M)]
    end = [m.start() for m in re.finditer(r"^  \}$", body, flags=re.M) if m.start() > cuts[-1]][0]
    return body[:cuts[0]], [body[a:b] for a, b in zip(cuts, cuts[1:] + [end])]


@pytest.mark.parametrize("name", ["ffn.cu", "fp4_gemm.cu"])
def test_barriers_are_waited_for_after_the_predecessor(name):
    """A wait on a barrier has a limit in cycles. Before the predecessor has ended, nothing
    has to arrive, so every role waits for it first: a long predecessor must not look
    like a hung barrier."""
    found = list(kernels(source(name)))
    assert len(found) == 2
    for kernel, body in found:
        before, parts = roles(body)
        assert len(parts) >= 3, kernel
        for i, part in enumerate(parts):
            first = re.search(r"\b(?:warp_wait|mbar_wait|wait_drain_bar)\s*\(", part)
            assert first, (kernel, i)
            assert "grid_dep_wait()" in before or "grid_dep_wait()" in part[:first.start()], (kernel, i)
