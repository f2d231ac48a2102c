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
