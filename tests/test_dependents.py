"""Kernels launched as programmatic dependents of whatever is before them on the stream: what their sources may not do (CPU)."""
import os
import re

import pytest

from helpers import ROOT

CSRC = os.path.join(ROOT, "exact_softmax_attention_gb300", "csrc")
FILES = ("attn_norm.cu", "attn_score.cu", "attn_score_tiles.cu", "attn_evict.cu", "score.cuh")


def code(name):
    """The source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", FILES)
def test_no_loads_of_constant_data(name):
    """Such a kernel is alive while the one before it still writes, so nothing that it reads is constant for its lifetime: loads through the
    read-only path (which the compiler may also move over the wait) are not allowed."""
    assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", code(name))


@pytest.mark.parametrize("name", FILES[:-1])
def test_every_dependent_kernel_waits(name):
    """Each __global__ function waits for the grid before it: a later kernel that waits for this one then knows that all before it is done.
    (split_q_kernel is an ordinary launch.)"""
    parts = re.split(r"__global__", code(name))[1:]
    assert parts
    for p in parts:
        kernel = re.search(r"(\w+_kernel)\s*\(", p).group(1)
        assert "grid_dependency_wait()" in p or kernel == "split_q_kernel", kernel


def test_the_parts_of_q_come_from_an_ordinary_launch():
    """score_tiles_kernel over 8-bit caches and score_join_kernel read lengths, pages, keys and old sums before they wait: whatever wrote those
    has ended by then, because split_q_kernel does not start before it has (and for bf16 the tile kernel waits before it lets dependents start)."""
    text = code("attn_score_tiles.cu")
    assert re.search(r"launch_kernel\(split_q_kernel<D>, [^;]*?, stream, \{\}, ", text)
    tiles = text.split("score_tiles_kernel(", 1)[1]
    wait, start = tiles.index("if (!F8) grid_dependency_wait();"), tiles.index("grid_dependents_launch();")
    assert wait < start
