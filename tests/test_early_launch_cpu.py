"""Kernels that are launched before the launch that feeds them has ended: how they read
what it writes, from their source."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lm_head_selected_gb300", "csrc")


def _kernels(text):
    """(parameters, body) of every __global__ function, without comments."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__", text):
        start = text.index("{", m.end())
        depth, at = 1, start + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield text[m.start():start], text[start:at]


def _waiting():
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            found += [(re.search(r"(\w+)\s*\($", head[:head.index("(", head.rindex("_kernel")) + 1]).group(1), body)
                      for head, body in _kernels(f.read()) if "griddepcontrol.wait" in body]
    return found


def test_there_are_such_kernels():
    assert {name for name, _ in _waiting()} == {"embedding_reduce_kernel", "layer_norm_join_kernel"}


@pytest.mark.parametrize("name,body", _waiting(), ids=[n for n, _ in _waiting()])
def test_nothing_is_read_through_the_read_only_path_or_before_the_wait(name, body):
    """The read-only path (__ldg) is for memory that no one writes while the kernel is resident,
    and neither it nor __ldcg need stay behind the wait when the compiler orders loads."""
    before, after = body.split("griddepcontrol.wait", 1)
    assert "load_written(" in after
    for load in ("__ldg(", "__ldcg(", "::load("):
        assert load not in body, (name, load)
    assert not re.search(r"load_written\(|\bp\.|\bpart\b", before)
