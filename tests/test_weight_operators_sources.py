"""Properties of the weight operators' kernels that no run can show, since no copy or product is ever late
enough here: what happens when a bounded wait gives up. Read from the sources, without a GPU."""
import glob
import os
import re

import pytest

from deformable_convolution_sparse_b200 import binding as B

CSRC = os.path.join(os.path.dirname(B.__file__), "csrc")
FILES = ("dcnv4_predictor_backward.cuh", "dcnv4_orthogonalize.cuh", "dcnv4_mx.cuh")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _block(text, at):
    """The braces that open at or after ``at``, with what is between them."""
    first = text.index("{", at)
    depth = 0
    for i in range(first, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[first:i + 1]
    raise AssertionError("unbalanced braces")


def _kernels(name):
    """(name, body) of every kernel of a source file."""
    text = _code(name)
    for m in re.finditer(r"__global__", text):
        body = _block(text, m.end())
        yield re.search(r"(\w+_kernel)\(", text[m.end():]).group(1), body


def test_converting_warps_give_up_as_a_whole():
    """The converting warps vote (Piece::landed), hand tiles over by __syncwarp and meet at named barriers: every
    bounded wait of theirs has one answer for the whole warp. Lanes that gave up one by one would leave the others
    in the vote for good."""
    seen = 0
    for name, body in _kernels("dcnv4_predictor_backward.cuh"):
        at = body.find("if (warp < 16) {")
        if at < 0:
            continue
        seen += 1
        branch = _block(body, at)
        assert "mbar_wait_bounded" not in branch, name
        assert "tc::warp_wait(" in branch and "hand_over(" in branch, name
    assert seen == 3


@pytest.mark.parametrize("file", FILES)
def test_a_kernel_that_gives_up_leaves_nothing_in_flight(file):
    """A kernel whose wait gave up waits once more, again with a limit, for the loads and products it has in flight
    before it frees its tensor memory and leaves: they would land in memory that is no longer its own."""
    seen = 0
    for name, body in _kernels(file):
        if "tc::alloc(" not in body:
            continue
        seen += 1
        if "tc::tma_load_3d(" in body:
            gave_up = _block(body, body.index("if (!__syncthreads_and(ok)) {"))
            assert "tc::drain_loads<" in gave_up and "tc::drain_products(drain)" in gave_up, name
            assert body.index("mbar_init(drain, 1)") < body.index("griddepcontrol"), name
            # every ring of loads is among them
            for bar in set(re.findall(r"tc::tma_load_3d\([^;]*&(\w+)\[", body)):
                assert f"({bar}, " in gave_up, (name, bar)
        else:
            # products only, one batch at a time: the same barrier is waited for again
            done = re.search(r"mbar_wait_bounded\(&?(done\w*)", body).group(1)
            gave_up = body[body.index("if (!ok)"):]
            assert len(re.findall(rf"mbar_wait_bounded\(&?{done}\b", body)) == 2, name
            assert re.search(rf"mbar_wait_bounded\(&?{done}\b", gave_up), name
            if "cp.async.cg" in body:
                assert "cp.async.wait_all" in _block(body, body.index("if (!ok)")), name
    assert seen > 0
