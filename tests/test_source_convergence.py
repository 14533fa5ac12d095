"""Aligned warp instructions (cluster barriers, TMEM loads and frees) are undefined on a warp that is not converged,
and no run on a GPU shows it: the grouped products' sources are read for the __syncwarp() in front of them."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_layer_top_b200", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _block(text, start):
    """The text of the braces that open behind `start`."""
    i = text.index("{", start)
    depth = 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[i:j + 1]
    raise AssertionError("unbalanced braces")


@pytest.mark.parametrize("function", ["cluster_barrier", "tmem_free_for"])
def test_wrappers_converge_their_warp_first(function):
    text = _source("grouped_common.cuh")
    body = _block(text, text.index(f"void {function}("))
    assert 0 <= body.find("__syncwarp()") < body.index("asm volatile")


@pytest.mark.parametrize("name", ["grouped_bf16.cu", "grouped_fp8.cu", "grouped_fp8_pair.cu"])
def test_kernels_use_the_wrapper(name):
    assert "barrier.cluster" not in _source(name)


def test_tmem_loads_behind_stores_that_branch_by_lane():
    """A loop over chunks that loads from TMEM and stores by lane converges the warp at its head."""
    text = _source("grouped_bf16.cu")
    loops = [_block(text, m.start()) for m in re.finditer(r"for \(int c = [^;]*;[^;]*;[^)]*\)", text)]
    loops = [b for b in loops if "tmem_ld" in b and ("store_columns16(" in b or "store_3d<" in b)]
    assert len(loops) == 2
    for body in loops:
        assert 0 <= body.find("__syncwarp()") < body.index("tmem_ld")


def test_a_hand_over_between_two_ctas_is_acquired_at_cluster_scope():
    """The peer arrives on peer_full behind writes to its own shared memory (release at cluster scope): a wait that
    acquires for its own CTA only does not order them."""
    common, kernel = _source("grouped_common.cuh"), _source("grouped_bf16.cu")
    assert "arrive_in_cluster_release(in_cta(&peer_full[stage], 0))" in kernel
    waits = re.findall(r"(\w+)\(&peer_full\[stage\]", kernel)
    assert waits and all("acquire.cluster" in _block(common, common.index(f"bool {w}(")) for w in set(waits) - {"in_cta"})
