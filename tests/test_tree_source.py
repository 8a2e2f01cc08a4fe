"""Rules that tree.cu keeps where breaking them could fault or race on a GPU:
they are read off the source, no run of the broken form shows them."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "invariant_sequence_decode_gb300", "csrc",
                      "tree.cu")


def kernel(name):
    """The kernel's body, without comments."""
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    body = text[re.search(r"\b" + name + r"\([^;]*?\)\s*\{", text).end():]
    depth = 1
    for i, c in enumerate(body):
        depth += (c == "{") - (c == "}")
        if depth == 0:
            return body[:i]
    raise AssertionError(name)


def test_only_encoded_maps_are_prefetched():
    """A short prefix's view has no tensor map: its place holds zeros."""
    body = kernel("tree_chunk_kernel")
    at = body.index("prefetch.tensormap")
    assert re.search(r"if \(b\.view\[view\]\.n_chunk > 0\)\s*asm volatile\(\"$", body[:at])


@pytest.mark.parametrize("name", ["tree_merge_kernel", "tree_short_kernel"])
def test_nothing_is_read_ahead_of_the_wait(name):
    """What earlier kernels wrote is visible to a kernel behind its own wait, whatever
    the kernel between them has waited for."""
    body = kernel(name)
    ahead = body[:body.index("pdl_wait()")]
    assert not re.search(r"ld_\w+\(|tree_key\(|__ldg|__ldcg|\b(q|part_o|part_ml|qp|mlp|po)\[|\*\s*(q|qp|mlp|po)\s*;", ahead)


def test_a_chunk_writes_none_of_its_results_before_its_last_product_is_awaited():
    """Maximum and sum go out with O: after an expired wait none of the three does."""
    body = kernel("tree_chunk_kernel")
    take = body[body.index("auto take = "):]
    take = take[:take.index("return done;")]
    assert body.count("part_ml[") == take.count("part_ml[") == 2 and "prev_row >= 0 && done" in take
    assert take.index("part_ml[") > take.index("mbar_wait(&bar.o_full")
