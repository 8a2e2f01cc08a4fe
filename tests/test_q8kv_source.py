"""Rules that the kernels of caches in 8 bits keep where breaking them could fault or race
on a GPU: they are read off the source, no run of the broken form shows them."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "invariant_sequence_decode_gb300", "csrc")


def kernel(source, name):
    """The kernel's body, without comments."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, source)).read())
    body = text[re.search(r"\b" + name + r"\([^;]*?\)\s*\{", text).end():]
    depth = 1
    for i, c in enumerate(body):
        depth += (c == "{") - (c == "}")
        if depth == 0:
            return body[:i]
    raise AssertionError(name)


def test_only_encoded_maps_are_prefetched():
    """A view without blocks has no tensor map: its place holds zeros."""
    body = kernel("q8kv.cu", "q8kv_chunk_kernel")
    at = body.index("prefetch.tensormap")
    assert re.search(r"if \(b\.view\[view\]\.n_chunk > 0\)\s*asm volatile\(\"$", body[:at])


@pytest.mark.parametrize("source,name", [("q8kv.cu", "q8kv_merge_kernel"), ("q8kv_seal.cu", "q8kv_seal_kernel"),
                                         ("rope_kv.cu", "qk_norm_rope_kernel"), ("q8kv.cu", "q8_produce")])
def test_nothing_is_read_ahead_of_the_wait(source, name):
    """What earlier kernels wrote is visible to a kernel behind its own wait."""
    body = kernel(source, name)
    ahead = body[:body.index("pdl_wait()")]
    # (a function that the kernel only defines there is called behind the wait)
    ahead = re.sub(r"auto \w+ = \[&\]\([^)]*\) \{.*?\};", "", ahead, flags=re.S)
    assert not re.search(r"ld_\w+\(|seal_load\(|tma_load|__ldg|(?<!b\.)\b(k|v|q|pos|row|qkv|part_o|part_ml|table)\[|\.start\(", ahead)


def test_q_is_read_and_results_are_written_behind_a_wait():
    """Both places that prepare q, and the results, whose place an earlier merge may still read."""
    body = kernel("q8kv.cu", "q8kv_chunk_kernel")
    calls = [m.start() for m in re.finditer(r"q8_prepare<S>\(", body)]
    waits = [m.start() for m in re.finditer(r"pdl_wait\(\)", body)]
    assert len(calls) == 3 and len(waits) == 2
    assert waits[0] < calls[0] < calls[1] and waits[1] < calls[2]
    assert "if (head == 0) pdl_wait();" in body[:calls[2]]


def test_a_chunk_writes_none_of_its_results_after_an_expired_wait():
    body = kernel("q8kv.cu", "q8kv_chunk_kernel")
    take = body[body.index("auto take = "):body.index("q8_each_run(b, Hkv, w, [&](const Q8Run& t) {\n            const Q8View& v")]
    assert "const int left = ok ? end_left - 8 * part : 0;" in take
    assert body.count("part_ml") == take.count("part_ml") and body.count("part_o +") == take.count("part_o +") == 1
    for store in re.finditer(r"(ml|po)\[[^\]]*\] = ", take):
        assert re.search(r"< left\)[^;]*(;[^;}]*)*$", take[:store.start()])
