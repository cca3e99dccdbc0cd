"""Waits of the append and of prefix attention that give up leave a warp
together, tell the rest of their block or cluster, and let copies in flight land
before shared and tensor memory go back."""
import re

import pytest

from test_warp_waits import _between, _source


@pytest.mark.parametrize("name,first,last,waits", [
    ("prefix.cu", "- MMA issuer\n", "- queries and keys\n", r"\bmbar_wait_warp(_cluster)?\("),
    ("prefix.cu", "- queries and keys\n", "- key tiles\n", r"\bmbar_wait_warp\("),
    ("prefix.cu", "- key tiles\n", "- P of the other half, for the MMA issuer\n", r"\bmbar_wait_warp\("),
    ("prefix.cu", "- P of the other half, for the MMA issuer\n", "- softmax\n", r"\bmbar_wait_warp\("),
    ("prefix.cu", "- softmax\n", "- epilogue\n", r"\bmbar_wait_warp\("),
    ("prefix.cu", "- epilogue\n", "// No barrier here:", r"\bmbar_wait_warp\("),
    ("append.cu", "append_bulk_kernel(const", "if (!ok) {", r"\bmbar_wait_warp\("),
])
def test_whole_warps_wait_as_one(name, first, last, waits):
    part = _between(_source(name), first, last)
    assert re.search(waits, part)
    # no other kind of wait, and none without a limit
    assert not re.search(r"\b(mbar_wait|mbar_try_wait\w*|mbar_wait_drain)\(", part)
    assert "barrier.sync" not in part and "bar.sync" not in part


@pytest.mark.parametrize("first,last", [
    ("- MMA issuer\n", "- queries and keys\n"), ("- queries and keys\n", "- key tiles\n"),
    ("- key tiles\n", "- P of the other half, for the MMA issuer\n"),
    ("- P of the other half, for the MMA issuer\n", "- softmax\n"), ("- epilogue\n", "// No barrier here:"),
])
def test_a_role_that_gives_up_tells_the_cluster(first, last):
    assert "give_up();" in _between(_source("prefix.cu"), first, last)


@pytest.mark.parametrize("name,first,last,waits", [
    ("prefix.cu", "if (*abort_flag) {", "tmem_dealloc_pair(", r"while \(clock64\(\) - t0 < "),
    ("append.cu", "if (!ok) {", "}  // namespace", r"mbar_wait_drain\("),
])
def test_copies_in_flight_land_first(name, first, last, waits):
    part = _between(_source(name), first, last)
    assert re.search(waits, part) and "DSA_STATUS_TIMEOUT" in part


def test_the_cluster_meets_before_and_after_the_delay():
    """Copies into another block's shared memory, and its tensor memory, outlive this one's roles."""
    end = _between(_source("prefix.cu"), "lists(std::true_type{});", "tmem_dealloc_pair(")
    assert end.count("cluster_sync_all();") == 2
    assert end.index("cluster_sync_all();") < end.index("*abort_flag") < end.rindex("cluster_sync_all();")
