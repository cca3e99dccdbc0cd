"""Waits that give up leave a warp together. The softmax warps of the attention
kernels vote and use the tensor memory's warp-wide instructions between their
waits, and the 4-bit copiers meet at warp barriers, so a wait that runs out in
some lanes has to end the loop in all of them."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deepseek_sparse_attention_score_gb300",
                    "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def _between(text, first, last):
    a = text.index(first)
    return text[a: text.index(last, a)]


@pytest.mark.parametrize("name,first,last", [
    ("attend_cache.cu", "- softmax\n", "- epilogue\n"),
    ("attend_cache.cu", "- epilogue\n", "const bool have_o"),
    ("attend_cache.cu", "gen.init(prm, t, ntok, split)", "tmem_st_wait();"),  # the queries' move into tensor memory
    ("attend_cache.cu", "void copy_keys(", "// The copier of the bf16 cache"),
    ("attend_cache.cu", "void issue_mmas(", "// A copier warp:"),
    ("attend.cu", "- softmax\n", "const bool have_o"),
    ("indexer.cu", "- epilogue\n", "tmem_dealloc("),
    ("attend.cu", "if (warp >= 4 && warp < 8) {", "tmem_st_wait();"),
])
def test_whole_warps_wait_as_one(name, first, last):
    part = _between(_source(name), first, last)
    assert re.search(r"\bmbar_wait_warp\(", part)
    assert not re.search(r"\bmbar_wait\(", part)


@pytest.mark.gpu
def test_a_wait_that_runs_out_in_half_of_a_warp():
    import torch

    import __graft_entry__

    __graft_entry__.build()
    import deepseek_sparse_attention_score_gb300 as dsa

    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.dsa_selftest_wait_timeout(st, limit_clocks=2_000_000)  # about a millisecond for each of its two waits
    torch.cuda.synchronize()
    assert st.item() == 8  # DSA_STATUS_TIMEOUT, and no lane took the second wait for met


@pytest.mark.parametrize("name,first,last,waits", [
    ("attend_cache.cu", "void copy_boxes(", "// The g-th run of", r"mbar_wait_drain\(br\.full"),
    ("attend.cu", "if (*abort_flag && lane == 0) {", "tmem_dealloc(", r"while \(clock64\(\) - t0 < "),
])
def test_copies_in_flight_are_waited_for_when_unwinding(name, first, last, waits):
    """A block that gives up waits (bounded) until its TMA boxes have landed:
    shared memory must not be written after the block has gone."""
    assert re.search(waits, _between(_source(name), first, last))
