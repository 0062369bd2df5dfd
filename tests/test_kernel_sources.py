"""Rules that the kernels' sources keep, which no run can show broken with certainty (no GPU needed)."""
import os
import re

import pytest

import split_kv_paged_splitkv_gb300._build as build


def code(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["append.cu", "key_weights.cu", "evict.cu", "cross_attend.cu"])
def test_no_read_only_loads_beside_a_running_writer(name):
    """These kernels start while the one before them on the stream may still write what they read (a query, a
    log-sum-exp, a length).  Loads of the read-only path promise that nothing writes meanwhile, and need not stay behind
    the wait for that kernel."""
    text = code(name)
    assert "wait_prerequisites" in text
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc|__restrict__", text)


@pytest.mark.parametrize("name", ["gqa_decode.cu", "mla_decode.cu"])
def test_the_decode_reads_its_inputs_with_plain_loads(name):
    """The append that turned the queries may be the kernel before, and lets the decode start before it has written
    them."""
    text = code(name)
    assert "wait_prerequisites" in text
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc", text)
