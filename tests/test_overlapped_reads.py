"""Kernels that may start while the stream's previous kernel still writes read what it
wrote by ordinary loads alone.  The read-only path (ld.global.nc, by __ldg or through
a pointer to const that is __restrict__) is for memory that nobody writes during the
kernel's lifetime, and a compiler may move such a load ahead of the wait."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "int4_weight_only_w4_gb300", "csrc")
TEXT = {f: re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read())
        for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh"))}
OVERLAPPED = [f for f, text in TEXT.items()
              if f.endswith(".cu") and "begin_after_previous();" in text]


def test_the_kernels_are_found():
    assert {"w4_kv_blocks.cu", "w4_select.cu", "w4_paged_attn.cu", "w4_attn_weights.cu",
            "w4_kv_gather.cu", "w4_kv_cache.cu", "w4_rope.cu"} <= set(OVERLAPPED)


@pytest.mark.parametrize("source", OVERLAPPED + [f for f in TEXT if f.startswith("w4_kv") or
                                                 f.startswith("w4_attn")])
def test_reads_are_ordinary_loads(source):
    text = TEXT[source]
    assert not re.findall(r"__ldg\s*\(", text)
    assert "ld.global.nc" not in text and ".nc." not in text
    assert not re.findall(r"const\s+[\w:]+\s*\*\s*__restrict__", text)
