"""What no run can show, read from the kernels' sources.

The end of a kernel after a wait that ran out needs a broken pipeline to run, so its order is checked in
the text: copies and MMAs in flight get their time (`linger`) before tensor memory is freed and before
any warp leaves. Launch rules go by the device's own SM count, which one machine cannot vary.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_mla_kv_qdecode_b200", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["page_scores.cu"])
def test_tensor_memory_is_freed_after_the_work_in_flight(name):
    code = _code(name)
    free = [m.start() for m in re.finditer(r"ptx::tmem_dealloc\(", code)]
    assert len(free) == 1
    # the last barrier of all threads, then the wait of every one of them, then the release
    barrier = code.rindex("__syncthreads();", 0, free[0])
    between = code[barrier:free[0]]
    assert re.search(r"if \(\*abort_flag\) ptx::linger\(\);", between), between
    assert "globaltimer" not in code[free[0]:code.index("\n}\n", free[0])]


def test_every_leaving_warp_of_the_digest_ring_waits():
    code = _code("qcache_read.cu")
    body = code[code.index("page_digest_ring_kernel(const DigestArgs"):]
    body = body[:body.index("\n}\n")]
    # both roles: the copying warp and the summing ones
    assert re.search(r"if \(!ok\) ptx::linger\(\);\s*return;", body)
    assert re.search(r"if \(!wait\(&m\.full\[s\][^{]*\{\s*ptx::linger\(\);\s*break;", body)


@pytest.mark.parametrize("name", ["page_scores.cu", "page_select.cu", "qcache_read.cu", "norm_rope.cu"])
def test_launch_rules_name_no_sm_count(name):
    assert not re.search(r"\b14[48]\b", _code(name))
