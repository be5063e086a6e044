"""What the kernels do after a bounded wait gave up, read off their source: no wait can be made to give up on a GPU
without holding its kernel for the whole limit, and a mistake here would hang it."""
import os
import re

import pytest

from normalisation_row_bf16_b200 import build as nbuild


def source(name):
    with open(os.path.join(nbuild.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name,waits", [("gated_ffn.cu", 1), ("gated_mxfp8.cu", 1), ("gemm_mxfp8.cu", 3)])
def test_epilogues_leave_by_vote(name, waits):
    """Whether a warp of an epilogue goes on to its next tcgen05.ld (.sync.aligned) is decided by all its lanes at
    once: each wait for a full accumulator, with the look at the failure flag, is inside a vote."""
    s = source(name)
    found = re.findall(r"[^;{}]*mbar_wait_bounded\(&S\.acc_full[^;]*;", s)
    assert len(found) == waits
    for stmt in found:
        assert re.search(r"__all_sync\(0xFFFFFFFFu, mbar_wait_bounded\(&S\.acc_full.*failed_flag", stmt, re.S), stmt


@pytest.mark.parametrize("kernel", ["ln_fwd_ring_kernel", "ln_bwd_kernel"])
def test_row_rings_stop_and_drain(kernel):
    """A ring whose wait gave up is fetched into no more (its stage's barrier is still armed) and its copies in flight
    are waited for before the block ends."""
    s = source("layernorm.cu")
    at = s.index("void __launch_bounds__", s.index("struct LnFwdRing")) if kernel == "ln_fwd_ring_kernel" else 0
    body = s[s.index(kernel + "(", at):]
    body = body[:body.index("\n}\n")]
    loop = body[body.index("bool ok = true;"):]
    guards = re.findall(r"if \(tid == 0([^{;]*?)\) (?:\{\s*if \(KEEP\) )?refill\(", loop)
    assert guards and all("&& ok &&" in g for g in guards), guards
    assert re.search(r"if \(tid == 0 && !ok\) drain\(", loop)
    if "A.partial" in loop:
        assert loop.index("drain(") < loop.index("if (!A.partial) return;")
