"""How the CTA pairs of the FP8 product order memory across the two CTAs, read
from the source: what one CTA announces to the other goes through a release at
cluster scope (or the fence of tensor memory) and an acquire at cluster scope,
and a pair that gives up waits for the copies of both. A missing order need not
show in a result, so no run can test it."""

from __future__ import annotations

import pathlib
import re

CSRC = pathlib.Path(__file__).resolve().parent.parent / "grads_taco_compress_gb300" / "csrc"


def test_arrivals_at_other_ctas_are_at_cluster_scope():
    """A release; or relaxed, where nothing but tensor memory is announced and
    its fence stands before the arrival."""
    found = set()
    for path in sorted(CSRC.glob("*.cu*")):
        for instr in re.findall(r"mbarrier\.arrive[\w.:]*", path.read_text()):
            if "shared::cluster" in instr:
                assert ".release.cluster." in instr or ".relaxed.cluster." in instr, (path.name, instr)
                found.add(instr)
    assert len(found) == 2
    _, body = pair_kernel()
    calls = [m.start() for m in re.finditer(r"arrive_even_read\(", body)]
    assert len(calls) == body.count("arrive_even_read(tempty0") == 2
    for at in calls:
        assert re.search(r"tc_fence_before\(\);\s*__syncwarp\(\);\s*if \(lane == 0\) $", body[:at])


def pair_kernel():
    source = (CSRC / "fp8_matmul.cu").read_text()
    start = source.index("matmul_pair_kernel(")
    return source, source[start:source.index("\n}\n", start)]


def test_waits_of_a_pair_acquire_at_cluster_scope():
    source, body = pair_kernel()
    # no other CTA touches the barriers of the CTA's own copy of `add` and of its tensor core's set of scale columns
    assert set(re.findall(r"wait_here\(base \+ S::(\w+)", body)) == {"added", "sdone"}
    assert set(re.findall(r"wait_pair\(base \+ S::(\w+)", body)) == {"empty", "tempty", "sfull", "full", "sempty",
                                                                     "tfull"}
    assert "wait_or_abort<true>" in source
    helper = (CSRC / "tcgen05.cuh").read_text()
    assert "mbarrier.try_wait.parity.acquire.cluster." in helper


def test_a_pair_that_gives_up_waits_for_the_copies_of_both_ctas():
    """The copies of both CTAs count on the even one's barriers, and the odd one
    may have issued stages that the even one has not."""
    _, body = pair_kernel()
    producer = body[:body.index("MMA issuer")]
    even, odd = producer.index("if (!ok && rank == 0)"), producer.index("else if (!ok)")
    assert "mbar_wait(base + S::full" in producer[even:odd]
    assert "kDrainNs" in producer[odd:]
