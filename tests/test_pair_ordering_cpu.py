"""Memory ordering between the two CTAs of the MXFP4 pair kernel, read from its
source: no run can show that an ordering is missing, only that it is written.

The second CTA's copies land in its own shared memory and are seen by its
warp 1, which tells the first CTA's MMA issuer; the issuer's MMAs then read that
memory.  A release and an acquire of CTA scope order nothing across two CTAs,
so every arrival at the other CTA releases, and every wait of the issuer for such
arrivals acquires, at cluster scope."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mxfp4_quantised_mixture_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, head):
    """The braces' content after the first ``head``."""
    at = text.index("{", text.index(head))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(head)


def test_arrivals_at_the_other_cta_release_at_cluster_scope():
    pair, tc = source("matmul_pair.cu"), source("tc_sm100.cuh")
    # warp 1 of the second CTA: waits for its copies, then arrives at the first CTA's barrier
    second = pair[pair.index("const uint32_t to = tc::cluster_addr(ready, 0);"):]
    second = body(second, "for (uint32_t i = first")
    assert "&full[s]" in second and "tc::mbar_arrive_cluster(to + s * 8)" in second
    arrive = body(tc, "void mbar_arrive_cluster(")
    fence = arrive.index("fence.release.sync_restrict::shared::cta.cluster")
    assert fence < arrive.index("mbarrier.arrive.relaxed.cluster.shared::cluster")


def test_the_issuer_acquires_at_cluster_scope():
    pair, common, tc = (source(n) for n in ("matmul_pair.cu", "matmul_common.cuh", "tc_sm100.cuh"))
    for barrier in ("ready", "dempty"):  # the two that the other CTA's threads arrive at
        waits = re.findall(r"all_wait(<true>)?\(&%s\[" % barrier, pair)
        assert waits and all(w == "<true>" for w in waits)
    assert "mbar_wait<CLUSTER>" in body(common, "bool all_wait(")
    assert "CLUSTER ? mbar_try_wait_cluster" in body(tc, "bool mbar_wait(")
    wait = body(tc, "bool mbar_try_wait_cluster(")
    poll = wait.index("mbarrier.try_wait.parity.relaxed.cluster")
    assert poll < wait.index("fence.acquire.sync_restrict::shared::cluster.cluster")
