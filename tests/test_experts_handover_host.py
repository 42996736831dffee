"""The hand-over between the two CTAs of a pair, by the source (no GPU needed): a tensor-core instruction that CTA 0 issues
reads what CTA 1 has put into its own shared memory.  Where that was written by ordinary stores, the barrier between the
CTAs has to order them: a release and an acquire at cluster scope (without a scope the instructions mean one CTA)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "qlora_block_absmax_b200", "csrc")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def function(text, name):
    """the body of an inline function, up to the closing brace in the first column"""
    at = re.search(r"\b" + name + r"\(uint64_t\* bar", text).start()
    return text[at:text.index("\n}", at)]


def test_gradient_pairs_hand_over_their_stores_at_cluster_scope():
    dx = source("gemm_experts_dx_sm100.cu")
    assert re.search(r"reinterpret_cast<uint4\*>\(arow", dx)  # the decoded tile: ordinary stores to shared memory
    told = re.findall(r"(\w+)\(&sm->peer_full\[", dx)
    arrivals = {f for f in told if "arrive" in f}
    waits = {f for f in told if "wait" in f}
    assert arrivals and waits
    common = source("experts.cuh")
    for f in arrivals:
        assert "mbarrier.arrive.release.cluster.shared::cluster.b64" in function(common, f), f
    for f in waits:
        tests = set(re.findall(r"(mbar_try_wait\w*)\(", function(common, f)))
        assert tests, f
        for t in tests:
            assert "mbarrier.try_wait.parity.acquire.cluster" in function(common, t), t
