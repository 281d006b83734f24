"""Arrivals from one CTA of a cluster on another's barrier (CPU, by the source): without a scope an mbarrier
arrival releases, and a wait acquires, inside one CTA only, so what crosses has to name the cluster.  No run shows
the lack of it reliably."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_vector_quantized_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_arrivals_on_another_ctas_barrier_release_to_the_cluster():
    found = 0
    for name in sorted(os.listdir(CSRC)):
        for asm in re.findall(r"asm volatile\((.*?)\);", source(name), re.S):
            for op in re.findall(r"mbarrier\.arrive[\w.:]*", asm):
                if "shared::cluster" in op and "tcgen05.commit" not in asm:
                    found += 1
                    assert re.search(r"\.(release|relaxed)\.cluster\.", op), (name, op)
    assert found


def test_a_relaxed_arrival_carries_tensor_memory_only():
    """Ordered by the tcgen05 fences; whoever uses it has waited for its stores and fenced just before."""
    text = source("vq_chunk_wide.cu")
    head = text[text.index("auto arrive_issuer"):]
    assert "mbar_arrive_at_tmem(bar, 0)" in head[:head.index("};")] and text.count("mbar_arrive_at_tmem(") == 1
    before = r"tmem_wait_st\(\);\s*tc_fence_before\(\);\s*__syncwarp\(\);\s*if \(lane == 0\) arrive_issuer\("
    assert len(re.findall(before, text)) == len(re.findall(r"arrive_issuer\(", text)) == 2


def test_the_issuer_of_a_pair_acquires_from_the_cluster():
    assert "mbarrier.try_wait.parity.acquire.cluster." in source("vq_device.cuh")
    text = source("vq_chunk_wide.cu")
    passed = set(re.findall(r"\bpass\((\w+)", text))  # what the second CTA passes on
    assert passed == {"start", "ready"}
    issuer = text[text.index("kScores = tc_idesc"):text.index("walk.start(")]
    for bar in passed | {"q_full"}:
        assert re.search(r"\bwait_both\(" + bar + r"\b", issuer) and not re.search(r"\bwait\(" + bar + r"\b", issuer)
    # no other release arrives over there
    assert len(re.findall(r"\bmbar_arrive_at\(", text)) == 1
