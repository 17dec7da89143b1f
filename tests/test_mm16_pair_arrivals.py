"""CPU: what one CTA of a pair leaves in its shared memory for MMAs that the other one issues is handed over in order at cluster
scope. The plain arrival on another CTA's barrier orders at CTA scope alone."""
import os
import re

from conftest import ROOT

TEXT = re.sub(r'"\s*"', "", open(os.path.join(ROOT, "quantized_moe_gb300", "csrc", "mm16_tc.cu")).read())


def body(name):
    return re.search(r"void " + name + r"\([^)]*\) \{(.*?)\n\}\n", TEXT, re.S).group(1)


def test_the_arrival_releases_and_the_wait_acquires_at_cluster_scope():
    arrive, acquire = body("mbar_arrive_leader"), body("mbar_acquire_pair")
    assert arrive.index("fence.release.sync_restrict::shared::cta.cluster") < arrive.index("mbarrier.arrive.relaxed.cluster.shared::cluster")
    assert acquire.index("mbarrier.test_wait.parity.relaxed.cluster") < acquire.index("fence.acquire.sync_restrict::shared::cluster.cluster")


def test_every_arrival_on_the_cleaners_barrier_of_the_leader_is_such_a_one():
    assert re.findall(r"(\w+)\(mapa\(su32\(clean ", TEXT) == ["mbar_arrive_leader"]
    wait = TEXT.index("mbar_wait(clean + s")
    assert TEXT.index("mbar_acquire_pair(clean + s", wait) < TEXT.index("mma<CG>(d,", wait)
    # the other arrivals on a leader's barrier hand accumulators back, with which no memory goes
    assert set(re.findall(r"mbar_arrive_cluster\(mapa\(su32\((\w+)", TEXT)) == {"acc_empty"}
