"""Arrivals at another CTA's barrier name the cluster as their scope, and what they hand
over from the arriving CTA's shared memory is released and acquired at that scope: the
CTA's own scope gives no order between two CTAs."""
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "mxfp4_routed_expert_select_gb300", "csrc")


def _sources():
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as fh:
            yield name, fh.read()


def test_arrivals_at_the_other_cta_have_cluster_scope():
    found = 0
    for name, text in _sources():
        for instr in re.findall(r"mbarrier\.arrive[\w.:]*\.shared::cluster[\w.:]*", text):
            if "::complete_tx" in instr:  # a copy's completion, not a thread's arrival
                continue
            found += 1
            assert ".cluster.shared::cluster" in instr, (name, instr)
    assert found >= 2


def test_staged_tiles_are_released_and_acquired():
    for name, text in _sources():
        kernels = text.count("pair_arrive(bar(")
        assert not kernels or "pair_acquire()" in text, name
    text = dict(_sources())["k3_tmem.cuh"]
    body = text[text.index("void pair_arrive("):]
    body = body[:body.index("\n}")]
    assert body.index("fence.release.sync_restrict::shared::cta.cluster") < body.index("mbarrier.arrive.relaxed.cluster")
