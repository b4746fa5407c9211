"""Arrivals and waits across blocks name a scope that reaches the other block.

A release or an acquire within the block orders nothing for a thread outside it, and
a run that happens to come out right does not show it: the sources are read."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_decode_ffn_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu*")))


def narrow(text: str) -> list:
    """mbarrier arrivals at an address in the cluster that are not of the cluster's scope."""
    return [i for i in re.findall(r"mbarrier\.arrive[\w.:]*", text) if ".shared::cluster" in i and ".cluster.shared::cluster" not in i]


def test_it_tells_them_apart():
    wide = "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
    assert narrow(wide) == [] and narrow("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];") == []
    assert len(narrow(wide.replace("release.cluster", "release.cta"))) == 1
    assert len(narrow("mbarrier.arrive.shared::cluster.b64 _, [%0];")) == 1     # the default is the block


@pytest.mark.parametrize("path", SOURCES, ids=[os.path.basename(p) for p in SOURCES])
def test_arrivals_at_another_block_reach_it(path):
    with open(path) as f:
        assert narrow(f.read()) == []


def test_tensor_memory_is_handed_back_across_blocks():
    """The MMA thread waits for the other block's reads of an accumulator at the cluster's scope."""
    with open(os.path.join(CSRC, "moe_matmul.cu")) as f:
        waits = re.findall(r"(\w+)\(acc_empty \+ u", f.read())
    assert "mbar_wait_cluster" in waits
