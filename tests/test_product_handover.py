"""What one CTA of a pair tells the other through its barriers, as the kernels' sources say it.

An arrival without a scope has the CTA's own: it orders nothing for a thread of another CTA, whatever the timing of a run makes of it.  So each arrival
at another CTA's barrier names the cluster's.
"""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "all_gather_tide_gb300", "csrc", "*.cu*")))
ARRIVAL = re.compile(r"mbarrier\.arrive[.:\w]*shared::cluster[.:\w]*")


def unordered(source):
    """Arrivals that may be at another CTA's barrier and do not have the cluster's scope."""
    return [x for x in ARRIVAL.findall(source) if not re.search(r"\.(release|relaxed)\.cluster\.", x)]


def test_the_search_finds_what_it_looks_for():
    assert unordered('asm("mbarrier.arrive.shared::cluster.b64 _, [%0];")') and unordered('"mbarrier.arrive.release.cta.shared::cluster.b64 _"')
    assert not unordered('"mbarrier.arrive.release.cluster.shared::cluster.b64 _" "mbarrier.arrive.shared::cta.b64 _"')


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_arrivals_at_another_cta_have_the_clusters_scope(path):
    with open(path) as f:
        source = f.read()
    assert unordered(source) == []


def test_the_products_wait_with_the_clusters_scope():
    """And so do the waits for them: the one form of a wait that the paired products use where both CTAs arrive."""
    with open(os.path.join(ROOT, "all_gather_tide_gb300", "csrc", "fp8_product_kernel.cu")) as f:
        source = f.read()
    assert ARRIVAL.search(source) and "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64" in source
    for barrier in ("scales_full[g.at]", "drained[tile & 1]", "taken"):  # those that both CTAs arrive at, as the products' thread waits for them
        assert re.search(r"wait\.both<Pair>\(&" + re.escape(barrier), source), barrier
