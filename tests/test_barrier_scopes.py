"""Scopes of the barrier arrivals in the kernels' inline PTX, read from the sources."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ragged_matmul_gb300", "csrc")


def _arrivals():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            for m in re.finditer(r"mbarrier\.arrive[\w.:]*", f.read()):
                yield os.path.basename(path), m.group(0)


def test_arrivals_that_may_leave_the_cta_have_cluster_scope():
    """A release at CTA scope orders nothing for a thread of the other CTA, so an arrival on a
    cluster address names the cluster's scope (the default scope is the CTA)."""
    found = list(_arrivals())
    assert found
    for path, text in found:
        if "shared::cluster" in text:
            assert ".cluster.shared::cluster" in text, f"{path}: {text}"
