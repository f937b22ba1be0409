"""Barriers of another CTA: every arrival there names the cluster as its scope (an arrival without a scope
orders nothing beyond its own CTA, and does not synchronise with the other CTA's wait), and every wait on a
barrier that other CTAs arrive on acquires at cluster scope."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mxfp4_mixture_experts_gb300", "csrc")


def instructions(pattern):
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        with open(path) as f:
            out += [(os.path.basename(path), m) for m in re.findall(pattern, f.read())]
    return out


def test_arrivals_on_other_ctas_name_the_cluster_scope():
    found = [(p, i) for p, i in instructions(r"mbarrier\.arrive[\w.:]*") if "shared::cluster" in i]
    assert found
    for path, i in found:
        assert ".cluster.shared::cluster" in i, (path, i)


def test_waits_that_name_the_cluster_acquire_there():
    found = [i for i in instructions(r"mbarrier\.try_wait\.parity[\w.:]*") if "cluster" in i[1]]
    assert found and all(".acquire.cluster." in i for _, i in found)
