"""Rules of the memory model that the device code keeps, read from its source (a
breach need not show in any output)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "activated_mlp_gemms_gb300", "csrc")


def test_remote_arrivals_are_at_cluster_scope():
    # an arrival at another CTA's barrier synchronises with its waiter only at a scope
    # that holds both
    found = 0
    for f in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        for op in re.findall(r"mbarrier\.arrive[\w.:]*", open(f).read()):
            if "shared::cluster" not in op:
                continue
            found += 1
            assert ".release.cluster." in op or ".relaxed.cluster." in op, (os.path.basename(f), op)
            # what publishes nothing but its own transaction count may be relaxed
            assert ".relaxed." not in op or ".expect_tx." in op, (os.path.basename(f), op)
    assert found >= 2
