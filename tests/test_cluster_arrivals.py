"""Arrivals on a barrier of another CTA say what they order (read from the sources; CPU only): without a scope they are released
to their own CTA alone, in which nobody waits for them."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_attention_gb300", "csrc")


def test_every_remote_arrival_has_the_clusters_scope():
    found = 0
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            for how in re.findall(r"mbarrier\.arrive([a-z_:.]*)\.shared::cluster\.b64 _", f.read()):
                found += 1
                assert how.endswith(".cluster"), (name, how)
    assert found >= 2
