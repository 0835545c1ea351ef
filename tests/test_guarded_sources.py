"""Every check of the guarded build has a status word to record in (read from the sources; CPU only)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_attention_gb300", "csrc")


def test_every_guard_has_a_status_word():
    """A check without one skips the access and tells nobody."""
    calls = 0
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            for word in re.findall(r"(?<!bool )guard_span\(([^,()]+(?:\([^()]*\))?),", f.read()):
                calls += 1
                assert word.strip() not in ("nullptr", "0", "NULL"), name
    assert calls > 50
