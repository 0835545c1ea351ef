"""The smaller cache's calls through the guarded build (see test_gpu_guarded.py): no check fires and the
results match the oracle."""
import os
import subprocess
import sys

import pytest

from mla_attention_gb300 import build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_guarded_build_runs_the_smaller_cache_clean():
    path = build.build(guard=True)
    r = subprocess.run([sys.executable, os.path.join(HERE, "guarded_cache_cases.py"), path], capture_output=True,
                       text=True, timeout=900, cwd=os.path.dirname(HERE))
    assert r.returncode == 0 and "guarded ok" in r.stdout, (r.stdout[-3000:] + r.stderr[-3000:])
