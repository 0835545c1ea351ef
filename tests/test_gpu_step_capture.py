"""The serving step's calls made for the first time in a process inside a stream capture: their set-up (attributes,
occupancy) may not disturb it.  Runs as a child process, where nothing was launched before."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import torch
import mla_attention_gb300 as m
d, g = torch.device("cuda", 0), torch.Generator().manual_seed(1)
bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(d)
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=d)
ws = torch.zeros(256, dtype=torch.uint8, device=d)
xs = [bf(T, 2, 1024) for T in (1, 9, 17, 30, 40, 64)]
w4 = torch.randint(0, 256, (2, 300, 512), generator=g).to(torch.uint8).to(d)
sc = [(0.5 + torch.rand((2, 300, 1024 // k), generator=g)).to(d) for k in (32, 64, 128)]
lens, new, state = i32([5, 0, 9]), i32([1, 9000, -3]), i32([0, 700])
table = torch.full((3, 700), -1, dtype=torch.int32, device=d)
table[0, 0], table[2, 0] = 700, 701
pool = torch.arange(702, dtype=torch.int32, device=d)
x, r, w = bf(33, 512), bf(33, 512), bf(512)
c, pe, cs = bf(33, 512), bf(33, 64), torch.randn((64, 64), generator=g).to(d)
at = torch.arange(33, dtype=torch.int32, device=d)
cache = torch.zeros((3, 16, 576), dtype=torch.bfloat16, device=d)

def calls():
    out = [m.mla_bmm_w4(x, w4, s, ws=ws) for x in xs for s in sc]
    for N in (9100, 500, 20000):
        out += m.mla_slot_map(lens, new, table, pool, state, 16, N, ws=ws)
    out += m.mla_rms_norm(x, w, residual=r)[:2]
    m.mla_kv_append(c, pe, at, at, cs, cache, norm_weight=w, ws=ws)
    return out + [cache]

torch.cuda.synchronize()
G = torch.cuda.CUDAGraph()
with torch.cuda.graph(G):
    got = calls()
G.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
for a, b in zip(got, calls()):
    assert torch.equal(a, b)
print("captured ok")
"""


def test_first_calls_inside_a_capture():
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0 and "captured ok" in r.stdout, r.stdout[-1000:] + r.stderr[-3000:]
