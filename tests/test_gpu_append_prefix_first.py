"""First calls of dsa_rope_append and dsa_prefix_mla in fresh processes: inside a
stream's capture, and from several threads at once, each with a stream and a
workspace of its own. Every call gives what a later one gives."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import sys, threading
sys.path.insert(0, {root!r})
import torch
import deepseek_sparse_attention_score_gb300 as dsa

dev = torch.device("cuda")
i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)
gen = torch.Generator().manual_seed(1)
rand = lambda *n: torch.randn(n, generator=gen).to(torch.bfloat16).to(dev)
kv, q, rows = rand(24, 64, 576), rand(3, 16, 576), rand(3, 576)
freqs = torch.linspace(1, 0.01, 32, dtype=torch.float64).to(dev)
# three requests behind 576 shared positions, the last row of each is new
first = list(range(10))
pages = i32(*first, 10, *first[:9], 11, 12, *first[:9], 13, 14)
meta = (i32(640, 640, 640), i32(0, 1, 2, 3), i32(0, 704, 1408, 2112), pages)
slots, pos = i32(9 * 64 + 63, 11 * 64 + 63, 13 * 64 + 63), i32(639, 639, 639)
prefix = i32(576)

def step(cache, ws, o, lse):
    dsa.dsa_rope_append([dsa.AppendTarget(rows, cache, rot_off=512)], pos, slots, freqs)
    dsa.dsa_prefix_mla(q, cache, *meta, prefix, max_kv=640, sm_scale=0.07, o=o, lse=lse, ws=ws)

def buffers():
    n = dsa.dsa_prefix_mla_workspace_size(3, 16, 1)
    return (kv.clone(), torch.zeros(n, dtype=torch.uint8, device=dev),
            torch.zeros(3, 16, 512, dtype=torch.bfloat16, device=dev), torch.zeros(3, 16, device=dev))

def same(a, b):
    assert all(torch.equal(x, y) for x, y in zip((a[0], a[2], a[3]), (b[0], b[2], b[3])))
"""

CAPTURE = SETUP + """
got, want = buffers(), buffers()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step(*got)
g.replay()
step(*want)
torch.cuda.synchronize()
same(got, want)
assert got[3].isfinite().all() and not torch.equal(got[0], kv)
print("as one")
"""

THREADS = SETUP + """
bufs, gate = [buffers() for _ in range(8)], threading.Barrier(8)
torch.cuda.synchronize()

def run(i):
    s = torch.cuda.Stream()
    gate.wait()
    with torch.cuda.stream(s):
        step(*bufs[i])
    s.synchronize()

ts = [threading.Thread(target=run, args=(i,)) for i in range(8)]
[t.start() for t in ts]
[t.join() for t in ts]
want = buffers()
step(*want)
torch.cuda.synchronize()
for b in bufs:
    same(b, want)
print("as one")
"""


@pytest.mark.parametrize("program", [CAPTURE, THREADS], ids=["capture", "threads"])
def test_first_calls(program):
    import __graft_entry__

    __graft_entry__.build()
    out = subprocess.run([sys.executable, "-c", program.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "as one" in out.stdout, out.stdout + out.stderr
