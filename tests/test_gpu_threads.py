"""First calls from several threads at once, each on a stream of its own, in a
fresh process: the per-kernel and per-device set-up is done under a lock, and
every thread gets what one thread alone gets."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys, threading
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import deepseek_sparse_attention_score_gb300 as dsa
import dsa_inputs as DI
from gpu_util import meta_to

dev = torch.device("cuda")
wl = DI.random_small(5, [1, 1, 1], [700, 64, 1025], H=16)
meta = meta_to(wl.rg, dev)
q, kv = wl.q[0].to(dev), wl.kv[0].to(dev)
N = wl.rg.num_pages * 64
i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)
sel = torch.arange(96, dtype=torch.int32, device=dev).repeat(3, 1)
pages = torch.arange(1, dtype=torch.int32, device=dev).repeat(3, 1)
small = dict(sm_scale=wl.sm_scale)
args = (i32(N), i32(0, N), i32(0, N), torch.arange(wl.rg.num_pages, dtype=torch.int32, device=dev))
torch.cuda.synchronize()

def work(i):
    cache = torch.zeros(wl.rg.num_pages, 64, 416, dtype=torch.uint8, device=dev)
    out = []
    calls = [
        lambda: dsa.dsa_window_mla(q, kv, *meta, max_kv=1025, sliding_window=100, num_sinks=4, **small),
        lambda: dsa.dsa_sparse_mla_decode(q, kv, *meta, sel, unit=1, **small),
        lambda: dsa.dsa_dense_mla(q, kv, *meta, max_kv=1025, **small),
        lambda: dsa.dsa_build_page_tables(i32(1, 2), i32(65, 70), torch.zeros(2, 4, dtype=torch.int32, device=dev),
                                          i32(5, 6, 7), T=4, PTW=5).slots,
        lambda: dsa.dsa_sparse_mla_decode_q4(q, dsa.dsa_q4_write_back(kv.view(N, 576), cache, *args), *meta, sel, unit=1,
                                             **small),
    ]
    for k in range(len(calls)):
        j = (k + i) % len(calls)  # threads begin with different kernels
        out.append((j, calls[j]()))
    return [t for _, t in sorted(out, key=lambda e: e[0])]

got, gate = [None] * 10, threading.Barrier(10)

def run(i):
    s = torch.cuda.Stream()
    gate.wait()
    with torch.cuda.stream(s):
        got[i] = work(i)
    s.synchronize()

ts = [threading.Thread(target=run, args=(i,)) for i in range(10)]
[t.start() for t in ts]
[t.join() for t in ts]
want = work(0)
torch.cuda.synchronize()
for g in got:
    assert all(torch.equal(a, b) for a, b in zip(g, want))
print("same")
"""


def test_first_calls_from_several_threads():
    import __graft_entry__

    __graft_entry__.build()
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(root=ROOT, tests=os.path.join(ROOT, "tests"))], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout + r.stderr
