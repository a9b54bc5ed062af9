"""Calls of different sizes from two host threads at a time, on streams of their
own, as the first calls of a process."""
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import threading, torch
from sparse_top_kv_gb300 import hs
hs.lib()

def work(W, budget, go, out):
    g = torch.Generator(device="cuda").manual_seed(W)
    score = torch.rand(2, W, generator=g, device="cuda")
    lens = torch.full((2,), W, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    go.wait()
    for _ in range(4):
        r = hs.evict_select(score, lens, budget, score_out=torch.empty_like(score),
                            lens_out=torch.empty_like(lens), stream=stream)
        stream.synchronize()
    kept = score[0].topk(budget).values.sort().values
    out.append(bool(torch.equal(r[0][0, :budget].sort().values, kept)))

go, out = threading.Barrier(4), []
sizes = [(600, 100), (30000, 2000), (9000, 500), (260000, 3000)]
threads = [threading.Thread(target=work, args=(*s, go, out)) for s in sizes]
for t in threads: t.start()
for t in threads: t.join()
assert out == [True] * 4, out
"""


@pytest.mark.parametrize("again", range(3))
def test_selections_of_different_sizes(again):
    res = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True,
                         timeout=120, cwd=Path(__file__).resolve().parent.parent)
    assert res.returncode == 0, res.stdout + res.stderr
