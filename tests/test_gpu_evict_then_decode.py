"""hs.evict and hs.paged_decode queued behind each other with nothing between
them: the attention kernel may start while the eviction still runs, and has to
see the lengths and rows that the eviction leaves (updated in place)."""
import math

import pytest
import torch

import paged_ref as ref
from sparse_top_kv_gb300 import hs

pytestmark = pytest.mark.gpu

# rows, heads, kv_heads, page, tokens, budget: one CTA that trims or clusters that
# select, then attention in clusters, dealt, or on the warp-level kernel.
CASES = {"trim_cluster": (40, 16, 2, 16, 68, 64), "trim_dealt": (64, 32, 8, 64, 2052, 2048),
         "trim_warps": (8, 8, 8, 12, 1004, 1000), "select_dealt": (40, 32, 8, 16, 3000, 700),
         "select_warps": (3, 8, 2, 64, 20000, 4000), "select_cluster": (4, 32, 2, 16, 5000, 100)}


@pytest.mark.parametrize("case", list(CASES))
@pytest.mark.parametrize("graph", [False, True])
def test_pair(case, graph):
    R, heads, kvh, page, T, B = CASES[case]
    d, scale, blocks = 128, 1 / math.sqrt(128), -(-T // page)
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    q, k0, v0 = rnd(R, heads, d), rnd(R * blocks, page, kvh, d), rnd(R * blocks, page, kvh, d)
    table = torch.randperm(R * blocks, generator=g, device="cuda").to(torch.int32).view(R, blocks)
    score0 = torch.rand(R, T, generator=g, device="cuda")
    full = torch.full((R,), T, dtype=torch.int32, device="cuda")
    full[R // 2] = B // 2
    k, v, score, lens = k0.clone(), v0.clone(), score0.clone(), full.clone()
    cap = min(B, T - B)
    moves = tuple(torch.zeros(*s, dtype=torch.int32, device="cuda") for s in ((R, cap), (R, cap), (R,)))
    out, lse = torch.empty_like(q), torch.empty(R, heads, device="cuda")
    ws = torch.empty(hs.paged_decode_workspace_bytes(R, heads, kvh, d, T, with_score=True),
                     dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def reset():
        for x, y in ((k, k0), (v, v0), (score, score0), (lens, full)):
            x.copy_(y)

    def evict():
        hs.evict(score, lens, B, k, v, table, moves=moves, status=status)

    def decode():
        hs.paged_decode(q, k, v, table, lens, scale, max_len=T, score=score, out=out, lse=lse,
                        workspace=ws, status=status)

    reset()
    evict()
    torch.cuda.synchronize()
    o, l, sc, tol = ref.paged_decode(q, k, v, table, lens, scale, score=score)
    decode()
    torch.cuda.synchronize()
    ref.check(out, o, tol[0], "out")
    ref.check(lse, l, tol[1], "lse")
    ref.check(score, sc, tol[2], "score")
    want = [x.clone() for x in (out, lse, score, lens, k, v)]

    def steps():
        reset()
        decode()  # over the whole context: leaves its lengths in every cache
        score.copy_(score0)
        evict()
        decode()
        evict()   # nothing left to give up
        return [x.clone() for x in (out, lse, score, lens, k, v)]

    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            got = steps()
    for _ in range(20):
        if graph:
            captured.replay()
        else:
            got = steps()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert int(status) == 0
