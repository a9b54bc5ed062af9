"""The operators of a budgeted cache together (pipeline.BudgetedDecoder): every
step's eviction against its definition on the state that it found, the caches
row by row, and the attention over what is left against the 64-bit one."""
import math

import pytest
import torch

import paged_ref as ref
from sparse_top_kv_gb300.pipeline import BudgetedDecoder

pytestmark = pytest.mark.gpu


def rows(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("dtype,page,kvh,heads,d", [(torch.bfloat16, 16, 4, 16, 128),
                                                    (torch.float16, 5, 2, 6, 64)])
@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("prompts,budget,capacity", [([40, 7, 0, 33], 32, 48),
                                                     ([64, 63, 1, 0], 64, 65)])
def test_steps(dtype, page, kvh, heads, d, graph, prompts, budget, capacity):
    g = torch.Generator().manual_seed(budget + page)
    R, recent, sinks = len(prompts), 8, 2
    dec = BudgetedDecoder(num_reqs=R, heads=heads, kv_heads=kvh, d=d, page_size=page,
                          budget=budget, capacity=capacity, scale=1 / math.sqrt(d),
                          recent=recent, num_sinks=sinks, dtype=dtype)
    held = [dict() for _ in range(R)]  # position -> (k row, v row) of what was ever written
    for r, n in enumerate(prompts):
        if n:
            k, v = (rows(g, n, kvh, d, dtype=dtype) for _ in range(2))
            dec.start(r, k, v)
            held[r] = {i: (k[i], v[i]) for i in range(n)}
    active = [n > 0 for n in prompts]
    for step in range(40):
        if step == 20:
            dec.stop(1)
            active[1] = False
        lens, score = dec.seq_lens.tolist(), dec.score.cpu()
        pos, nxt = dec.positions.cpu(), dec.next_pos.tolist()
        q = rows(g, R, heads, d, dtype=dtype)
        k, v = (rows(g, R, kvh, d, dtype=dtype) for _ in range(2))
        if graph and step == 1:
            dec.capture()
        out, lse = dec.replay(q, k, v) if graph and step >= 1 else dec.step(q, k, v)
        torch.cuda.synchronize()
        assert int(dec.status) == 0
        for r in range(R):
            if not active[r]:
                assert int(dec.seq_lens[r]) == 0
                assert not out[r].any() and (lse[r] == -math.inf).all()
                continue
            # What the eviction kept, by its definition.
            p, s = pos[r].tolist(), score[r].tolist()
            order = sorted(range(lens[r]), key=lambda i: (
                not (p[i] < sinks or p[i] >= nxt[r] - recent), -s[i], i))
            kept = {p[i] for i in order[:budget]} | {nxt[r]}
            held[r][nxt[r]] = (k[r], v[r])
            n = int(dec.seq_lens[r])
            now = dec.positions[r, :n].tolist()
            assert n == min(lens[r], budget) + 1 and set(now) == kept and len(now) == n
            pages = dec.block_table[r].long()
            for i, t in enumerate(now):
                for cache, row in ((dec.k_cache, held[r][t][0]), (dec.v_cache, held[r][t][1])):
                    assert torch.equal(cache[pages[i // page], i % page], row)
        # The attention over the rows in their present places; the scores that
        # it started from: the kept ones moved along, 0 for the new token.
        before = torch.zeros(R, dec.capacity, device="cuda")
        for r in range(R):
            if active[r]:
                old = {p: score[r, i] for i, p in enumerate(pos[r, :lens[r]].tolist())}
                for i, t in enumerate(dec.positions[r, :int(dec.seq_lens[r])].tolist()):
                    before[r, i] = old.get(t, 0.0)
        o, l, sc, tol = ref.paged_decode(q, dec.k_cache, dec.v_cache, dec.block_table,
                                         dec.seq_lens, dec.scale, score=before)
        ref.check(out, o, tol[0], "out")
        ref.check(lse, l, tol[1], "lse")
        for r in range(R):
            m = int(dec.seq_lens[r])
            ref.check(dec.score[r, :m], sc[r, :m], tol[2][r, :m], "score")


def test_refusals():
    kw = dict(num_reqs=1, heads=4, kv_heads=2, d=64, page_size=16, scale=1.0)
    with pytest.raises(ValueError):
        BudgetedDecoder(budget=16, capacity=16, **kw)
    dec = BudgetedDecoder(budget=16, **kw)
    for n in (0, 17):
        with pytest.raises(ValueError):
            dec.start(0, torch.zeros(n, 2, 64), torch.zeros(n, 2, 64))


@pytest.mark.parametrize("kw,error", [(dict(dtype=torch.float8_e4m3fn), TypeError),
                                      (dict(dtype=torch.float32), TypeError),
                                      (dict(recent=30, num_sinks=4), ValueError),
                                      (dict(recent=-1), ValueError)])
def test_refused_at_set_up(kw, error):
    with pytest.raises(error):
        BudgetedDecoder(num_reqs=2, heads=4, kv_heads=2, d=64, page_size=16, budget=32,
                        scale=0.1, **kw)
