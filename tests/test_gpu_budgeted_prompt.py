"""BudgetedDecoder: a prompt longer than the budget is cut by the attention that
its tokens have had, given or computed from the prompt's last queries."""
import math

import pytest
import torch

import paged_ref as ref
from sparse_top_kv_gb300.pipeline import BudgetedDecoder

pytestmark = pytest.mark.gpu


def decoder(dtype=torch.bfloat16, **kw):
    kw = {**dict(num_reqs=2, heads=8, kv_heads=2, d=64, page_size=16, budget=32, capacity=200,
                 scale=1 / 8, recent=4, num_sinks=2, dtype=dtype), **kw}
    return BudgetedDecoder(**kw)


def rows(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def step(dec, g):
    args = [rows(g, dec.num_reqs, h, dec.d, dtype=dec.k_cache.dtype)
            for h in (dec.heads, dec.kv_heads, dec.kv_heads)]
    dec.step(*args)
    torch.cuda.synchronize()


def kept_after(dec, r, score, n):
    """Positions that the first step keeps, by the definition, and its token's."""
    safe = [p < dec.num_sinks or p >= n - dec.recent for p in range(n)]
    order = sorted(range(n), key=lambda i: (not safe[i], -float(score[i]), i))
    return set(order[:dec.budget]) | {n}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_given_scores(dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    dec, n = decoder(dtype), 150
    score = torch.rand(n, generator=g, device="cuda")
    dec.start(0, rows(g, n, 2, 64, dtype=dtype), rows(g, n, 2, 64, dtype=dtype), score=score)
    assert torch.equal(dec.score[0, :n], score) and not dec.score[0, n:].any()
    step(dec, g)
    assert set(dec.positions[0, :33].tolist()) == kept_after(dec, 0, score, n)


@pytest.mark.parametrize("decay", [1.0, 0.9])
@pytest.mark.parametrize("n,queries", [(150, 1), (150, 100), (199, 199), (20, 7)])
def test_scores_of_the_last_queries(n, queries, decay):
    g = torch.Generator(device="cuda").manual_seed(n + queries)
    dec = decoder(score_decay=decay)
    k, v, q = rows(g, n, 2, 64), rows(g, n, 2, 64), rows(g, queries, 8, 64)
    # One token in the middle that the last query looks at.
    k[n // 2] = q[-1].view(2, 4, 64).mean(1)
    dec.start(1, k, v, q=q)
    want, bound = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
    table = dec.block_table[1:].expand(queries, -1).contiguous()
    lens = torch.arange(n - queries + 1, n + 1, dtype=torch.int32, device="cuda")
    zero = torch.zeros(queries, n, device="cuda")
    _, _, w, tol = ref.paged_decode(q, dec.k_cache, dec.v_cache, table, lens, dec.scale, score=zero)
    for j in range(queries):
        want = want * decay + w[j].cpu()
        bound = bound * decay + tol[2][j].cpu()
    # Up to 200 fp32 sums and products on top of each call's own bound.
    bound += 2.0 ** -24 * (2 * queries + 8) * want
    assert bool(((dec.score[1, :n].double().cpu() - want).abs() <= bound).all())
    assert not dec.score[1, n:].any()
    assert int(dec.seq_lens[1]) == n
    if n > dec.budget:
        found = dec.score[1, :n].clone()
        step(dec, g)
        now = set(dec.positions[1, :33].tolist())
        assert now == kept_after(dec, 1, found, n)
        # (A hundred other queries may outweigh the last one.)
        assert queries > 1 or n // 2 in now


def test_queries_of_any_layout():
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v, q = rows(g, 60, 2, 64), rows(g, 60, 2, 64), rows(g, 9, 8, 64)
    found = []
    for x in (q, q.transpose(1, 2).contiguous().transpose(1, 2), q.float().cpu()):
        dec = decoder()
        dec.start(0, k, v, q=x)
        found.append(dec.score)
    assert all(torch.equal(x, found[0]) for x in found)


def test_without_scores_the_first_places_stay():
    g = torch.Generator(device="cuda").manual_seed(3)
    dec = decoder()
    dec.start(0, rows(g, 150, 2, 64), rows(g, 150, 2, 64))
    step(dec, g)
    assert set(dec.positions[0, :33].tolist()) == set(range(28)) | {146, 147, 148, 149, 150}
