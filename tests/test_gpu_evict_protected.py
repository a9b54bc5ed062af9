"""hs_evict_select where more tokens are protected than the budget holds (a
`next_pos` behind the positions, or none given after earlier evictions): the
protected ones go by score, then by place, like any others."""
import numpy as np
import pytest
import torch

from sparse_top_kv_gb300 import hs

pytestmark = pytest.mark.gpu


def inputs(rows, W, fill, seed):
    g = torch.Generator().manual_seed(seed)
    score = torch.round(torch.randn(rows, W, generator=g) * 50) / 50
    if fill == "odd":
        pick = torch.randint(0, 8, (rows, W), generator=g)
        for i, x in enumerate([float("nan"), float("inf"), -float("inf"), 0.0, -0.0]):
            score[pick == i] = x
    elif fill == "equal":
        score[:] = 0.5
    elif fill == "nan":
        score[:] = float("nan")
    return score, torch.stack([torch.randperm(W, generator=g) for _ in range(rows)]).to(torch.int32)


def check(score, pos, lens, budget, recent, sinks, next_pos, in_place):
    """Bits of scores, positions, lengths and moves against the definition."""
    s, p = score.cuda(), pos.cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    nxt = None if next_pos is None else torch.tensor(next_pos, dtype=torch.int32, device="cuda")
    out = {} if in_place else dict(score_out=torch.full_like(s, 7.0), lens_out=torch.zeros_like(n),
                                   positions_out=torch.full_like(p, -5))
    so, po, lo, (src, dst, cnt) = hs.evict_select(s, n, budget, recent=recent, num_sinks=sinks,
                                                  positions=p, next_pos=nxt, **out)
    torch.cuda.synchronize()
    so, po, src, dst, cnt = (x.cpu().numpy() for x in (so, po, src, dst, cnt))
    want_s = score.numpy().copy() if in_place else np.full_like(score.numpy(), 7.0)
    want_p = pos.numpy().copy() if in_place else np.full_like(pos.numpy(), -5)
    for r, T in enumerate(lens):
        x, q = score[r, :T].numpy(), pos[r, :T].numpy()
        safe = (q < sinks) | (q >= (T if next_pos is None else next_pos[r]) - recent)
        order = np.lexsort((np.arange(T), np.isnan(x), np.where(np.isnan(x), np.inf, -x), ~safe))
        kept = np.sort(order[:budget])
        low, high = kept[kept < budget], kept[kept >= budget]
        holes = np.setdiff1d(np.arange(budget), low)
        assert int(lo[r]) == budget and cnt[r] == len(holes)
        assert np.array_equal(src[r, :len(high)], high)
        assert np.array_equal(dst[r, :len(holes)], holes)
        want_s[r, low], want_p[r, low] = x[low], q[low]
        want_s[r, budget:T] = 0.0
        want_s[r, holes], want_p[r, holes] = x[high], q[high]
    assert np.array_equal(so.view(np.int32), want_s.view(np.int32))
    assert np.array_equal(po, want_p)


# One CTA that trims a few tokens, one that selects, clusters, and slices that
# shared memory does not hold.
@pytest.mark.parametrize("W,budget", [(72, 64), (70, 64), (5000, 4996), (3000, 700), (40000, 9000),
                                      (90000, 20000), (330000, 8000)])
@pytest.mark.parametrize("fill", ["random", "odd", "equal", "nan"])
@pytest.mark.parametrize("in_place", [True, False])
def test_more_protected_than_budget(W, budget, fill, in_place):
    score, pos = inputs(3, W, fill, W)
    # From next_pos - recent on all are protected: the whole request, one more
    # than the budget, exactly the budget, one less.
    for keep in (W, budget + 1, budget, budget - 1):
        check(score, pos, [W, W - 1, budget + 1], budget, 3, 2, [W - keep + 2 + 3] * 3, in_place)


def test_positions_behind_a_length_without_next_pos():
    """next_pos NULL counts from the length, which lies far below the positions."""
    score, pos = inputs(2, 600, "random", 1)
    check(score, pos * 3, [600, 300], 256, 16, 4, None, True)
