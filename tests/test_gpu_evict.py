"""hs_evict_select / hs_evict_move / hs_evict against their definition, token
by token on the CPU (exact: choices and copies)."""
import numpy as np
import pytest
import torch

from sparse_top_kv_gb300 import hs

pytestmark = pytest.mark.gpu


def oracle(score, T, budget, recent, sinks, positions, next_pos):
    """Kept places and moves [(src, dst)] of one request."""
    if T <= budget:
        return list(range(T)), []
    def rank(i):
        p = positions[i]
        s = float(score[i])
        return (0 if p < sinks or p >= next_pos - recent else 1,
                float("inf") if s != s else -s, 1 if s != s else 0, i)
    kept = sorted(sorted(range(T), key=rank)[:budget])
    holes = [i for i in range(budget) if i not in set(kept)]
    return kept, list(zip([i for i in kept if i >= budget], holes))


def check(score, lens, budget, *, recent=0, sinks=0, positions=None, next_pos=None, max_len=None,
          in_place=True, **kw):
    R, W = score.shape
    dev = "cuda"
    ds, dl = score.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    dp = None if positions is None else positions.to(dev)
    dn = None if next_pos is None else torch.tensor(next_pos, dtype=torch.int32, device=dev)
    out = {}
    if not in_place:
        out = dict(score_out=torch.full_like(ds, 77.0), lens_out=torch.full_like(dl, -9),
                   positions_out=torch.full((R, W), -5, dtype=torch.int32, device=dev))
    s_in, p_in = ds.clone(), None if dp is None else dp.clone()
    so, po, lo, (src, dst, cnt) = hs.evict_select(ds, dl, budget, recent=recent, num_sinks=sinks,
                                                  positions=dp, next_pos=dn, max_len=max_len,
                                                  **out, **kw)
    torch.cuda.synchronize()
    so, lo, src, dst, cnt = (x.cpu() for x in (so, lo, src, dst, cnt))
    po = None if po is None else po.cpu()
    want_s = score.clone() if in_place else torch.full_like(score, 77.0)
    base_p = (positions if positions is not None else
              torch.arange(W, dtype=torch.int32).expand(R, W))
    want_p = base_p.clone() if in_place else torch.full((R, W), -5, dtype=torch.int32)
    for r, n in enumerate(lens):
        T = min(max(n, 0), W if max_len is None else max_len)
        kept, moves = oracle(score[r].numpy(), T, budget, recent, sinks, base_p[r].tolist(),
                             next_pos[r] if next_pos is not None else T)
        assert lo[r] == min(T, budget) and cnt[r] == len(moves), (r, n)
        assert src[r, :len(moves)].tolist() == [m[0] for m in moves]
        assert dst[r, :len(moves)].tolist() == [m[1] for m in moves]
        for i in kept:
            if i < budget:
                want_s[r, i], want_p[r, i] = score[r, i], base_p[r, i]
        if T > budget:
            want_s[r, budget:T] = 0.0
        for a, b in moves:
            want_s[r, b], want_p[r, b] = score[r, a], base_p[r, a]
    assert torch.equal(so.view(torch.int32), want_s.view(torch.int32))
    if po is not None:
        assert torch.equal(po, want_p)
    if not in_place:
        assert torch.equal(ds.view(torch.int32), s_in.view(torch.int32))
        assert dp is None or torch.equal(dp, p_in)
    return src, dst, cnt


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lens,budget,recent,sinks", [
    ([9], 8, 0, 0), ([9, 8, 0, 1, -3], 8, 4, 4), ([100, 33, 64, 65], 64, 16, 4),
    ([1000, 17, 999], 1, 0, 0), ([1000, 513], 500, 500, 0), ([5000, 4999, 2049], 2048, 256, 4),
    ([2049] * 9, 2048, 0, 0), ([20000, 3], 19999, 5, 0), ([40000, 39999], 100, 50, 50)])
def test_select(lens, budget, recent, sinks, in_place):
    g = torch.Generator().manual_seed(budget)
    W = max(max(lens), 1) + 3
    score = torch.rand(len(lens), W, generator=g)
    score[torch.rand(len(lens), W, generator=g) < 0.2] = 0.0
    positions = torch.stack([torch.randperm(W, generator=g) * 2 for _ in lens]).to(torch.int32)
    next_pos = [2 * W + 1] * len(lens)
    check(score, lens, budget, recent=recent, sinks=sinks, in_place=in_place)
    check(score, lens, budget, recent=recent, sinks=sinks, in_place=in_place,
          positions=positions, next_pos=next_pos)


@pytest.mark.parametrize("fill", ["equal", "zeros", "nan", "mixed", "ordered", "negative"])
def test_ties_and_odd_scores(fill):
    g = torch.Generator().manual_seed(1)
    W = 3001
    score = torch.randn(3, W, generator=g)
    if fill == "equal":
        score[:] = 0.25
    elif fill == "zeros":
        score = torch.where(score > 0, 0.0, -0.0)
    elif fill == "nan":
        score[:] = float("nan")
    elif fill == "mixed":
        pick = torch.randint(0, 6, (3, W), generator=g)
        for i, x in enumerate([float("nan"), float("inf"), -float("inf"), 3.4e38, 1e-45]):
            score[pick == i] = x
    elif fill == "ordered":
        score = torch.arange(W).float().expand(3, W).clone()
    elif fill == "negative":
        score = -score.abs()
    for budget in (1, 700, 3000):
        check(score, [W, 1500, 701], budget)
        check(score, [W, 1500, 701], budget, recent=min(budget, 33))


@pytest.mark.parametrize("rows,W,budget", [(1, 131072, 2048), (2, 300000, 70000), (3, 33000, 32999),
                                           (200, 700, 512), (1, 400000, 399999)])
def test_long_and_wide(rows, W, budget):
    """Clusters of every size, slices that shared memory does not hold."""
    g = torch.Generator(device="cuda").manual_seed(W)
    score = torch.rand(rows, W, generator=g, device="cuda")
    score = torch.where(score < 0.3, 0.0, torch.round(score * 5000) / 5000)
    lens = torch.full((rows,), W, dtype=torch.int32, device="cuda")
    before = score.clone()
    so, _, lo, (src, dst, cnt) = hs.evict_select(score, lens, budget, recent=64, num_sinks=4)
    torch.cuda.synchronize()
    key = before.cpu().numpy().astype(np.float64)
    for r in range(rows):
        k = key[r].copy()
        k[:4] = k[W - 64:] = np.inf
        kept = np.sort(np.lexsort((np.arange(W), -k))[:budget])
        holes = np.setdiff1d(np.arange(budget), kept)
        n = int(cnt[r])
        assert int(lo[r]) == budget and n == len(holes)
        assert (src[r, :n].cpu().numpy() == kept[kept >= budget]).all()
        assert (dst[r, :n].cpu().numpy() == holes).all()
        want = np.zeros(W)
        want[kept[kept < budget]] = key[r][kept[kept < budget]]
        want[holes] = key[r][kept[kept >= budget]]
        assert (so[r].cpu().numpy() == want).all()


def caches(pages, page, kvh, d, dtype, n=2):
    g = torch.Generator(device="cuda").manual_seed(pages)
    bits = [torch.randint(0, 255, (pages, page, kvh, d * dtype.itemsize), generator=g,
                          device="cuda", dtype=torch.uint8) for _ in range(n)]
    return [b.view(dtype) for b in bits]


def same_bits(a, b):
    """Random bytes hold NaN codes, which differ from themselves as numbers."""
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype,page,kvh,d", [(torch.bfloat16, 16, 8, 128),
                                              (torch.bfloat16, 64, 1, 576),
                                              (torch.float8_e4m3fn, 7, 3, 64),
                                              (torch.uint8, 1, 1, 656),
                                              (torch.float16, 32, 12, 64)])
@pytest.mark.parametrize("layout", ["packed", "heads_first", "single"])
def test_moves(dtype, page, kvh, d, layout):
    lens, budget = [500, 20, 0, 333, 201], 200
    R, W = len(lens), 512
    blocks = -(-W // page)
    g = torch.Generator().manual_seed(3)
    score = torch.rand(R, W, generator=g).cuda()
    table = torch.randperm(R * blocks + 2, generator=g)[:R * blocks].view(R, blocks)
    table = table.to(torch.int32).cuda()
    k, v = caches(R * blocks + 2, page, kvh, d, dtype)
    if layout == "heads_first":
        k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
    if layout == "single":
        v = None
    raw = [None if c is None else c.contiguous().view(torch.uint8).clone() for c in (k, v)]
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moves = hs.evict(score, dl, budget, k, v, table, recent=10, num_sinks=2, status=status)[3]
    torch.cuda.synchronize()
    assert int(status) == 0 and dl.tolist() == [min(n, budget) for n in lens]
    src, dst, cnt = (m.cpu() for m in moves)
    assert cnt.sum() > 0
    tab = table.cpu()
    for c, old in zip((k, v), raw):
        if c is None:
            continue
        want = old.clone()
        for r in range(R):
            s, t = src[r, :cnt[r]].long(), dst[r, :cnt[r]].long()
            want[tab[r][t // page].long(), t % page] = old[tab[r][s // page].long(), s % page]
        assert torch.equal(c.contiguous().view(torch.uint8), want)
        hs.evict_move(moves, k, v, table)  # again: nothing changes
        assert torch.equal(c.contiguous().view(torch.uint8), want)


def test_bad_pages_are_skipped_and_reported():
    score = torch.arange(64.0, device="cuda").view(1, 64).contiguous()  # keeps the last ones
    k, v = caches(8, 16, 2, 64, torch.bfloat16)
    table = torch.tensor([[0, 1, 8, 3]], dtype=torch.int32, device="cuda")
    old = k.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([64], dtype=torch.int32, device="cuda")
    hs.evict(score, lens, 32, k, v, table, status=status)
    torch.cuda.synchronize()
    assert int(status) == 6
    want = old.clone()
    want[1] = old[3]  # places 48..63 -> 16..31; 32..47 stood on the bad page
    assert same_bits(k, want)


def test_longer_than_max_len_is_cut_and_reported():
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(0)
    check(torch.rand(2, 50, generator=g), [45, 20], 16, max_len=40, status=status)
    assert int(status) == 6


def test_captured_step_and_other_stream():
    """A step captured once and replayed at other lengths and scores."""
    R, W, B = 4, 80, 64
    k, v = caches(R * 5, 16, 2, 64, torch.bfloat16)
    table = torch.arange(R * 5, dtype=torch.int32, device="cuda").view(R, 5)
    score = torch.zeros(R, W, device="cuda")
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    moves = tuple(torch.zeros(*s, dtype=torch.int32, device="cuda") for s in ((R, B), (R, B), (R,)))
    side = torch.cuda.Stream()
    hs.evict(score, lens, B, k, v, table, moves=moves, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs.evict(score, lens, B, k, v, table, moves=moves)
    g = torch.Generator().manual_seed(1)
    for n in ([65, 64, 80, 0], [70, 3, 65, 66]):
        s = torch.rand(R, W, generator=g)
        score.copy_(s)
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        old = k.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [min(x, B) for x in n]
        for r in range(R):
            _, mv = oracle(s[r].numpy(), n[r], B, 0, 0, list(range(W)), n[r])
            assert int(moves[2][r]) == len(mv)
            for a, b in mv:
                assert same_bits(k[table[r, b // 16].long(), b % 16],
                                 old[table[r, a // 16].long(), a % 16])


@pytest.mark.parametrize("change,error", [
    ("score64", TypeError), ("cpu", ValueError), ("narrow", ValueError), ("positions", TypeError),
    ("lens", ValueError), ("cap", hs.HSError), ("protected", hs.HSError), ("budget", hs.HSError),
    ("rows16", hs.HSError), ("table", hs.HSError), ("v", ValueError)])
def test_refusals(change, error):
    score = torch.zeros(2, 64, device="cuda")
    lens = torch.tensor([64, 3], dtype=torch.int32, device="cuda")
    k, v = caches(8, 16, 2, 64, torch.bfloat16)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    kw, budget = {}, 32
    if change == "score64":
        score = score.double()
    elif change == "cpu":
        lens = lens.cpu()
    elif change == "narrow":
        kw["max_len"] = 65
    elif change == "positions":
        kw["positions"] = torch.zeros(2, 64, dtype=torch.int64, device="cuda")
    elif change == "lens":
        lens = lens[:1]
    elif change == "cap":
        kw["moves"] = tuple(torch.zeros(*s, dtype=torch.int32, device="cuda")
                            for s in ((2, 31), (2, 31), (2,)))
    elif change == "protected":
        kw.update(recent=30, num_sinks=3)
    elif change == "budget":
        budget = 0
    elif change == "rows16":
        k, v = (x[..., :60].contiguous() for x in (k, v))
    elif change == "table":
        table = table[:, :3].contiguous()
    elif change == "v":
        v = v[:4]
    with pytest.raises(error):
        hs.evict(score, lens, budget, k, v, table, **kw)


@pytest.mark.parametrize("budget,over", [(1024, 8), (5, 8), (2048, 1), (4100, 8), (1, 3)])
@pytest.mark.parametrize("fill", ["random", "equal", "nan"])
def test_a_few_tokens_over(budget, over, fill):
    """Requests at most a few tokens over the budget (a decode step's case)."""
    W = budget + over
    g = torch.Generator().manual_seed(W)
    lens = [W, budget, budget + 1, 0, max(1, budget - 3), W - 1, W]
    score = torch.rand(len(lens), W, generator=g)
    if fill == "equal":
        score[:] = -1.0
    elif fill == "nan":
        score[torch.rand(len(lens), W, generator=g) < 0.5] = float("nan")
    positions = torch.stack([torch.randperm(W, generator=g) * 3 for _ in lens]).to(torch.int32)
    for in_place in (True, False):
        check(score, lens, budget, in_place=in_place)
        check(score, lens, budget, recent=budget // 2, sinks=budget // 4, in_place=in_place,
              positions=positions, next_pos=[3 * W + 1] * len(lens))


@pytest.mark.parametrize("layout", ["packed", "heads_first", "single"])
def test_a_few_tokens_over_moves(layout):
    R, B, W, page = 6, 40, 48, 16
    k, v = caches(R * 3 + 1, page, 3, 64, torch.bfloat16)
    if layout == "heads_first":
        k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
    if layout == "single":
        v = None
    g = torch.Generator().manual_seed(5)
    table = torch.randperm(R * 3, generator=g).view(R, 3).to(torch.int32).cuda()
    table[4, 2] = 99  # a bad page: its rows are skipped and reported
    score = torch.rand(R, W, generator=g).cuda()
    score[4, 40:] = 9.0
    lens = torch.tensor([48, 41, 40, 0, 48, 45], dtype=torch.int32, device="cuda")
    old = [None if c is None else c.contiguous().clone() for c in (k, v)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    src, dst, cnt = (m.cpu() for m in hs.evict(score, lens, B, k, v, table, status=status)[3])
    assert int(status) == 6 and cnt.tolist()[2:4] == [0, 0] and cnt[4] == 8
    tab = table.cpu()
    for c, was in zip((k, v), old):
        if c is None:
            continue
        want = was.clone()
        for r in (0, 1, 5):
            for s, t in zip(src[r, :cnt[r]].tolist(), dst[r, :cnt[r]].tolist()):
                want[tab[r, t // page].long(), t % page] = was[tab[r, s // page].long(), s % page]
        assert same_bits(c, want)


@pytest.mark.parametrize("given", ["all", "least"])
def test_extension_and_general_path_agree(given, monkeypatch):
    hs.lib()
    if hs._binding is None:
        pytest.skip("Python headers were not there at build time")
    taken = []

    class Spy:
        def evict(self, *a):
            taken.append(binding.evict(*a))
            return taken[-1]

    binding = hs._binding
    R, W, B, page = 5, 96, 40, 16
    g = torch.Generator().manual_seed(8)
    first = torch.rand(R, W, generator=g)
    table = torch.randperm(R * 6, generator=g).view(R, 6).to(torch.int32).cuda()
    base = caches(R * 6, page, 2, 64, torch.bfloat16)
    got = []
    for mod in (Spy(), None):
        monkeypatch.setattr(hs, "_binding", mod)
        k, v = (c.clone() for c in base)
        score = first.cuda()
        lens = torch.tensor([96, 41, 40, 0, 70], dtype=torch.int32, device="cuda")
        moves = tuple(torch.zeros(*s, dtype=torch.int32, device="cuda")
                      for s in ((R, B), (R, B), (R,)))
        kw = {}
        if given == "all":
            kw = dict(max_len=W, recent=5, num_sinks=2, score_out=torch.ones(R, W, device="cuda"),
                      positions=torch.arange(W, dtype=torch.int32, device="cuda").repeat(R, 1),
                      next_pos=lens.clone(), lens_out=torch.empty_like(lens),
                      positions_out=torch.zeros(R, W, dtype=torch.int32, device="cuda"),
                      status=torch.zeros(1, dtype=torch.int32, device="cuda"))
        r = hs.evict(score, lens, B, k, v, table, moves=moves, **kw)
        torch.cuda.synchronize()
        got.append([x for x in (*r[:3], *moves, k, v) if x is not None])
        assert r[0] is kw.get("score_out", score) and r[2] is kw.get("lens_out", lens)
    assert taken == [0]
    for a, b in zip(*got):
        assert same_bits(a, b)
    monkeypatch.setattr(hs, "_binding", Spy())
    with pytest.raises(hs.HSError):
        hs.evict(first.cuda(), lens, 0, k, v, table, moves=moves)
    assert taken[-1] == 1


@pytest.mark.parametrize("kw", [dict(budget=(1 << 32) + 8), dict(recent=1 << 32),
                                dict(num_sinks=1 << 31), dict(max_len=(1 << 32) + 16)])
def test_sizes_past_32_bits_are_refused(kw):
    score = torch.zeros(2, 64, device="cuda")
    lens = torch.tensor([64, 3], dtype=torch.int32, device="cuda")
    k, v = caches(8, 16, 2, 64, torch.bfloat16)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    kw = {**dict(budget=16), **kw}
    budget = kw.pop("budget")
    with pytest.raises(ValueError):
        hs.evict(score, lens, budget, k, v, table, **kw)
    with pytest.raises(ValueError):
        hs.evict_select(score, lens, budget, **kw)


def test_memory_of_a_call_on_another_stream():
    """The move lists that a call makes for itself are not handed out again
    while the other stream still works with them."""
    R, W, B = 4, 256, 64
    g = torch.Generator().manual_seed(9)
    score, (k, v) = torch.rand(R, W, generator=g).cuda(), caches(R * 16, 16, 2, 64, torch.bfloat16)
    table = torch.arange(R * 16, dtype=torch.int32, device="cuda").view(R, 16)
    results = []
    for stream in (None, torch.cuda.Stream()):
        s, kc, vc = score.clone(), k.clone(), v.clone()
        lens = torch.full((R,), W, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(40_000_000)
        hs.evict(s, lens, B, kc, vc, table, stream=stream)
        junk = [torch.full((R, B), -1, dtype=torch.int32, device="cuda") for _ in range(6)]
        torch.cuda.synchronize()
        results.append((s, lens, kc, vc))
        assert len(junk) == 6
    for a, b in zip(*results):
        assert same_bits(a, b)


@pytest.mark.parametrize("given", ["none", "positions", "outputs"])
@pytest.mark.parametrize("lens,budget", [([300, 64, 65, 0, 200, 128], 64), ([5000], 1000),
                                         ([20000, 9000, 40000], 2048), ([900] * 40, 450)])
def test_both_steps_in_one_call(lens, budget, given):
    """hs_evict moves scores and positions along with the rows; hs_evict_select
    moves them itself."""
    R, W, page = len(lens), max(lens) + 3, 16
    g = torch.Generator().manual_seed(R + budget)
    blocks = -(-W // page)
    score = torch.rand(R, W, generator=g)
    score[:, ::7] = score[:, 1:2]
    pos = torch.stack([torch.randperm(W, generator=g) for _ in range(R)]).to(torch.int32)
    k, v = caches(R * blocks, page, 2, 64, torch.bfloat16)
    table = torch.randperm(R * blocks, generator=g).to(torch.int32).view(R, blocks).cuda()
    results = []
    for split in (False, True):
        s, kc, vc = score.cuda(), k.clone(), v.clone()
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        kw = dict(recent=20, num_sinks=3)
        if given != "none":
            kw.update(positions=pos.cuda(),
                      next_pos=torch.full((R,), W, dtype=torch.int32, device="cuda"))
        if given == "outputs":
            kw.update(score_out=torch.full_like(s, 5.0), lens_out=torch.full_like(ln, -7),
                      positions_out=torch.full((R, W), -3, dtype=torch.int32, device="cuda"))
        if split:
            so, po, lo, moves = hs.evict_select(s, ln, budget, **kw)
            hs.evict_move(moves, kc, vc, table)
        else:
            so, po, lo, moves = hs.evict(s, ln, budget, kc, vc, table, **kw)
        torch.cuda.synchronize()
        results.append([s, so, lo, moves[2], kc, vc] + ([] if po is None else [po]))
    assert int(results[0][3].sum()) > 0
    for a, b in zip(*results):
        assert same_bits(a, b)
