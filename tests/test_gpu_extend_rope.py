"""hs.paged_extend (bit-exact) and hs.rope_append against plain definitions."""
import math
import random

import pytest
import torch

import step_ref

pytestmark = pytest.mark.gpu

BF, FP, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def extend(new, lens, table, ring, ends, page, max_tokens, in_place=False):
    from sparse_top_kv_gb300 import hs
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.tensor(table, **i32).view(len(new), len(table[0]) if table else 0)
    ring, lens = torch.tensor(ring, **i32), torch.tensor(lens, **i32)
    ends = torch.tensor(ends, dtype=torch.int64, device="cuda")
    status = torch.zeros(1, **i32)
    ends_out = ends if in_place else torch.zeros_like(ends)
    lens_out, attend, cu, slot, req, pos = hs.paged_extend(
        torch.tensor(new, **i32), lens, table, ring, ends, page, max_tokens,
        lens_out=None if in_place else torch.zeros_like(lens), ring_out=ends_out, status=status)
    return [x.tolist() for x in (table, ring, ends_out, lens_out, attend, cu, slot, req, pos)] + [
        status.item()]


def compare(new, lens, table, ring, ends, page, max_tokens):
    want = step_ref.extend(new, lens, table, ring, ends, page, max_tokens)
    for in_place in (False, True):
        got = extend(new, lens, table, ring, ends, page, max_tokens, in_place)
        names = "table ring ends lens attend cu slot row pos".split()
        for name, a, b in zip(names, got, want):
            assert a == b, name
        assert got[-1] == want[-1]


def state(rng, rows, page, blocks, spare, most):
    lens = [rng.randrange(0, min(most, blocks * page) + 1) for _ in range(rows)]
    held = [-(-t // page) for t in lens]
    pages = sum(held) + spare
    perm = list(range(pages))
    rng.shuffle(perm)
    table, at = [], 0
    for h in held:
        table.append(perm[at:at + h] + [-1] * (blocks - h))
        at += h
    ring, start = [-1] * pages, rng.randrange(0, 1 << 40)
    for i in range(spare):
        ring[(start + i) % pages] = perm[at + i]
    return lens, table, ring, [start, start + spare]


@pytest.mark.parametrize("rows", [1, 2, 7, 33, 300, 4096])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_extend_random(rows, page):
    rng = random.Random(rows * 100 + page)
    for spare in (0, 1, 5, rows, 40 * rows):
        lens, table, ring, ends = state(rng, rows, page, 12, max(1, spare), 10 * page)
        new = [rng.choice([0, 1, 1, 1, 3, -1, -2, -10 ** 9, page, 5 * page, rng.randrange(1, 99)])
               for _ in range(rows)]
        total = sum(max(0, n) for n in new)
        for cap in {total, total + 7, max(0, total - 3), total // 2}:
            compare(new, lens, table, ring, ends, page, cap)


def test_extend_edges():
    compare([5], [0], [[-1] * 3], [4, 9, 2], [0, 3], 2, 5)       # exactly the ring
    compare([7], [0], [[-1] * 3], [4, 9, 2], [0, 3], 2, 9)       # past the table
    compare([5, 1], [0, 1], [[-1] * 4, [8, -1, -1, -1]], [4, 9, 2], [0, 2], 2, 9)  # first refused
    compare([-3, 4], [3, 0], [[0, 1], [-1, -1]], [2, 2], [7, 7], 2, 4)  # given back, not taken at once
    compare([2 ** 31 - 1, 1], [4, 1], [[0, 1], [2, -1]], [5, 3, 3], [3, 4], 2, 3)
    compare([0, 0], [-5, 2], [[-1, -1], [1, -1]], [0, 0], [0, 1], 2, 0)
    compare([5], [0], [[-1] * 3], [1, 0, 2], [2, 5], 2, 5)
    compare([5, 1], [0, 1], [[-1] * 4, [2, -1, -1, -1]], [0, 1, 0], [0, 2], 2, 9)
    compare([-3, 4], [3, 0], [[0, 1], [-1, -1]], [1, 0], [7, 7], 2, 4)
    assert extend([], [], [], [1, 2], [0, 2], 4, 3)[:-1] == [
        [], [1, 2], [0, 2], [], [], [0], [-1] * 3, [-1] * 3, [-1] * 3]


def test_extend_impossible_states_change_nothing():
    for ends in ([5, 2], [0, 9], [-3, 0]):
        got = extend([3, -2], [2, 2], [[0, -1, -1], [1, -1, -1]], [4, 5, 6], ends, 2, 3)
        assert got[-1] == 6 and got[2] == ends and got[3] == [2, 2] and got[1] == [4, 5, 6]
    got = extend([1, 1], [99, 2], [[0, -1], [1, -1]], [4, 5, 6], [0, 3], 2, 2)  # past its table
    assert got[-1] == 6 and got[3] == [99, 3] and got[4] == [0, 3] and got[6][0] == -1
    got = extend([-4], [4], [[0, 1]], [4, 5, 6], [0, 2], 2, 0)  # more than the ring holds
    assert got[-1] == 6 and got[3] == [4] and got[2] == [0, 2]
    got = extend([1], [1], [[77]], [4, 5, 6], [0, 3], 2, 1)  # a page that is none
    assert got[-1] == 6 and got[6] == [-1]


def test_extend_captured_steps():
    """A captured step, replayed, takes and gives back pages as eager steps do."""
    from sparse_top_kv_gb300 import hs
    rng = random.Random(5)
    lens, table, ring, ends = state(rng, 9, 4, 8, 60, 20)
    i32 = dict(dtype=torch.int32, device="cuda")
    t = dict(new=torch.zeros(9, **i32), lens=torch.tensor(lens, **i32),
             table=torch.tensor(table, **i32), ring=torch.tensor(ring, **i32),
             ends=torch.tensor(ends, device="cuda"))
    outs = [torch.zeros(n, **i32) for n in (9, 10, 40, 40, 40)]
    def step():
        return hs.paged_extend(t["new"], t["lens"], t["table"], t["ring"], t["ends"], 4, 40,
                               attend_lens=outs[0], cu_new=outs[1], slot=outs[2], row_req=outs[3],
                               positions=outs[4])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(12):
        new = [rng.choice([1, 1, 1, 4, 0, -5]) for _ in range(9)]
        t["new"].copy_(torch.tensor(new))
        g.replay()
        table, ring, ends, lens, *rest = step_ref.extend(new, lens, table, ring, ends, 4, 40)
        got = [t["table"], t["ring"], t["ends"], t["lens"], *outs]
        assert [x.tolist() for x in got] == [table, ring, ends, lens, *rest[:-1]]


def rope(tokens, heads, kv_heads, d, rot, *, dtype=BF, cache=None, interleaved=False, scaling=None,
         far=1 << 20, in_place=False, page=16, strided=False, scales=True, seed=0):
    from sparse_top_kv_gb300 import hs
    g = torch.Generator().manual_seed(seed)
    cache = cache or dtype
    qkv = torch.randn(tokens, heads + 2 * kv_heads, d, generator=g).to(dtype).cuda()
    q, k, v = qkv.split([heads, kv_heads, kv_heads], 1)
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    q0 = q.clone()
    pages = -(-2 * tokens // page) + 1
    slot = torch.randperm(pages * page, generator=g)[:tokens].to(torch.int32)
    pos = torch.randint(0, far, (tokens,), generator=g, dtype=torch.int32)
    if tokens > 3:
        pos[1], slot[2] = -1, -1
    inv, m = hs.rope_frequencies(rot, scaling=scaling, factor=4.0, original_len=4096)
    caches = [torch.full((pages, page, kv_heads, d), 3.0).to(cache).cuda() for _ in "kv"]
    ks = vs = None
    if cache == E4 and scales:
        ks, vs = (torch.rand(kv_heads, generator=g).cuda() * 0.01 + 0.01 for _ in "kv")
    q_out = q if in_place else torch.full((tokens, heads, d), 5.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hs.rope_append(q, k, v, pos.cuda(), slot.cuda(), hs.rope_turns(inv), *caches,
                   interleaved=interleaved, mscale=m, k_scale=ks, v_scale=vs, q_out=q_out,
                   status=status)
    assert status.item() == 0
    live = (pos >= 0).cuda()
    p, w = pos.cuda().clamp_min(0), inv.cuda()
    ref = step_ref.rope(q0, p, w, interleaved, m)
    err = (q_out.double() - ref).abs() - step_ref.rope_bound(q0, ref, w, interleaved, m, dtype)
    assert not heads or err[live].max() <= 0, f"q: {err[live].max()} over"
    left = q0 if in_place else torch.full_like(q0, 5.0)
    assert torch.equal(q_out[~live], left[~live])
    there = live & (slot >= 0).cuda()
    at = slot.cuda().long()[there]
    for c, x, s, key in ((caches[0], k, ks, True), (caches[1], v, vs, False)):
        rows = c.flatten(0, 1)
        want = step_ref.rope(x, p, w, interleaved, m) if key else x.double()
        sc = None if cache != E4 else (s if s is not None else torch.ones(kv_heads).cuda())[:, None].double()
        tol = step_ref.rope_bound(x, want, w, interleaved, m, cache, sc)
        want = want if sc is None else (want / sc).clamp(-448, 448)
        if not key and sc is None:
            assert torch.equal(rows[at], x[there])
        got = rows[at].double()
        over = ((got - want[there]).abs() - tol[there]).max()
        assert over <= 0, f"{'k' if key else 'v'}: {over} over"
        rest = torch.ones(rows.shape[0], dtype=torch.bool, device="cuda")
        rest[at] = False
        assert (rows[rest].float() == 3).all(), "other places stay"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (64, 32), (64, 64), (256, 128), (80, 80),
                                   (80, 16), (128, 24), (72, 72), (40, 6), (128, 0), (1024, 1024),
                                   (8, 2)])
def test_rope(interleaved, dtype, cache, d, rot):
    if cache == E4 and d % 16:
        pytest.skip("an 8-bit cache's rows are multiples of 16")
    rope(19, 6, 2, d, rot, dtype=dtype, cache=cache, interleaved=interleaved)


@pytest.mark.parametrize("tokens", [1, 2, 5, 333])
@pytest.mark.parametrize("strided", [False, True])
def test_rope_tokens_and_strides(tokens, strided):
    rope(tokens, 32, 8, 128, 128, strided=strided, in_place=strided)
    rope(tokens, 5, 1, 64, 32, strided=strided, cache=E4, scales=False)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn"])
def test_rope_scaled(scaling):
    rope(64, 4, 2, 128, 128, scaling=scaling, far=1 << 21)


def test_rope_far_positions_are_exact():
    """Near 2^31 the angle is the exact product's, modulo whole turns."""
    from fractions import Fraction
    from sparse_top_kv_gb300 import hs
    turns = hs.rope_turns(hs.rope_frequencies(64)[0])
    pos = torch.tensor([2 ** 31 - 1, 2 ** 31 - 2, 123456789], dtype=torch.int32).cuda()
    q = torch.zeros(3, 1, 64, dtype=FP, device="cuda")
    q[:, :, :32] = 1.0
    y = hs.rope_append(q, None, None, pos, None, turns, None, None).double().cpu()
    for i, p in enumerate(pos.tolist()):
        for j, t in enumerate(turns.tolist()):
            a = 2 * math.pi * float(Fraction(p * t, 2 ** 64) % 1)
            # 2 pi 2^-26 of the angle, 8 u of sinpi / cospi, half a step of fp16.
            assert abs(y[i, 0, j] - math.cos(a)) <= 2 ** -11 + 1e-6
            assert abs(y[i, 0, j + 32] - math.sin(a)) <= 2 ** -11 + 1e-6


def test_rope_parts_nan_and_bad_slots():
    from sparse_top_kv_gb300 import hs
    turns = hs.rope_turns(hs.rope_frequencies(128)[0])
    k = torch.randn(4, 2, 128, device="cuda").to(BF)
    v = torch.randn(4, 2, 128, device="cuda").to(BF)
    v[0, 0, 3], v[0, 0, 4], v[0, 0, 5] = math.nan, math.inf, -1e30
    caches = [torch.zeros(3, 16, 2, 128, device="cuda").to(E4) for _ in "kv"]
    slot = torch.tensor([7, 48, 2 ** 31 - 1, 47], dtype=torch.int32).cuda()
    pos = torch.tensor([0, 1, 2, 3], dtype=torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert hs.rope_append(None, k, v, pos, slot, turns, *caches, status=status) is None
    assert status.item() == 6
    rows = caches[1].flatten(0, 1).float()
    assert rows[7, 0, 3].isnan() and rows[7, 0, 4] == 448 and rows[7, 0, 5] == -448
    assert (rows[[i for i in range(48) if i not in (7, 47)]] == 0).all()
    assert torch.equal(rows[47], v[3].float().clamp(-448, 448).to(E4).float())
    # Position 0 leaves a row as it is.
    assert torch.equal(caches[0].flatten(0, 1)[7].float(), k[0].float().to(E4).float())


def test_refusals():
    from sparse_top_kv_gb300 import hs
    i32 = dict(dtype=torch.int32, device="cuda")
    z = torch.zeros(4, **i32)
    ends = torch.zeros(2, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        hs.paged_extend(z, z.long(), z.view(4, 1), z, ends, 4, 8)
    with pytest.raises(ValueError):
        hs.paged_extend(z, z[:3], z.view(4, 1), z, ends, 4, 8)
    with pytest.raises(ValueError):
        hs.paged_extend(z, z, z.view(4, 1), z, ends, 4, -1)
    with pytest.raises(TypeError):
        hs.paged_extend(z, z, z.view(4, 1), z, z[:2], 4, 8)
    with pytest.raises(hs.HSError):
        hs.paged_extend(z, z, z.view(4, 1), z, ends, 0, 8)
    with pytest.raises(ValueError):
        hs.paged_extend(z, z, z.view(4, 1), z, ends, 4, 8, slot=z)
    q = torch.zeros(4, 2, 64, dtype=BF, device="cuda")
    c = torch.zeros(1, 16, 2, 64, dtype=BF, device="cuda")
    t = hs.rope_turns(hs.rope_frequencies(64)[0])
    ok = dict(q=q, k=q, v=q, positions=z, slot=z, turns=t, k_cache=c, v_cache=c)
    for bad in (dict(q=q.float()), dict(k=q.half()), dict(v=q[:3]), dict(positions=z.long()),
                dict(slot=None), dict(v=None), dict(turns=t.int()), dict(k_cache=c.float(), v_cache=c.float()),
                dict(v_cache=None), dict(turns=torch.cat([t, t])), dict(q_out=q[:, :1]),
                dict(k_scale=torch.ones(2, device="cuda")), dict(q=q.transpose(0, 1)),
                dict(q=None, k=None)):
        with pytest.raises((TypeError, ValueError, hs.HSError)):
            hs.rope_append(**{**ok, **bad})
