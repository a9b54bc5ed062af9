"""The operators of a step of several new tokens per request together
(pipeline.PagedBatch): tables and lengths against their definition, the caches
row by row, and the attention over them against the 64-bit one."""
import math

import pytest
import torch

import paged_ref
import step_ref
from sparse_top_kv_gb300 import hs
from sparse_top_kv_gb300.pipeline import PagedBatch

pytestmark = pytest.mark.gpu

BF, FP, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn

# Places: a prompt in chunks, drafted tokens that are taken back, single tokens, a
# request that ends and whose pages are taken again, and one that finds no room.
STEPS = [[37, 0, 5, 1], [40, 3, 1, 1], [1, -2, 1, 60], [1, 4, 0, 70], [0, 0, -6, 1], [1, 1, 30, 1],
         [-200, 1, 33, 1], [64, 1, 1, 1], [1, -1, 1, 0], [0, 0, 0, 0], [9, 80, 1, 1]]


@pytest.mark.parametrize("dtype,cache,heads,kvh,d,page,window", [
    (BF, BF, 8, 2, 128, 16, 0), (FP, FP, 6, 2, 64, 5, 24), (BF, E4, 8, 1, 256, 16, 0),
    (FP, E4, 4, 4, 128, 8, 40)])
@pytest.mark.parametrize("graph", [False, True])
def test_steps(dtype, cache, heads, kvh, d, page, window, graph):
    g = torch.Generator().manual_seed(page + d)
    R, layers, most, room = 4, 2, 90, 128
    scales = {}
    if cache == E4:
        scales = {n: torch.rand(layers, kvh, generator=g) * 0.02 + 0.01
                  for n in ("k_scale", "v_scale")}
    inv, mscale = hs.rope_frequencies(d // 2, scaling="linear", factor=2.0)
    pages = 200 // page
    b = PagedBatch(num_reqs=R, layers=layers, heads=heads, kv_heads=kvh, d=d, page_size=page,
                   num_pages=pages, max_len=room, max_tokens=most, scale=1 / math.sqrt(d),
                   inv_freq=inv, mscale=mscale, window=window, num_sinks=2 if window else 0,
                   dtype=dtype, cache_dtype=cache, **scales)
    side = torch.cuda.Stream()
    seen = set()
    for i, new in enumerate(STEPS):
        state = (b.seq_lens.tolist(), b.block_table.tolist(), b.free_ring.tolist(),
                 b.ring_pos.tolist())
        was = [(b.k_cache[l].float(), b.v_cache[l].float()) for l in range(layers)]
        # A model's projection gives q, k and v in one row a token; the rows
        # behind the last token are NaN.
        x = torch.randn(layers, most, heads + 2 * kvh, d, generator=g)
        x[:, sum(max(0, n) for n in new):] = math.nan
        x = x.to(dtype).cuda()
        qs, ks, vs = x[:, :, :heads], x[:, :, heads:heads + kvh], x[:, :, heads + kvh:]
        b.out.fill_(7.0)
        lens = torch.tensor(new, dtype=torch.int32, device="cuda")
        if graph and i == 2:
            b.capture()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side if i % 2 else torch.cuda.current_stream()):
            (b.replay if graph and i >= 2 else b.step)(lens, qs, ks, vs)
        torch.cuda.synchronize()

        table, ring, ends, held, attend, cu, slot, req, pos, status = step_ref.extend(
            new, state[0], state[1], state[2], state[3], page, most)
        assert b.seq_lens.tolist() == held and b.attend_lens.tolist() == attend
        assert b.cu_new.tolist() == cu and b.ring_pos.tolist() == ends
        assert b.slot.tolist() == slot and b.positions.tolist() == pos and b.row_req.tolist() == req
        assert b.free_ring.tolist() == ring
        for r in range(R):
            n = -(-held[r] // page)
            assert b.block_table[r, :n].tolist() == table[r][:n]
        in_use = [p for r in range(R) for p in table[r][:-(-held[r] // page)]]
        free = [ring[j % pages] for j in range(ends[0], ends[1])]
        assert sorted(in_use + free) == list(range(pages))  # none lost, none twice
        seen.add(status)
        if status:
            with pytest.raises(hs.HSError):
                b.check()
        b.check()

        live = torch.tensor([s >= 0 for s in slot])
        at = torch.tensor(slot, device="cuda")[live.cuda()].long()
        p = torch.tensor(pos, device="cuda")[live.cuda()]
        for l in range(layers):
            # The caches: the new tokens' rows, and nothing else.
            for c, old, rows, rot, name in ((b.k_cache[l], was[l][0], ks[l], True, "k_scale"),
                                            (b.v_cache[l], was[l][1], vs[l], False, "v_scale")):
                src = rows[live.cuda()]
                want = step_ref.rope(src, p, inv.cuda(), False, mscale) if rot else src.double()
                sc = scales[name][l].cuda().double()[:, None] if scales else None
                bound = step_ref.rope_bound(src, want, inv.cuda(), False, mscale, cache, sc)
                got = c.reshape(-1, kvh, d)[at].double()
                paged_ref.check(got, want if sc is None else want / sc, bound, name)
                now, old = c.float().reshape(-1, kvh, d), old.reshape(-1, kvh, d)
                now[at], old[at] = 0, 0
                assert torch.equal(now, old)
        # The attention, over what the cache holds.  (q_rot is the last layer's.)
        l = layers - 1
        src = qs[l][live.cuda()]
        want = step_ref.rope(src, p, inv.cuda(), False, mscale)
        paged_ref.check(b.q_rot[live.cuda()].double(), want,
                        step_ref.rope_bound(src, want, inv.cuda(), False, mscale, dtype), "q")
        for l in range(layers):
            q = step_ref.rope(qs[l], torch.tensor(pos, device="cuda"), inv.cuda(), False,
                              mscale).to(dtype) if l < layers - 1 else b.q_rot
            if l < layers - 1:
                # (rotated by the operator: bit-exact)
                q = torch.zeros_like(b.q_rot)
                hs.rope_append(qs[l], None, None, b.positions, None, b.turns, None, None,
                               mscale=mscale, q_out=q)
            ref, ref_lse, (tol, tol_lse), written = step_ref.prefill(
                q, b.k_cache[l], b.v_cache[l], b.block_table, b.cu_new, b.attend_lens, b.scale,
                window=window, sinks=b.num_sinks,
                **{n: t[l].cuda() for n, t in scales.items()})
            mask = written & live.cuda()
            paged_ref.check(b.out[l][mask].double(), ref[mask], tol[mask], "out")
            paged_ref.check(b.lse[l][mask].double(), ref_lse[mask], tol_lse[mask], "lse")
            assert (b.out[l][~written] == 7).all()
    assert seen == {0, 3}


def test_stop_gives_the_pages_back():
    b = PagedBatch(num_reqs=2, heads=4, kv_heads=2, d=64, page_size=16, max_len=64, num_pages=4,
                   max_tokens=64, scale=0.125)
    x = torch.randn(1, 64, 8, 64, device="cuda").to(BF)
    rows = x[:, :, :4], x[:, :, 4:6], x[:, :, 6:]
    new = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    out = b.step(new, *rows)[0].clone()
    b.stop(1)
    again = b.step(new.flip(0), *rows)[0]
    b.check()
    assert b.seq_lens.tolist() == [64, 0] and torch.equal(out, again)
    b.step(new, *rows)
    with pytest.raises(hs.HSError):
        b.check()
    assert b.seq_lens.tolist() == [64, 0]


def test_drafts_taken_back_leave_no_trace():
    """Tokens that were given up again do not change what comes after."""
    def run(draft):
        g = torch.Generator().manual_seed(0)
        b = PagedBatch(num_reqs=1, heads=4, kv_heads=2, d=128, page_size=16, max_len=200,
                       max_tokens=50, scale=0.1)
        for n in (50, 1, 1):
            x = torch.randn(1, 50, 8, 128, generator=g).to(BF).cuda()
            rows = x[:, :, :4], x[:, :, 4:6], x[:, :, 6:]
            if draft and n == 1:
                y = torch.full_like(x, math.inf)
                b.step(torch.tensor([20], dtype=torch.int32, device="cuda"), y[:, :, :4],
                       y[:, :, 4:6], y[:, :, 6:])
                b.grow(torch.tensor([-20], dtype=torch.int32, device="cuda"))
            out, lse = b.step(torch.tensor([n], dtype=torch.int32, device="cuda"), *rows)
        b.check()
        return out[:, :1].clone(), lse[:, :1].clone()

    for a, c in zip(run(False), run(True)):
        assert torch.equal(a, c)


def test_a_last_page_is_used_to_its_end():
    """max_len 100 with pages of 16: 112 tokens are held and attended to."""
    g = torch.Generator().manual_seed(1)
    b = PagedBatch(num_reqs=1, heads=4, kv_heads=2, d=64, page_size=16, max_len=100,
                   max_tokens=56, scale=0.125)
    n = torch.tensor([56], dtype=torch.int32, device="cuda")
    for _ in range(2):
        x = torch.randn(1, 56, 8, 64, generator=g).to(BF).cuda()
        b.step(n, x[:, :, :4], x[:, :, 4:6], x[:, :, 6:])
    b.check()
    ref, ref_lse, (tol, tol_lse), _ = step_ref.prefill(
        b.q_rot, b.k_cache[0], b.v_cache[0], b.block_table, b.cu_new, b.attend_lens, b.scale)
    assert b.seq_lens.tolist() == [112]
    paged_ref.check(b.out[0].double(), ref, tol, "out")
    paged_ref.check(b.lse[0].double(), ref_lse, tol_lse, "lse")
    b.step(n.clamp(max=1), x[:, :, :4], x[:, :, 4:6], x[:, :, 6:])
    with pytest.raises(hs.HSError):
        b.check()
