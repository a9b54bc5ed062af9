"""Memory that the paged-cache calls make for themselves on a stream other than the
current one: a block that the current stream has let go may still be read or written
there, so none of them may be used by the other stream."""
import pytest
import torch

from sparse_top_kv_gb300 import hs

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def state():
    g = torch.Generator().manual_seed(0)
    i32 = dict(dtype=torch.int32, device="cuda")
    page, pages, R, T = 16, 64, 3, 300
    rnd = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()
    return dict(q=rnd(R, 16, 128), k=rnd(pages, page, 2, 128), v=rnd(pages, page, 2, 128),
                kn=rnd(R, 2, 128), vn=rnd(R, 2, 128), score=torch.rand(R, T, generator=g).cuda(),
                table=torch.arange(R * 20, **i32).view(R, 20), lens=torch.full((R,), T, **i32),
                cu=torch.arange(R + 1, **i32), new=torch.ones(R, **i32), ring=torch.arange(64, **i32),
                ends=torch.tensor([0, 4], device="cuda"), turns=hs.rope_turns(hs.rope_frequencies(128)[0]),
                slot=torch.tensor([5, 99, 1000], **i32))


def decode(s, stream):
    return hs.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], 0.1, stream=stream)


def prefill(s, stream):
    return hs.paged_prefill(s["q"], s["k"], s["v"], s["table"], s["cu"], s["lens"], 0.1, stream=stream)


def extend(s, stream):
    return hs.paged_extend(s["new"], s["lens"], s["table"], s["ring"], s["ends"], 16, 40,
                           lens_out=s["lens"].clone(), ring_out=s["ends"].clone(), stream=stream)[1:]


def rope(s, stream):
    return [hs.rope_append(s["q"], s["kn"], s["vn"], s["lens"], s["slot"], s["turns"], s["k"],
                           s["v"], stream=stream)]


def evict(s, stream):
    return hs.evict_select(s["score"], s["lens"], 100, score_out=s["score"].clone(),
                           lens_out=s["lens"].clone(), stream=stream)[3]


@pytest.mark.parametrize("call", [decode, prefill, extend, rope, evict])
def test_blocks_that_were_let_go_are_not_used(call):
    s = state()
    side = torch.cuda.Stream()
    want = [t.clone() for t in call(s, None)]
    torch.cuda.synchronize()
    for _ in range(3):
        # Blocks of the results' sizes, let go while the current stream works on.
        held = [torch.empty_like(t) for t in want for _ in range(4)]
        at = {t.data_ptr() for t in held}
        torch.cuda._sleep(2_000_000)
        for t in held:
            t.zero_()
        del held, t
        got = call(s, side)
        assert not at & {t.data_ptr() for t in got}
        torch.cuda.synchronize()
        # (A move list means nothing behind its count.)
        if call is evict:
            assert torch.equal(got[2], want[2])
        else:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("call", [decode, prefill, extend, rope, evict])
def test_results_are_held_for_the_current_stream(call):
    """Results that are let go while the current stream still reads them."""
    s = state()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(s, side)
    torch.cuda.current_stream().wait_stream(side)
    want = [t.clone() for t in got]
    torch.cuda._sleep(40_000_000)
    late = [t.clone() for t in got]
    shapes = [(t.shape, t.dtype) for t in got]
    del got
    with torch.cuda.stream(side):
        junk = [torch.full(n, 77, dtype=d, device="cuda") for n, d in shapes for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(late, want))
    assert junk
