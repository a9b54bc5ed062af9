"""hs.paged_prefill against the 64-bit definition: chunks of new tokens over
paged caches, at the sizes, layouts and masks where it can go wrong."""
import math

import pytest
import torch

import paged_ref
import step_ref

pytestmark = pytest.mark.gpu

BF, FP, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def setup(new, lens, heads, kv_heads, d, page, dtype=BF, cache=None, *, pad=0, seed=0, blocks=0,
          scales=None, layout="bshd"):
    """A call's tensors; places that no request holds are NaN."""
    g = torch.Generator().manual_seed(seed)
    cache = cache or dtype
    R = len(new)
    blocks = blocks or max(1, max(-(-max(t, 1) // page) for t in lens))
    pages = R * blocks + 2
    table = torch.randperm(pages, generator=g)[:R * blocks].to(torch.int32).view(R, blocks)

    def make():
        shape = (pages, page, kv_heads, d) if layout == "bshd" else (pages, kv_heads, page, d)
        x = torch.randn(shape, generator=g)
        x = x if layout == "bshd" else x.transpose(1, 2)
        held = torch.zeros(pages, page, dtype=torch.bool)
        for r, T in enumerate(lens):
            for t in range(min(max(T, 0), blocks * page)):
                held[table[r, t // page], t % page] = True
        x[~held] = math.nan
        y = x.to(cache)
        return y.cuda() if layout == "bshd" else y.transpose(1, 2).contiguous().cuda().transpose(1, 2)

    s = dict(q=torch.randn(sum(new) + pad, heads, d, generator=g).to(dtype).cuda(), k=make(),
             v=make(), table=table.cuda(),
             cu=torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda(),
             lens=torch.tensor(lens, dtype=torch.int32).cuda(), scale=1 / math.sqrt(d), k_scale=None,
             v_scale=None, status=torch.zeros(1, dtype=torch.int32).cuda())
    if scales or (scales is None and cache == E4):
        s["k_scale"] = (torch.rand(kv_heads, generator=g) + 0.5).cuda()
        s["v_scale"] = (torch.rand(kv_heads, generator=g) + 0.5).cuda()
    return s


def call(s, window=0, sinks=0, max_len=None, **kw):
    from sparse_top_kv_gb300 import hs
    out = torch.full_like(s["q"], 7.0) if s["q"].is_contiguous() else torch.full(
        s["q"].shape, 7.0, dtype=s["q"].dtype, device="cuda")
    lse = torch.full(s["q"].shape[:2], 7.0, device="cuda")
    kw = {"out": out, "lse": lse, "status": s["status"], **kw}
    return hs.paged_prefill(s["q"], s["k"], s["v"], s["table"], s["cu"], s["lens"], s["scale"],
                            window=window, num_sinks=sinks, max_len=max_len, k_scale=s["k_scale"],
                            v_scale=s["v_scale"], **kw)


def check(s, window=0, sinks=0, max_len=None, status=0, **kw):
    out, lse = call(s, window, sinks, max_len, **kw)
    ref, ref_lse, (tol, tol_lse), written = step_ref.prefill(
        s["q"], s["k"], s["v"], s["table"], s["cu"], s["lens"], s["scale"], window=window,
        sinks=sinks, max_len=max_len, k_scale=s["k_scale"], v_scale=s["v_scale"])
    assert s["status"].item() == status
    for got, want, bound, what in ((out, ref, tol, "out"), (lse, ref_lse, tol_lse, "lse")):
        got, want, bound = got[written].double(), want[written], bound[written]
        nan = want.isnan()
        assert torch.equal(got.isnan(), nan), f"{what}: NaN elsewhere"
        paged_ref.check(*(torch.where(nan, 0.0, x) for x in (got, want, bound)), what)
    assert (out[~written] == 7).all() and (lse[~written] == 7).all(), "rows of no request"
    return out, lse


SHAPES = [(32, 8, 128), (12, 12, 64), (16, 1, 256), (4, 4, 128), (10, 2, 64), (7, 1, 128),
          (24, 2, 128), (6, 3, 256), (40, 1, 128)]


@pytest.mark.parametrize("heads,kv_heads,d", SHAPES)
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)])
def test_shapes_and_types(heads, kv_heads, d, dtype, cache):
    check(setup([1, 37, 0, 130, 5], [1, 300, 12, 130, 77], heads, kv_heads, d, 16, dtype, cache,
                pad=3))


@pytest.mark.parametrize("page", [1, 3, 16, 24, 32, 64, 100, 256])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (BF, E4)])
def test_page_sizes(page, dtype, cache):
    check(setup([33, 2, 70], [200, 129, 70], 8, 2, 128, page, dtype, cache))


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257])
@pytest.mark.parametrize("extra", [0, 1, 127, 128, 129, 1000])
def test_lengths(n, extra):
    check(setup([n], [n + extra], 8, 2, 128, 16, seed=n))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (64, 0), (128, 1), (100, 200), (129, 4),
                                          (700, 0), (5000, 3)])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, E4)])
def test_windows(window, sinks, dtype, cache):
    check(setup([150, 1, 40], [700, 600, 40], 8, 2, 128, 16, dtype, cache), window, sinks)


def test_many_short_and_one_long_request():
    new = [1] * 40 + [500] + [3] * 9
    lens = [1 + 37 * i % 900 for i in range(40)] + [2000] + [3 + 100 * i for i in range(9)]
    check(setup(new, lens, 8, 2, 128, 16))


def test_long_context_is_split():
    check(setup([5], [20000], 32, 8, 128, 64))
    check(setup([300], [9000], 4, 1, 64, 64, FP))


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, FP), (BF, E4)])
def test_what_a_query_does_not_attend_to_has_no_effect(dtype, cache):
    """NaN and infinities in later tokens' rows, and in tokens that have left
    the window: only the queries that attend to them see them."""
    n, T = 90, 333
    for window in (0, 60):
        s = setup([n], [T], 8, 2, 128, 16, dtype, cache, seed=3)
        for t, what in ((T - 1, math.nan), (T - 45, math.inf), (T - 46, -math.inf), (100, math.nan)):
            if window == 0 and t == 100:
                continue
            if cache == E4 and not math.isnan(what):
                what = math.nan
            pg, at = s["table"][0, t // 16].item(), t % 16
            s["v"][pg, at, 1, 3] = what
            s["v"][pg, at, 0, 70] = what
        s["k"][s["table"][0, (T - 10) // 16].item(), (T - 10) % 16, 1, 5] = math.nan
        check(s, window=window)


@pytest.mark.parametrize("dtype,heads,kv_heads,d,window,sinks,page", [
    (BF, 8, 2, 128, 0, 0, 16), (FP, 8, 2, 128, 150, 3, 128), (BF, 16, 1, 64, 150, 3, 32),
    (FP, 16, 1, 64, 0, 0, 16), (BF, 3, 3, 128, 150, 3, 16), (FP, 33, 1, 64, 150, 3, 16),
    (BF, 80, 40, 64, 0, 0, 32)])
def test_few_tokens_over_e4m3_caches(dtype, heads, kv_heads, d, window, sinks, page):
    """Units of one query tile; rows that are not finite, some in part."""
    new = [1, 0, 5, 2, 1, 3, 60, 1] + [1] * 60
    lens = [700, 0, 5, 131, 1, 900, 400, 2500] + [1 + 29 * i for i in range(60)]
    if heads // kv_heads > 32:
        new[6] = 1
    s = setup(new, lens, heads, kv_heads, d, page, dtype, E4, seed=d + heads)
    for r, back in ((0, 151), (5, 150), (5, 2), (6, 400), (7, 1), (5, 152), (7, 152)):
        t = lens[r] - back
        s["v"][s["table"][r, t // page].item(), t % page, 0, d - 2] = math.nan
    check(s, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, FP), (BF, E4)])
@pytest.mark.parametrize("scale", [-0.07, 0.0])
def test_scales_that_are_not_positive(dtype, cache, scale):
    s = setup([70, 3], [500, 130], 8, 2, 128, 16, dtype, cache)
    s["scale"] = scale
    check(s)
    if cache == E4:
        s["k_scale"] = s["k_scale"] * torch.tensor([-1.0, 1.0], device="cuda")
        check(s, window=100, sinks=2)


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, E4)])
@pytest.mark.parametrize("heads,d", [(16, 256), (16, 128)])
def test_infinite_values_ahead_of_many_tiles(heads, d, dtype, cache):
    """Where the window begins: rows that a part of the queries sees are added
    apart, while the tiles behind them are under way."""
    lens = [690 + i for i in range(160)]
    s = setup([8] * 160, lens, heads, 1, d, 16, dtype, cache, seed=5)
    for r, T in enumerate(lens):
        for back, dim in ((563, 3), (565, d - 1)):
            t = T - back
            s["v"][s["table"][r, t // 16].item(), t % 16, 0, dim] = (
                math.nan if cache == E4 or r % 2 else math.inf)
    check(s, window=560)


def test_queries_before_position_zero_and_empty_requests():
    s = setup([4, 3, 0, 5], [0, 2, 9, -3], 8, 2, 128, 16, pad=2)
    out, lse = check(s)
    assert (out[:5] == 0).all() and (lse[:5] == -math.inf).all()


def test_minus_infinite_logits():
    s = setup([6], [20], 8, 2, 128, 16)
    s["k"][:, :, 0, 0] = -math.inf
    s["q"][:, :4, 0] = 1.0
    s["q"][:, :4, 1:] = 0.0
    s["k"][:, :, 0, 1:] = 1.0
    out, lse = call(s)
    assert (out[:6, :4] == 0).all() and (lse[:6, :4] == -math.inf).all()
    assert torch.isfinite(out[:6, 4:]).all()


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, FP), (BF, E4)])
def test_growing_logits(dtype, cache):
    """Maxima that move from tile to tile, by much and by little, for some heads
    only, and a token that outweighs all others."""
    s = setup([140], [900], 8, 2, 128, 16, dtype, cache)
    t = torch.arange(900)
    pg, at = s["table"][0].cpu()[t // 16].long(), t % 16
    k = torch.randn(900, 128) * 0.1
    k[:, 0] = (t // 128).float() * 12
    k[:, 1] = t * 0.02
    k[500, 2] = 300
    for x, w in ((0, 1.0), (1, 0.3)):
        s["k"][pg.cuda(), at.cuda(), x] = (k * w).to(cache).cuda()
    s["q"][:, ::2, 0] = 4.0
    s["q"][:, 1, 2] = 8.0
    check(s)


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, FP), (BF, E4)])
def test_small_weights_behind_a_sink_without_value(dtype, cache):
    s = setup([64], [400], 4, 2, 128, 16, dtype, cache)
    pg = s["table"][0, 0].item()
    s["q"][:, :, 0] = 8.0
    s["k"][:, :, :, 0] = 0.0
    s["k"][pg, 0, :, 0] = 20.0  # 14.1 above the others: their weights are 2^-20
    s["v"][pg, 0] = 0.0
    check(s)


@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
@pytest.mark.parametrize("cache", [BF, E4])
def test_strided_queries_and_cache_layouts(layout, cache):
    s = setup([20, 77], [150, 300], 8, 2, 128, 32, BF, cache, layout=layout)
    wide = torch.randn(97, 12, 128, device="cuda").to(BF)
    s["q"] = wide[:, :8]
    check(s)


def test_broadcast_cache():
    """One page's rows for every page, and one head's for both."""
    s = setup([20], [64], 8, 2, 128, 16)
    for c in "kv":
        s[c] = torch.randn(1, 16, 1, 128, device="cuda").to(BF).expand(6, 16, 2, 128)
    check(s)


def test_bad_pages_are_skipped():
    s = setup([40, 9], [333, 100], 8, 2, 128, 16)
    s["table"][0, 3], s["table"][0, 20], s["table"][1, 0] = -1, 1 << 20, 5000
    check(s, status=6)


def test_length_past_the_bound():
    check(setup([40, 9], [333, 100], 8, 2, 128, 16), max_len=256, status=6)


def test_cu_new_out_of_order_stays_inside():
    s = setup([40, 9], [333, 100], 8, 2, 128, 16)
    s["cu"].copy_(torch.tensor([-5, 60, 30]))
    call(s)
    assert s["status"].item() == 6


def test_results_do_not_depend_on_timing_or_workspace():
    from sparse_top_kv_gb300 import hs
    s = setup([100, 3, 257], [3000, 2000, 900], 32, 8, 128, 16)
    n = hs.paged_prefill_workspace_bytes(s["q"].shape[0], 3, 32, 8, 128, s["table"].shape[1] * 16)
    ref = None
    for i in range(5):
        ws = torch.full((n + 512,), 255 - i, dtype=torch.uint8, device="cuda")
        got = call(s, workspace=ws)
        assert ref is None or (torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]))
        ref = got


def test_one_token_matches_decode():
    from sparse_top_kv_gb300 import hs
    s = setup([1] * 5, [1, 20, 333, 64, 1000], 16, 4, 128, 16)
    out, lse = check(s)
    ref, ref_lse = hs.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"])
    assert (out.float() - ref.float()).abs().max() < 0.02 and (lse - ref_lse).abs().max() < 1e-4


def test_captured_on_another_stream_and_two_at_once():
    s, t = (setup([64, 7], [800, 90], 8, 2, 128, 16, seed=i) for i in (1, 2))
    want = [call(x)[0] for x in (s, t)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for x, st in zip((s, t), streams):
            st.wait_stream(torch.cuda.current_stream())
            got.append(call(x, stream=st)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], device="cuda")
    with torch.cuda.graph(g):
        call(s, out=out, lse=lse, workspace=ws)
    for x in (t, s):
        for name in ("q", "k", "v", "table", "cu", "lens"):
            if x is not s:
                s.setdefault("old", {})[name] = s[name].clone()
                s[name].copy_(x[name])
            else:
                s[name].copy_(s["old"][name])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0] if x is s else want[1])


def test_refusals():
    from sparse_top_kv_gb300 import hs
    s = setup([4], [20], 8, 2, 128, 16)
    for name, bad, err in (("q", s["q"].float(), TypeError), ("q", s["q"][:, :, :64], ValueError),
                           ("q", s["q"][0], ValueError), ("q", s["q"].transpose(0, 1), ValueError),
                           ("k", s["k"].half(), TypeError), ("v", s["v"][:1], ValueError),
                           ("cu", s["cu"].long(), TypeError), ("cu", s["cu"][:1], ValueError),
                           ("lens", s["lens"].cpu(), ValueError),
                           ("table", s["table"].long(), TypeError)):
        with pytest.raises((err, ValueError, hs.HSError)):
            call({**s, name: bad})
    with pytest.raises(hs.HSError):
        call(s, max_len=10000)
    with pytest.raises(hs.HSError):
        call({**s, "k_scale": torch.ones(2, device="cuda")})
    with pytest.raises(ValueError):
        call(s, workspace=torch.empty(64, 64, device="cuda").t()[:, :3])
    with pytest.raises(ValueError):
        call(s, out=torch.empty(4, 8, 64, dtype=BF, device="cuda"))


def test_cold_cache_loads_land_in_any_order():
    s = setup([5] * 6, [4000 - 37 * i for i in range(6)], 16, 4, 128, 16)
    flush = torch.empty(48 << 20, dtype=torch.int32, device="cuda")
    want = call(s)
    for _ in range(60):
        flush.fill_(1)
        got = call(s)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert s["status"].item() == 0
