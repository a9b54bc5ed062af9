"""hs_paged_decode against its 64-bit definition: types, head layouts,
lengths, windows, strides, what stands in places that must not be read,
running scores, streams and captured graphs."""
import math

import pytest
import torch

import paged_ref as ref
from sparse_top_kv_gb300 import hs

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


def make(lens, heads, kv_heads, d, page, *, kind="bf16", seed=0, spare=3, qt=None, blocks=None,
         poison=False):
    """Caches with a random block table; `poison` fills every place that no
    request's tokens occupy with NaN codes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    R = len(lens)
    blocks = max(1, max(-(-max(x, 0) // page) for x in lens)) if blocks is None else blocks
    P = R * blocks + spare
    kt = TYPES[kind]
    qt = qt or (torch.float16 if kind == "fp16" else torch.bfloat16)
    table = torch.randperm(P, generator=g, device="cuda")[:R * blocks].to(torch.int32)
    table = table.view(R, blocks).contiguous()
    base = torch.bfloat16 if kind == "e4m3" else kt
    k = torch.randn(P, page, kv_heads, d, generator=g, device="cuda").to(base)
    v = torch.randn(P, page, kv_heads, d, generator=g, device="cuda").to(base)
    if poison:
        used = torch.zeros(P, page, dtype=torch.bool, device="cuda")
        for r, n in enumerate(lens):
            t = torch.arange(max(n, 0), device="cuda")
            used[table[r].long()[t // page], t % page] = True
        k[~used] = math.nan
        v[~used] = math.nan
    q = torch.randn(R, heads, d, generator=g, device="cuda").to(qt)
    scales = (None, None)
    if kind == "e4m3":
        k, v = k.to(kt), v.to(kt)
        scales = tuple(torch.rand(kv_heads, generator=g, device="cuda") + 0.5 for _ in range(2))
    return dict(q=q, k=k, v=v, table=table, scales=scales, scale=1 / math.sqrt(d),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def run_and_check(s, *, window=0, sinks=0, max_len=None, score=None, decay=1.0, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = None if score is None else score.clone()
    out, lse = hs.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"],
                               window=window, num_sinks=sinks, max_len=max_len,
                               k_scale=s["scales"][0], v_scale=s["scales"][1], score=score,
                               score_decay=decay, status=status, **kw)
    torch.cuda.synchronize()
    o, l, sc, tol = ref.paged_decode(s["q"], s["k"].to(torch.float32), s["v"].to(torch.float32),
                                     s["table"], s["lens"], s["scale"], window=window,
                                     sinks=sinks, max_len=max_len, k_scale=s["scales"][0],
                                     v_scale=s["scales"][1], score=before, decay=decay)
    ref.check(out, o, tol[0], "out")
    ref.check(lse, l, tol[1], "lse")
    if score is not None:
        ref.check(score, sc, tol[2], "score")
    return out, lse, int(status.item())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (8, 8), (32, 8), (15, 3), (16, 1), (24, 2),
                                            (40, 1)])
def test_types_and_heads(kind, d, heads, kv_heads):
    s = make([1, 15, 16, 17, 130, 0, 333], heads, kv_heads, d, 16, kind=kind, seed=d + heads,
             poison=kind != "e4m3")
    *_, status = run_and_check(s)
    assert status == 0


@pytest.mark.parametrize("page", [1, 3, 16, 48, 64, 256])
@pytest.mark.parametrize("lens", [[1], [2, 1], [1000], [0, 0], [129, 4097, 7],
                                  list(range(1, 70))])
def test_pages_and_lengths(page, lens):
    s = make(lens, 8, 2, 64, page, seed=page + len(lens), poison=True)
    *_, status = run_and_check(s)
    assert status == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,kv_heads", [([20000], 8), ([9000, 1, 12345, 800], 4),
                                           ([5000] * 12, 8), ([40001], 1)])
def test_split_contexts(kind, lens, kv_heads):
    """Contexts that several CTAs share, units ending inside a CTA's run."""
    s = make(lens, 4 * kv_heads, kv_heads, 128, 64, kind=kind, seed=3)
    run_and_check(s)


def test_e4m3_with_fp16_query():
    s = make([5, 700, 33], 8, 2, 128, 16, kind="e4m3", qt=torch.float16)
    run_and_check(s)


def test_e4m3_large_and_small_queries():
    s = make([400, 90], 8, 2, 128, 16, kind="e4m3", seed=9)
    s["q"][0] *= 1e30
    s["scale"] *= 1e-30
    run_and_check(s)
    s["q"][0] *= 1e-38
    s["q"][0] *= 1e-20
    s["q"][1] = 0.0
    s["scale"] = 1e3
    run_and_check(s)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (100, 0), (256, 4), (5000, 4), (17, 64)])
@pytest.mark.parametrize("scored", [False, True])
def test_window_and_sinks(window, sinks, scored):
    lens = [1, 3, 50, 260, 1000, 0, 4097]
    s = make(lens, 16, 4, 128, 16, seed=window)
    # Pages that hold no attended token are never looked up.
    for r, n in enumerate(lens):
        seen = {t // 16 for t in ref.visible(n, window, sinks)}
        for b in range(s["table"].shape[1]):
            if b not in seen:
                s["table"][r, b] = 1 << 30
    score = torch.rand(len(lens), s["table"].shape[1] * 16, device="cuda") if scored else None
    *_, status = run_and_check(s, window=window, sinks=sinks, score=score)
    assert status == 0


@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("kind,heads,kv_heads,d", [("bf16", 32, 8, 128), ("fp16", 12, 12, 64),
                                                   ("e4m3", 16, 1, 256), ("bf16", 3, 1, 128)])
def test_running_scores(decay, kind, heads, kv_heads, d):
    lens = [1, 0, 700, 2049, 16, 33]
    s = make(lens, heads, kv_heads, d, 16, kind=kind, seed=7)
    n = s["table"].shape[1] * 16
    wide = torch.rand(len(lens), n + 5, device="cuda")
    score = wide[:, :2049]  # ends inside a page, its rows further apart than they are long
    if decay == 0.0:
        wide.fill_(math.nan)  # the old value is not read
        for r, T in enumerate(lens):
            wide[r, T:] = 2.0
    keep = wide.clone()
    run_and_check(s, score=score, decay=decay)
    for r, T in enumerate(lens):
        assert torch.equal(wide[r, T:], keep[r, T:])  # behind the context: as it was
    if decay == 0.0:
        for r, T in enumerate(lens):
            # Each head's weights sum to 1: fp32 sums of up to 2049 terms.
            assert abs(float(wide[r, :T].double().sum()) - (heads if T else 0)) <= heads * 2e-3


def test_scored_call_gives_the_same_output():
    s = make([700, 33, 5000], 16, 4, 128, 16, seed=5)
    out, lse, _ = run_and_check(s)
    score = torch.zeros(3, s["table"].shape[1] * 16, device="cuda")
    out2, lse2, _ = run_and_check(s, score=score)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_cache_layouts_and_strided_query():
    s = make([100, 37, 64], 16, 4, 128, 16, seed=11)
    want, want_lse, _ = run_and_check(s)
    k, v = s["k"], s["v"]
    # [pages, heads, page, d] storage, and K and V interleaved in one buffer.
    for store in (lambda x: x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3),
                  lambda x: torch.stack([x, x], 1)[:, 0]):
        s["k"], s["v"] = store(k), store(v)
        assert not s["k"].is_contiguous()
        got, got_lse, _ = run_and_check(s)
        assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    s["k"], s["v"] = k, v
    fused = torch.randn(3, 16 * 128 + 64, device="cuda").to(torch.bfloat16)
    fused[:, :16 * 128] = s["q"].view(3, -1)
    s["q"] = fused[:, :16 * 128].unflatten(1, (16, 128))
    got, _, _ = run_and_check(s)
    assert torch.equal(got, want)


def test_bad_pages_are_skipped_and_reported():
    s = make([100, 50, 40], 8, 2, 64, 16, seed=2)
    s["table"][0, 2] = -1
    s["table"][1, 0] = s["k"].shape[0]
    s["table"][2, :3] = 1 << 30
    out, lse, status = run_and_check(s)
    assert status == 6 and hs.STATUS_NAMES[status] == "HS_ERR_BAD_INDEX"
    assert not out[2].any() and (lse[2] == -math.inf).all()


def test_longer_than_max_len_is_cut_and_reported():
    s = make([100, 40], 8, 2, 64, 16, seed=2)
    *_, status = run_and_check(s, max_len=64)
    assert status == 6
    *_, status = run_and_check(s, max_len=112)
    assert status == 0


def test_lowest_values_and_minus_infinity():
    s = make([64, 64, 64], 8, 2, 64, 16, seed=4)
    low = torch.finfo(torch.bfloat16).min
    s["q"][:] = 1.0
    s["k"][s["table"][0].long()] = low / 128   # every logit hugely negative, finite
    s["k"][s["table"][1].long()] = -math.inf   # every logit -inf: no weight anywhere
    s["k"][s["table"][2, 0].long()] = -math.inf  # the first page masks itself
    out, lse, _ = run_and_check_nonfinite(s)
    o0 = s["v"][s["table"][0].long()].flatten(0, 1).double().mean(0)
    # Equal logits: the plain mean, rounded once (values below 1: 2^-9).
    assert (out[0].double().view(2, 4, 64) - o0[:, None]).abs().max() <= 2.0 ** -9
    assert not out[1].any() and (lse[1] == -math.inf).all()
    assert torch.isfinite(out[2]).all()
    s["k"][s["table"][0, 1].long(), 3] = math.nan  # an attended NaN shows
    out, lse, _ = run_and_check_nonfinite(s)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.isfinite(out[2]).all()


def run_and_check_nonfinite(s):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = hs.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"],
                               status=status)
    torch.cuda.synchronize()
    return out, lse, int(status.item())


def test_offsets_past_32_bits():
    """The last pages of a cache of more than 2^32 bytes."""
    page, kvh, d = 64, 8, 128
    P = (1 << 32) // (page * kvh * d * 2) + 40
    k = torch.zeros(P, page, kvh, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(1)
    for c in (k, v):
        c[-20:] = torch.randn(20, page, kvh, d, generator=g, device="cuda").to(torch.bfloat16)
    table = (P - 1 - torch.arange(20, device="cuda")).to(torch.int32).view(2, 10)
    s = dict(q=torch.randn(2, 32, d, generator=g, device="cuda").to(torch.bfloat16), k=k, v=v,
             table=table, scales=(None, None), scale=0.1,
             lens=torch.tensor([640, 601], dtype=torch.int32, device="cuda"))
    run_and_check(s)


def test_repeatable_and_on_another_stream():
    s = make([3000, 1, 777, 20000], 32, 8, 128, 16, seed=6)
    ws = torch.empty(hs.paged_decode_workspace_bytes(4, 32, 8, 128, s["table"].shape[1] * 16),
                     dtype=torch.uint8, device="cuda")
    out, lse, _ = run_and_check(s, workspace=ws)
    ws.fill_(255)  # nothing is kept in it
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        o2, l2 = hs.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"],
                                 workspace=ws, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_captured_graph_follows_lengths():
    s = make([64, 64, 64], 8, 2, 128, 16, seed=8)
    score = torch.zeros(3, 64, device="cuda")
    ws = torch.empty(hs.paged_decode_workspace_bytes(3, 8, 2, 128, 64, with_score=True),
                     dtype=torch.uint8, device="cuda")
    out = torch.empty_like(s["q"])
    lse = torch.empty(3, 8, device="cuda")

    def call():
        hs.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"], score=score,
                        score_decay=0.0, out=out, lse=lse, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([64, 1, 0], [17, 63, 5]):
        s["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        score.zero_()
        graph.replay()
        torch.cuda.synchronize()
        o, l, sc, tol = ref.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"],
                                         score=torch.zeros_like(score), decay=0.0)
        ref.check(out, o, tol[0], "out")
        ref.check(lse, l, tol[1], "lse")
        ref.check(score, sc, tol[2], "score")


def test_no_requests():
    s = make([4], 8, 2, 64, 16)
    out, lse = hs.paged_decode(s["q"][:0], s["k"], s["v"], s["table"][:0], s["lens"][:0], 1.0)
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)


@pytest.mark.parametrize("change,error", [
    (dict(q="float"), TypeError), (dict(k="double"), TypeError), (dict(v="short"), ValueError),
    (dict(seq_lens="long"), TypeError), (dict(seq_lens="cpu"), ValueError),
    (dict(table="long"), TypeError), (dict(q="heads"), ValueError),
    (dict(score="narrow"), ValueError), (dict(lse="half"), TypeError),
    (dict(k="mixed"), TypeError), (dict(d="odd"), hs.HSError), (dict(scale="bf16"), hs.HSError),
    (dict(k="unaligned"), hs.HSError)])
def test_refusals(change, error):
    s = make([20, 30], 8, 2, 64, 16)
    q, k, v, table, lens, kw = s["q"], s["k"], s["v"], s["table"], s["lens"], {}
    if change.get("q") == "float":
        q = q.float()
    if change.get("q") == "heads":
        q = q.transpose(1, 2).contiguous().transpose(1, 2)
    if change.get("k") == "double":
        k = v = k.double()
    if change.get("k") == "mixed":
        k, v = k.half(), v
    if change.get("k") == "unaligned":
        k = torch.zeros(k.numel() + 8, dtype=k.dtype, device="cuda")[1:1 + k.numel()].view(k.shape)
    if change.get("v") == "short":
        v = v[:-1]
    if change.get("seq_lens") == "long":
        lens = lens.long()
    if change.get("seq_lens") == "cpu":
        lens = lens.cpu()
    if change.get("table") == "long":
        table = table.long()
    if change.get("score") == "narrow":
        kw.update(score=torch.zeros(2, 20, device="cuda"), max_len=30)
    if change.get("lse") == "half":
        kw["lse"] = torch.zeros(2, 8, dtype=torch.float16, device="cuda")
    if change.get("d") == "odd":
        q, k, v = (x[..., :48].contiguous() for x in (q, k, v))
    if change.get("scale") == "bf16":
        kw["k_scale"] = torch.ones(2, device="cuda")
    with pytest.raises(error):
        hs.paged_decode(q, k, v, table, lens, 1.0, **kw)


@pytest.mark.parametrize("rows,most,page", [(33, 900, 16), (70, 5000, 16), (400, 150, 16),
                                            (1100, 40, 16), (70, 700, 12)])
def test_many_requests(rows, most, page):
    """More requests than a warp has lanes, empty ones among them, first and
    last, and runs of CTAs that span several."""
    g = torch.Generator().manual_seed(rows)
    lens = torch.randint(0, most, (rows,), generator=g)
    lens[torch.rand(rows, generator=g) < 0.3] = 0
    lens[0] = lens[-1] = lens[-2] = 0
    lens[rows // 2] = most
    s = make(lens.tolist(), 8, 4, 64, page, seed=rows, poison=True)
    score = torch.zeros(rows, s["table"].shape[1] * page, device="cuda")
    *_, status = run_and_check(s, score=score)
    assert status == 0


@pytest.mark.parametrize("heads,kv_heads", [(288, 32), (600, 8), (257, 257)])
def test_many_heads(heads, kv_heads):
    s = make([300, 1, 0, 77], heads, kv_heads, 64, 16, seed=heads)
    score = torch.rand(4, s["table"].shape[1] * 16, device="cuda")
    run_and_check(s, score=score, decay=0.5)


def test_nothing_cached():
    s = make([0, 0, -5], 8, 2, 128, 16)
    score = torch.full((3, 16), 4.0, device="cuda")
    out, lse, status = run_and_check(s, score=score)
    assert status == 0 and not out.any() and (lse == -math.inf).all() and (score == 4.0).all()


@pytest.mark.parametrize("page", [16, 32, 48, 64, 7])
@pytest.mark.parametrize("kind,d", [("e4m3", 128), ("e4m3", 256), ("bf16", 128), ("fp16", 64)])
def test_what_is_not_attended_has_no_effect(kind, d, page):
    """NaN behind the contexts and in unused pages, at every way of cutting a
    call (few and many tiles)."""
    for lens in ([33, 1, 100], [3000, 47, 0, 2500, 1777, 900, 31, 4000]):
        s = make(lens, 16, 4, d, page, kind=kind, seed=page + d, poison=True)
        *_, status = run_and_check(s)
        assert status == 0


@pytest.mark.parametrize("page", [16, 32, 5])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_nan_stays_in_its_head(kind, page):
    for lens in ([40, 300], [4000, 2000, 3000, 1500, 2500, 3500]):
        s = make(lens, 16, 8, 128, page, kind=kind, seed=page)
        want, want_lse, _ = run_and_check(s)
        at = s["table"][1, 17 // page].long(), 17 % page
        s["v"][at[0], at[1], 3] = math.nan
        s["k"][at[0], at[1], 6] = math.nan
        out, lse, _ = run_and_check_nonfinite_scaled(s)
        heads = torch.ones(16, dtype=torch.bool, device="cuda")
        heads[6:8] = heads[12:14] = False
        assert torch.isnan(out[1, 6:8]).all() and torch.isnan(out[1, 12:14]).all()
        assert torch.equal(out[1, heads], want[1, heads])
        assert torch.equal(lse[1, :12], want_lse[1, :12]) and torch.isnan(lse[1, 12:14]).all()
        rest = [r for r in range(len(lens)) if r != 1]
        assert torch.equal(out[rest], want[rest]) and torch.equal(lse[rest], want_lse[rest])


def run_and_check_nonfinite_scaled(s):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = hs.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"],
                               k_scale=s["scales"][0], v_scale=s["scales"][1], status=status)
    torch.cuda.synchronize()
    return out, lse, int(status.item())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("scored", [False, True])
def test_extension_and_general_path_agree(kind, scored, monkeypatch):
    """The extension module's common case and the general path of the binding
    make the same call; what the extension does not take is refused as before."""
    hs.lib()
    if hs._binding is None:
        pytest.skip("Python headers were not there at build time")
    taken = []

    class Spy:
        def paged_decode(self, *a):
            taken.append(binding.paged_decode(*a))
            return taken[-1]

    binding = hs._binding
    s = make([100, 7, 0, 333], 8, 2, 128, 16, kind=kind, seed=3)
    n = s["table"].shape[1] * 16
    ws = torch.empty(hs.paged_decode_workspace_bytes(4, 8, 2, 128, n, window=50, num_sinks=4,
                                                     with_score=True),
                     dtype=torch.uint8, device="cuda")
    got = []
    for mod in (Spy(), None):
        monkeypatch.setattr(hs, "_binding", mod)
        score = torch.full((4, n - 3), 0.5, device="cuda") if scored else None
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.empty_like(s["q"])
        lse = torch.empty(4, 8, device="cuda")
        r = hs.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"], window=50,
                            num_sinks=4, k_scale=s["scales"][0], v_scale=s["scales"][1],
                            score=score, score_decay=0.25, out=out, lse=lse, workspace=ws,
                            status=status)
        torch.cuda.synchronize()
        assert r[0] is out and r[1] is lse and int(status) == 0
        got.append((out, lse) + ((score,) if scored else ()))
    assert taken == [0]
    for a, b in zip(*got):
        assert torch.equal(a, b)
    # Left to the general path: a workspace that is too small, a strided query.
    monkeypatch.setattr(hs, "_binding", Spy())
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    wide = torch.empty(4, 8 * 128 + 8, dtype=s["q"].dtype, device="cuda")
    wide[:, :8 * 128] = s["q"].view(4, -1)
    for q, w in ((s["q"], small), (wide[:, :8 * 128].unflatten(1, (8, 128)), ws)):
        out = torch.empty_like(s["q"])
        hs.paged_decode(q, s["k"], s["v"], s["table"], s["lens"], s["scale"], window=50,
                        num_sinks=4, k_scale=s["scales"][0], v_scale=s["scales"][1], out=out,
                        lse=torch.empty(4, 8, device="cuda"), workspace=w)
        assert taken[-1] is None and torch.equal(out, got[0][0])
    with pytest.raises(hs.HSError):  # an error of the C call through the extension
        hs.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"], window=-1,
                        k_scale=s["scales"][0], v_scale=s["scales"][1], out=out,
                        lse=torch.empty(4, 8, device="cuda"), workspace=ws)
    assert taken[-1] == 1


@pytest.mark.parametrize("kw", [dict(window=1 << 32), dict(num_sinks=(1 << 32) + 4)])
def test_sizes_past_32_bits_are_refused(kw):
    s = make([20, 30], 8, 2, 64, 16)
    with pytest.raises(ValueError):
        hs.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"], **kw)


def test_memory_of_a_call_on_another_stream():
    """The workspace that a call makes for itself is not handed out again while
    the other stream still works with it."""
    s = make([3000, 1, 777, 20000], 32, 8, 128, 16, seed=6)
    args = (s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"])
    want, want_lse = hs.paged_decode(*args)
    n = hs.paged_decode_workspace_bytes(4, 32, 8, 128, s["table"].shape[1] * 16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    out, lse = hs.paged_decode(*args, stream=side)
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse) and len(junk) == 3


def test_largest_head_count():
    # Shapes near the limit on heads: the grid of the finishing kernel.
    s = make([40, 0], 65536, 8192, 64, 16)
    run_and_check(s)


def long_bound(s, tokens=200000):
    """The same requests in a table that could hold `tokens` each: the bound on
    the lengths decides how a call is cut."""
    page = s["k"].shape[1]
    pad = max(0, -(-tokens // page) - s["table"].shape[1])
    s["table"] = torch.nn.functional.pad(s["table"], (0, pad), value=-1)
    return s


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (32, 8), (15, 3), (16, 1), (40, 1)])
def test_short_requests_under_a_long_bound(kind, d, heads, kv_heads):
    s = long_bound(make([1, 15, 16, 17, 130, 0, 333], heads, kv_heads, d, 16, kind=kind,
                        seed=d + heads, poison=kind != "e4m3"))
    *_, status = run_and_check(s)
    assert status == 0


@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("lens", [[1], [2, 1], [0, 0], [129, 4097, 7], list(range(1, 70))])
def test_pages_under_a_long_bound(page, lens):
    s = long_bound(make(lens, 8, 2, 64, page, seed=page + len(lens), poison=True))
    score = torch.rand(len(lens), s["table"].shape[1] * page, device="cuda")
    *_, status = run_and_check(s, score=score)
    assert status == 0


@pytest.mark.parametrize("kind,heads,kv_heads,d", [
    ("bf16", 32, 8, 128), ("fp16", 12, 12, 64), ("e4m3", 32, 8, 128), ("bf16", 16, 1, 256),
    ("e4m3", 16, 1, 256), ("bf16", 48, 4, 64), ("fp16", 24, 1, 128)])
@pytest.mark.parametrize("lens", [
    [100], [300], [511], [1000], [1025], [4000], [8192], [500, 0, 3], [0, 900, 0, 128, 127],
    [130] * 12, [7, 256, 0, 64, 200, 0] * 5, [90, 0, 128, 1] * 16, [33] * 128])
def test_units_of_clusters(kind, heads, kv_heads, d, lens):
    """Short bounds: every unit has CTAs of its own, one or a cluster (some
    without a tile), with one KV head or several."""
    s = make(lens, heads, kv_heads, d, 16, kind=kind, seed=len(lens) + d, poison=kind != "e4m3")
    n = s["table"].shape[1] * 16
    out, lse, status = run_and_check(s)
    score = torch.rand(len(lens), n, device="cuda")
    out2, lse2, status2 = run_and_check(s, score=score, decay=0.5)
    assert status == status2 == 0
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("rows,window,sinks", [(1, 700, 4), (3, 130, 0), (18, 256, 4),
                                               (40, 20, 17), (70, 64, 4)])
def test_windows_of_clusters(rows, window, sinks):
    g = torch.Generator().manual_seed(rows)
    lens = torch.randint(0, 3000, (rows,), generator=g)
    lens[0] = 2999
    s = make(lens.tolist(), 32, 8, 128, 16, seed=rows)
    score = torch.rand(rows, s["table"].shape[1] * 16, device="cuda")
    run_and_check(s, window=window, sinks=sinks)
    *_, status = run_and_check(s, window=window, sinks=sinks, score=score)
    assert status == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_clusters_skip_bad_pages(kind):
    """A CTA of a cluster whose pages are all bad has no token to add."""
    s = make([600, 600, 40], 8, 2, 128, 16, kind=kind, seed=4)
    s["table"][0, 8:16] = -1
    s["table"][1, :] = s["k"].shape[0]
    s["table"][2, 1] = 1 << 30
    out, lse, status = run_and_check(s)
    assert status == 6 and not out[1].any() and (lse[1] == -math.inf).all()


@pytest.mark.parametrize("kind,d,heads,kv_heads", [("fp16", 256, 16, 16), ("bf16", 256, 16, 1),
                                                   ("bf16", 128, 32, 8), ("fp16", 64, 8, 8)])
@pytest.mark.parametrize("page", [16, 128])
def test_partial_tiles_many_times(kind, d, heads, kv_heads, page):
    """NaN behind the contexts: a tile's unused rows are cleared after they
    have been loaded and before they are multiplied, however the loads of
    neighbouring tiles fall."""
    g = torch.Generator().manual_seed(d)
    lens = torch.randint(0, 964, (64,), generator=g)
    lens[torch.rand(64, generator=g) < 0.3] = 963
    s = long_bound(make(lens.tolist(), heads, kv_heads, d, page, kind=kind, seed=d, poison=True))
    want, want_lse, _ = run_and_check(s)
    for _ in range(60):
        out, lse = hs.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"])
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_calls_on_two_streams_at_once():
    """Each with its own workspace: dealt calls, clusters and the warp-level
    kernel side by side."""
    shapes = [long_bound(make([3000, 5, 777, 9000], 32, 8, 128, 16, seed=1)),
              make([260] * 16, 64, 8, 128, 16, seed=2), make([1500, 40, 3], 32, 8, 128, 16, seed=3)]
    wants, spaces = [], []
    for s in shapes:
        wants.append(run_and_check(s)[:2])
        n = hs.paged_decode_workspace_bytes(*s["q"].shape[:2], s["k"].shape[2], 128,
                                            s["table"].shape[1] * 16)
        spaces.append([torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)])
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[[] for _ in shapes] for _ in streams]
    torch.cuda.synchronize()
    for it in range(30):
        for j, stream in enumerate(streams):
            i = (it + j) % len(shapes)
            s = shapes[i]
            with torch.cuda.stream(stream):
                outs[j][i].append(hs.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"],
                                                  s["scale"], workspace=spaces[i][j]))
    torch.cuda.synchronize()
    for per_stream in outs:
        for (want, want_lse), got in zip(wants, per_stream):
            assert all(torch.equal(o, want) and torch.equal(l, want_lse) for o, l in got)
