"""The operators of decoding over a whole paged KV cache that is kept to a
budget, as cases to be measured:

  decode   one new token's attention over every cached token of its request
           (hs.paged_decode): GQA / MHA / MQA, bf16, fp16 or E4M3 caches, an
           optional window with sinks;
  scored   the same call, also adding each cached token's attention weight,
           summed over the query heads, to the request's running scores;
  evict    hs.evict: a request that holds more tokens than its budget keeps
           the newest, the sinks and the highest running scores; the kept
           rows behind the budget move into the holes in front of it.

`run` makes the framework's calls where `own` is true and computes the same
with elementary torch operations where it is false.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
WORKSPACE_BYTES = 64 << 20


def _decode(name, rows, heads, kv_heads, d, page, ctx, *, dtype="bf16", ragged=False, pad=0,
            window=0, sinks=0, scored=False):
    return dict(name=name, op="scored" if scored else "decode", rows=rows, heads=heads,
                kv_heads=kv_heads, d=d, page=page, ctx=ctx, dtype=dtype, ragged=ragged, pad=pad,
                window=window, sinks=sinks)


def _evict(name, rows, kv_heads, d, page, ctx, budget, *, recent, sinks, ragged=False, mla=False,
           mixed=False):
    return dict(name=name, op="evict", rows=rows, kv_heads=kv_heads, d=d, page=page, ctx=ctx,
                budget=budget, recent=recent, sinks=sinks, ragged=ragged, mla=mla, mixed=mixed)


def listed():
    return [
        # One user's chat turn: latency is all that counts.
        _decode("decode_one_1k", 1, 32, 8, 128, 64, 1024),
        # A small fp16 model with one KV head per query head, mixed odd lengths.
        _decode("decode_mha_fp16_odd", 8, 12, 12, 64, 16, 777, dtype="fp16", ragged=True),
        # One shared KV head of width 256 for 16 query heads.
        _decode("decode_mqa_256", 24, 16, 1, 256, 32, 5001, ragged=True),
        # A full serving batch, contexts spread up to 64 K tokens.
        _decode("decode_gqa_64k", 16, 32, 8, 128, 16, 65536, ragged=True),
        # One very long document: few rows, all of the GPU on one context.
        _decode("decode_one_131k", 1, 32, 8, 128, 64, 131072),
        # A large batch over an 8-bit cache, the last slots of the batch unused.
        _decode("decode_fp8_8k", 64, 32, 8, 128, 64, 8192, dtype="e4m3", ragged=True, pad=5),
        # A sliding-window layer with sinks in the same batch.
        _decode("decode_window", 16, 32, 8, 128, 16, 65536, window=256, sinks=4),
        # A budgeted cache being scored: the step before an eviction.
        _decode("scored_one_2k", 1, 32, 8, 128, 64, 2049, scored=True),
        _decode("scored_batch_4k", 32, 32, 8, 128, 16, 4113, scored=True, ragged=True),
        # Steady state: each request is one token over its budget.
        _evict("evict_step", 64, 8, 128, 64, 2049, 2048, recent=256, sinks=4, mixed=True),
        # After a prompt: contexts up to 64 K tokens cut to the budget.
        _evict("evict_prompt", 16, 8, 128, 16, 65536, 4096, recent=256, sinks=4, ragged=True),
        # Latent rows (one 1152-byte row per token) cut to the sparse set's size.
        _evict("evict_latent", 32, 1, 576, 64, 32768, 2048, recent=128, sinks=4, mla=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    page = rng.choice([16, 32, 64])
    op = rng.choice(["decode", "decode", "scored", "evict"])
    if op == "evict":
        mla = rng.random() < 0.3
        kv_heads, d = (1, 576) if mla else (rng.choice([1, 2, 4, 8]), rng.choice([64, 128]))
        rows, ctx = _log(rng, 1, 64), _log(rng, 64, 65536)
        while rows * ctx * kv_heads * d > 16 * 65536 * 1024 // 2:
            rows = max(1, rows // 2)
        budget = max(8, min(ctx, _log(rng, max(8, ctx // 16), ctx)))
        return _evict("", rows, kv_heads, d, page, ctx, budget, recent=rng.randrange(0, budget // 2 + 1),
                      sinks=rng.choice([0, 0, 1, 4]), ragged=rng.random() < 0.5, mla=mla, mixed=rng.random() < 0.5)
    kv_heads, d = rng.choice([1, 2, 3, 4, 8, 12]), rng.choice([64, 128, 128, 256])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    rows, ctx = _log(rng, 1, 96), _log(rng, 1, 65536 if op == "decode" else 16384)
    while rows * ctx * kv_heads * d > 16 * 65536 * 1024 // 2:
        rows = max(1, rows // 2)
        if rows == 1:
            ctx = min(ctx, 16384)
    window = rng.choice([0, 0, 0, rng.randrange(1, 600)])
    return _decode("", rows, kv_heads * group, kv_heads, d, page, ctx,
                   dtype=rng.choice(["bf16", "bf16", "fp16", "e4m3"]), ragged=rng.random() < 0.7,
                   pad=rng.choice([0, 0, 1]) if rows > 2 else 0, window=window,
                   sinks=rng.choice([0, 1, 4]) if window else 0, scored=op == "scored")


def _lens(case):
    """Cached tokens per request: all of `ctx`, or spread evenly up to it in a
    mixed order; the last `pad` slots of a batch hold no request."""
    R, T = case["rows"], case["ctx"]
    lens = [T] * R
    if case["ragged"]:
        lens = [max(1, T * ((r * 7) % R + 1) // R) if R % 7 else max(1, T * (r + 1) // R) for r in range(R)]
    for r in range(R - case.get("pad", 0), R):
        lens[r] = 0
    return lens


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda")
    R, T, page = case["rows"], case["ctx"], case["page"]
    blocks = -(-T // page)
    pages = R * blocks
    kvh, d = case["kv_heads"], case["d"]
    table = torch.randperm(pages, generator=g, **dev).to(torch.int32).view(R, blocks)
    lens = torch.tensor(_lens(case), dtype=torch.int32, **dev)
    s = dict(case=case, block_table=table, seq_lens=lens,
             status=torch.zeros(1, dtype=torch.int32, **dev))

    def cache(dt):
        c = torch.randn(pages, page, kvh, d, generator=g, dtype=torch.bfloat16 if dt == torch.float8_e4m3fn
                        else dt, **dev)
        return c.to(dt)

    if case["op"] == "evict":
        s["k_cache"] = cache(torch.bfloat16)
        s["v_cache"] = None if case["mla"] else cache(torch.bfloat16)
        # Running scores: a few heavy tokens, a long tail, and many tokens
        # that no head ever looked at (equal scores).
        u = torch.rand(R, T, generator=g, **dev)
        s["score"] = torch.where(torch.rand(R, T, generator=g, **dev) < 0.1, torch.zeros_like(u),
                                 0.01 / (u + 1e-4))
        # Positions in the order of the prompt or, `mixed`, after evictions:
        # some positions are gone, and rows that filled holes stand anywhere.
        pos = torch.arange(T, dtype=torch.int32, **dev).expand(R, T)
        if case["mixed"]:
            pos = torch.randint(1, 4, (R, T), generator=g, dtype=torch.int32, **dev).cumsum(1, dtype=torch.int32) - 1
        last = pos.gather(1, (lens.long() - 1).clamp_min(0)[:, None])[:, 0]
        s["next_pos"] = torch.where(lens > 0, last + 1, 0).to(torch.int32)
        if case["mixed"]:
            key = torch.rand(R, T, generator=g, **dev)
            key[torch.arange(T, **dev)[None] >= lens[:, None]] = 2.0
            pos = pos.gather(1, key.argsort(1))
        s["positions"] = pos.contiguous()
        s["score_out"] = torch.rand(R, T, generator=g, **dev)
        s["positions_out"] = torch.full((R, T), -1, dtype=torch.int32, **dev)
        s["lens_out"] = torch.zeros(R, dtype=torch.int32, **dev)
        s["moves"] = (torch.zeros(R, case["budget"], dtype=torch.int32, **dev),
                      torch.zeros(R, case["budget"], dtype=torch.int32, **dev),
                      torch.zeros(R, dtype=torch.int32, **dev))
        return s
    kv = DTYPES[case["dtype"]]
    qt = torch.float16 if kv == torch.float16 else torch.bfloat16
    s["q"] = torch.randn(R, case["heads"], d, generator=g, dtype=qt, **dev)
    s["k_cache"], s["v_cache"] = cache(kv), cache(kv)
    s["k_scale"] = s["v_scale"] = None
    if kv == torch.float8_e4m3fn:
        s["k_scale"] = torch.rand(kvh, generator=g, **dev) + 0.5
        s["v_scale"] = torch.rand(kvh, generator=g, **dev) + 0.5
    s["scale"] = 1.0 / math.sqrt(d)
    s["score"] = torch.rand(R, T, generator=g, **dev) if case["op"] == "scored" else None
    s["out"] = torch.zeros(R, case["heads"], d, dtype=qt, **dev)
    s["lse"] = torch.zeros(R, case["heads"], **dev)
    s["workspace"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, **dev)
    return s


def run(s):
    c = s["case"]
    if own:
        from sparse_top_kv_gb300 import hs
        if c["op"] == "evict":
            hs.evict(s["score"], s["seq_lens"], c["budget"], s["k_cache"], s["v_cache"], s["block_table"],
                     recent=c["recent"], num_sinks=c["sinks"], positions=s["positions"],
                     next_pos=s["next_pos"], score_out=s["score_out"], positions_out=s["positions_out"],
                     lens_out=s["lens_out"], moves=s["moves"], status=s["status"])
            out = [s["lens_out"], s["moves"][2], s["score_out"], s["positions_out"], s["k_cache"]]
            return out if s["v_cache"] is None else out + [s["v_cache"]]
        hs.paged_decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], s["scale"],
                        window=c["window"], num_sinks=c["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                        score=s["score"], out=s["out"], lse=s["lse"], workspace=s["workspace"],
                        status=s["status"])
        return [s["out"], s["lse"]] if s["score"] is None else [s["out"], s["lse"], s["score"]]
    return _plain_evict(s, c) if c["op"] == "evict" else _plain_decode(s, c)


def _plain_decode(s, c):
    lens = s["seq_lens"].long()[:, None]
    if c["window"]:
        # The positions that the window and the sinks reach, nothing else.
        win = torch.arange(c["window"], device="cuda")[None] + (lens - c["window"]).clamp_min(0)
        snk = torch.arange(c["sinks"], device="cuda")[None].expand(c["rows"], -1)
        live = torch.cat([win < lens, (snk < lens) & (snk < (lens - c["window"]))], 1)
        pos = torch.cat([win, snk], 1).clamp_max(c["ctx"] - 1)
    else:
        pos = torch.arange(c["ctx"], device="cuda")[None].expand(c["rows"], -1)
        live = pos < lens
    slot = s["block_table"].long().gather(1, pos // c["page"]) * c["page"] + pos % c["page"]
    slot = torch.where(live, slot, 0)
    k = s["k_cache"].flatten(0, 1)[slot].float()
    v = s["v_cache"].flatten(0, 1)[slot].float()
    if s["k_scale"] is not None:
        k = k * s["k_scale"][:, None]
        v = v * s["v_scale"][:, None]
    q = s["q"].float().view(c["rows"], c["kv_heads"], -1, c["d"])
    x = torch.einsum("rgud,rtgd->rgut", q, k) * s["scale"]
    x = torch.where(live[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    l = p.sum(-1, keepdim=True)
    lse = (torch.log(l) + m).view(c["rows"], -1)
    w = p / torch.where(l > 0, l, 1.0)
    out = torch.einsum("rgut,rtgd->rgud", w, v).reshape(s["q"].shape).to(s["q"].dtype)
    if s["score"] is None:
        return [out, lse]
    s["score"].scatter_add_(1, pos, w.sum((1, 2)))
    return [out, lse, s["score"]]


def _plain_evict(s, c):
    R, T, B, page = c["rows"], c["ctx"], c["budget"], c["page"]
    lens = s["seq_lens"].long()[:, None]
    idx = torch.arange(T, device="cuda")[None].expand(R, -1)
    live = idx < lens
    kept_anyway = live & ((s["positions"] < c["sinks"]) | (s["positions"] >= s["next_pos"][:, None] - c["recent"]))
    # Order: the tokens that are kept anyway, then by score, then by index.
    by_score = torch.sort(s["score"], dim=1, descending=True, stable=True).indices
    kind = (kept_anyway.int() + live.int()).gather(1, by_score)
    order = by_score.gather(1, torch.sort(kind, dim=1, descending=True, stable=True).indices)
    rank = torch.empty_like(order).scatter_(1, order, idx)
    keep = live & (rank < B)
    hole, tail = live & ~keep & (idx < B), keep & (idx >= B)
    src = torch.sort(torch.where(tail, idx, T), dim=1).values
    take = torch.where(hole, src.gather(1, (hole.long().cumsum(1) - 1).clamp_min(0)), idx)[:, :B]
    new_lens = lens.clamp_max(B)
    stay = idx[:, :B] < new_lens
    s["lens_out"].copy_(new_lens[:, 0])
    s["moves"][2].copy_(hole.sum(1))
    for name in ("score", "positions"):
        out = s[name + "_out"]
        out[:, :B] = torch.where(stay, s[name].gather(1, take), out[:, :B])
    # The places that the request gives up start from 0 for the next token there.
    s["score_out"].copy_(torch.where((idx >= new_lens) & live, 0.0, s["score_out"]))
    table = s["block_table"].long()
    dst = table.gather(1, idx[:, :B] // page) * page + idx[:, :B] % page
    frm = table.gather(1, take // page) * page + take % page
    caches = [s["k_cache"]] if s["v_cache"] is None else [s["k_cache"], s["v_cache"]]
    for cache in caches:
        rows = cache.flatten(0, 1)
        rows[dst.flatten()] = rows[frm.flatten()]
    return [s["lens_out"], s["moves"][2], s["score_out"], s["positions_out"]] + caches


def exact(case, seed):
    """What `run` returns, request by request from the definition in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(s, case)
    R, H, G, d, page = case["rows"], case["heads"], case["kv_heads"], case["d"], case["page"]
    out = torch.zeros(R, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((R, H), -math.inf, dtype=torch.float64, device="cuda")
    score = None if s["score"] is None else s["score"].double()
    for r, n in enumerate(_lens(case)):
        t = list(range(n))
        if case["window"]:
            t = [i for i in t if i >= n - case["window"] or i < case["sinks"]]
        if not t:
            continue
        t = torch.tensor(t, device="cuda")
        at = s["block_table"][r].long()[torch.div(t, page, rounding_mode="floor")], t % page
        for g in range(G):
            K, V = s["k_cache"][at][:, g].double(), s["v_cache"][at][:, g].double()
            if s["k_scale"] is not None:
                K, V = K * s["k_scale"][g].double(), V * s["v_scale"][g].double()
            hs_ = slice(g * (H // G), (g + 1) * (H // G))
            z = s["q"][r, hs_].double() @ K.T / math.sqrt(d)
            lse[r, hs_] = torch.logsumexp(z, 1)
            w = torch.exp(z - lse[r, hs_, None])
            out[r, hs_] = w @ V
            if score is not None:
                score[r].index_add_(0, t, w.sum(0))
    return [out, lse] if score is None else [out, lse, score]


def _exact_evict(s, case):
    score, pos = s["score"].cpu().numpy().astype(np.float64), s["positions"].cpu().numpy()
    nxt, B = s["next_pos"].cpu().numpy(), case["budget"]
    score_out, pos_out = s["score_out"].cpu().numpy().astype(np.float64), s["positions_out"].cpu().numpy()
    lens, moved = np.zeros(case["rows"], np.int32), np.zeros(case["rows"], np.int32)
    for r, n in enumerate(_lens(case)):
        order = np.arange(n)
        if n > B:
            safe = (pos[r, :n] < case["sinks"]) | (pos[r, :n] >= nxt[r] - case["recent"])
            kept = np.lexsort((np.arange(n), -score[r, :n], ~safe))[:B]
            holes = np.setdiff1d(np.arange(B), kept)
            order = np.arange(B)
            order[holes] = np.sort(kept[kept >= B])
            moved[r] = len(holes)
        lens[r] = len(order)
        score_out[r, len(order):n] = 0.0
        score_out[r, :len(order)], pos_out[r, :len(order)] = score[r][order], pos[r][order]
    return [lens, moved, score_out, pos_out, None] + ([] if s["v_cache"] is None else [None])


def work(case):
    R, d, lens = case["rows"], case["d"], _lens(case)
    if case["op"] == "evict":
        row = case["kv_heads"] * d * 2 * (1 if case["mla"] else 2)
        # Scores and positions read once, the kept ones written once, the given
        # up scores cleared; the
        # moved rows (as many as kept tokens lie behind the budget, taken as
        # spread evenly over the context) read and written once.
        B = case["budget"]
        moved = sum(-(-(n - B) * B // n) for n in lens if n > B)
        return {"bytes": sum(8 * n + 8 * min(n, B) + 4 * max(0, n - B) for n in lens) + 2 * row * moved, "flops": 0.0}
    if case["window"]:
        lens = [min(n, case["window"] + case["sinks"]) for n in lens]
    elt = 1 if case["dtype"] == "e4m3" else 2
    n = sum(lens)
    byt = 2 * n * case["kv_heads"] * d * elt + 2 * R * case["heads"] * d * 2 + 4 * R * case["heads"]
    byt += 4 * sum(-(-x // case["page"]) for x in lens) + (8 * n if case["op"] == "scored" else 0)
    return {"bytes": byt, "flops": 4.0 * n * case["heads"] * d}
