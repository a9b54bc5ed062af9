"""The operators of serving new tokens over a paged KV cache, several of a
request at once, as cases to be measured:

  extend   requests grow by a step's new tokens or give tokens up: pages from
           and to a ring of free ones, the block tables, and for each token
           its request, position and slot (hs.paged_extend);
  rope     rotary positions on the step's queries and keys, and the rotated
           keys and the values into their slots of the cache (hs.rope_append);
  prefill  the step's queries, causally, over every cached token of their
           request, the step's own among them (hs.paged_prefill).

`run` makes the framework's calls where `own` is true and computes the same
with elementary torch operations where it is false.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
WORKSPACE_BYTES = 128 << 20
CELLS = 1 << 31  # attention weights of a call, all heads: bounds the plain form's memory


def _extend(name, rows, page, ctx, chunk, *, mixed=False, tight=False, pad=0):
    return dict(name=name, op="extend", rows=rows, page=page, ctx=ctx, chunk=chunk, mixed=mixed,
                tight=tight, pad=pad)


def _rope(name, rows, chunk, heads, kv_heads, d, rot, page, ctx, *, dtype="bf16", cache=None,
          interleaved=False, factor=1.0, pad=0):
    return dict(name=name, op="rope", rows=rows, chunk=chunk, heads=heads, kv_heads=kv_heads, d=d,
                rot=rot, page=page, ctx=ctx, dtype=dtype, cache=cache or dtype,
                interleaved=interleaved, factor=factor, pad=pad)


def _prefill(name, rows, chunk, heads, kv_heads, d, page, ctx, *, dtype="bf16", cache=None,
             ragged=False, window=0, sinks=0, pad=0):
    return dict(name=name, op="prefill", rows=rows, chunk=chunk, heads=heads, kv_heads=kv_heads,
                d=d, page=page, ctx=ctx, dtype=dtype, cache=cache or dtype, ragged=ragged,
                window=window, sinks=sinks, pad=pad)


def listed():
    return [
        # A decode step of a serving batch: every request grows by one token.
        _extend("extend_step", 64, 16, 8192, 1),
        # A busy server's step: prompts of up to 1 K tokens enter, most
        # requests decode, some end or take back guessed tokens.
        _extend("extend_mixed", 512, 16, 8192, 1024, mixed=True, pad=777),
        # One user's decode step: latency is all that counts.
        _rope("rope_one", 1, 1, 32, 8, 128, 128, 64, 1024),
        # A long prompt's chunk, positions stretched to a long context.
        _rope("rope_chunk", 2, 4096, 32, 8, 128, 128, 64, 65536, factor=8.0),
        # Half of each head rotated, neighbouring pairs, into an 8-bit cache.
        _rope("rope_fp8_odd", 9, 457, 16, 4, 128, 64, 16, 5001, cache="e4m3", interleaved=True,
              pad=5),
        # A chat turn's short message on top of a cached conversation.
        _prefill("prefill_turn", 1, 32, 32, 8, 128, 64, 1024),
        # Guessed tokens being verified: few per request, long contexts.
        _prefill("prefill_verify", 16, 5, 32, 8, 128, 16, 8192, ragged=True),
        # Fresh prompts of odd lengths, a small fp16 model with one KV head per
        # query head.
        _prefill("prefill_fresh_fp16", 8, 777, 12, 12, 64, 16, 777, dtype="fp16", ragged=True,
                 pad=3),
        # One chunk of a long document.
        _prefill("prefill_chunk_32k", 1, 2048, 32, 8, 128, 64, 32768),
        # A sliding-window layer with sinks.
        _prefill("prefill_window", 4, 1024, 32, 8, 128, 16, 16384, window=1024, sinks=4),
        # A batch of chunks over an 8-bit cache.
        _prefill("prefill_fp8", 8, 512, 32, 8, 128, 64, 8192, cache="e4m3", ragged=True),
        # One shared KV head of width 256 for 16 query heads.
        _prefill("prefill_mqa_256", 4, 513, 16, 1, 256, 32, 5001, ragged=True, pad=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    op = rng.choice(["extend", "rope", "prefill", "prefill", "prefill"])
    page = rng.choice([16, 32, 64])
    if op == "extend":
        rows, ctx = _log(rng, 1, 1024), _log(rng, 64, 16384)
        mixed = rng.random() < 0.6
        chunk = min(_log(rng, 1, 2048), ctx) if mixed else rng.choice([1, 1, 2, 5])
        while rows * ctx > 512 * 8192:
            rows //= 2
        return _extend("", rows, page, ctx, chunk, mixed=mixed, tight=rng.random() < 0.3,
                       pad=rng.choice([0, 1, 129]))
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    cache = rng.choice([dtype, dtype, "e4m3"])
    kv_heads, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 128, 256])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    rows, chunk = _log(rng, 1, 32), _log(rng, 1, 4096)
    if op == "rope":
        while rows * chunk * (heads + 2 * kv_heads) * d > 8192 * 48 * 128:
            chunk = max(1, chunk // 2)
            rows = rows if chunk > 1 else max(1, rows // 2)
        return _rope("", rows, chunk, heads, kv_heads, d, d // rng.choice([1, 1, 2, 4]), page,
                     chunk + rng.randrange(0, 4096), dtype=dtype, cache=cache,
                     interleaved=rng.random() < 0.5, factor=rng.choice([1.0, 1.0, 4.0, 32.0]),
                     pad=rng.choice([0, 1, 33]))
    ctx = max(chunk, _log(rng, 1, 32768))
    while rows * chunk * ctx * heads > CELLS or rows * ctx * kv_heads * d > 1 << 28:
        rows, chunk = max(1, rows // 2), max(1, chunk // 2)
        if rows * chunk == 1:
            ctx = max(1, ctx // 2)
    window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    return _prefill("", rows, chunk, heads, kv_heads, d, page, ctx, dtype=dtype, cache=cache,
                    ragged=rng.random() < 0.6, window=window,
                    sinks=rng.choice([0, 1, 4]) if window else 0, pad=rng.choice([0, 0, 7]))


def _spread(n, i, rows):
    """n times a number in (0, 1], each of rows / rows, in a mixed order."""
    k = (i * 7) % rows + 1 if rows % 7 else i + 1
    return max(1, n * k // rows)


def _step_lens(case):
    """(tokens held before the step, tokens asked for) of each request."""
    lens, new = [], []
    for r in range(case["rows"]):
        held = _spread(case["ctx"], r, case["rows"])
        n = case["chunk"]
        if case["mixed"]:
            if r % 8 == 0:
                held, n = 0, _spread(case["chunk"], r, case["rows"])  # a prompt enters
            else:
                n = 0 if r % 8 == 3 else -held if r % 8 == 5 else -3 if r % 16 == 9 else 1
        lens.append(held)
        new.append(n)
    return lens, new


def _chunk_lens(case):
    """(tokens with the step's, the step's tokens) of each request."""
    R = case["rows"]
    if not case.get("ragged"):
        return [case["ctx"]] * R, [case["chunk"]] * R
    new = [_spread(case["chunk"], r, R) for r in range(R)]
    return [max(n, _spread(case["ctx"], R - 1 - r, R)) for r, n in enumerate(new)], new


def _inv_freq(case):
    """Frequencies whose long waves are stretched by the context's factor: the
    dims that turn less than once over the first 4096 tokens entirely, those
    that turn more than 32 times not at all (the ramp between is linear)."""
    inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])
    if case["factor"] == 1.0:
        return inv, 1.0
    turns = 4096 * inv / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    return inv * keep + inv / case["factor"] * (1 - keep), 0.1 * math.log(case["factor"]) + 1


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    R, page = case["rows"], case["page"]
    s = dict(case=case, status=torch.zeros(1, **i32))
    if case["op"] == "extend":
        lens, new = _step_lens(case)
        blocks = -(-(case["ctx"] + case["chunk"]) // page)
        used = sum(-(-n // page) for n in lens)
        grown = sum(-(-(n + max(m, 0)) // page) for n, m in zip(lens, new)) - used
        pages = used + max(1, grown // 2 if case["tight"] else grown + 7)
        perm = torch.randperm(pages, generator=g, **dev).to(torch.int32)
        held = torch.tensor([-(-n // page) for n in lens], **dev)
        at = held.cumsum(0) - held
        j = torch.arange(blocks, **dev)
        s["block_table"] = torch.where(j < held[:, None], perm[(at[:, None] + j).clamp_max(used - 1)], -1)
        # The ring stands anywhere: as many pages were taken as came back.
        start = int(torch.randint(0, 1 << 40, (1,), generator=g, **dev))
        s["free_ring"] = torch.full((pages,), -1, **i32)
        s["free_ring"][(start + torch.arange(pages - used, **dev)) % pages] = perm[used:]
        s["ring_pos"] = torch.tensor([start, start + pages - used], dtype=torch.int64, **dev)
        s["seq_lens"] = torch.tensor(lens, **i32)
        s["new_lens"] = torch.tensor(new, **i32)
        s["max_tokens"] = N = sum(max(0, n) for n in new) + case["pad"]
        s["lens_out"], s["attend_lens"] = torch.zeros(R, **i32), torch.zeros(R, **i32)
        s["ring_out"] = torch.zeros(2, dtype=torch.int64, **dev)
        s["cu_new"] = torch.zeros(R + 1, **i32)
        for name in ("slot", "row_req", "positions"):
            s[name] = torch.zeros(N, **i32)
        return s
    dtype, kv = DTYPES[case["dtype"]], DTYPES[case["cache"]]
    H, G, d = case["heads"], case["kv_heads"], case["d"]
    blocks = -(-case["ctx"] // page)
    pages = R * blocks
    table = torch.randperm(pages, generator=g, **dev).to(torch.int32).view(R, blocks)
    s["k_scale"] = s["v_scale"] = None
    if kv == torch.float8_e4m3fn:
        s["k_scale"] = torch.rand(G, generator=g, **dev) + 0.5
        s["v_scale"] = torch.rand(G, generator=g, **dev) + 0.5
    lens, new = _chunk_lens(case)
    N = sum(new) + case["pad"]

    def rows_of(n, heads):
        return torch.randn(n, heads, d, generator=g, dtype=dtype, **dev)

    if case["op"] == "rope":
        # The rows of one product, as a fused projection leaves them.
        qkv = torch.randn(N, (H + 2 * G) * d, generator=g, dtype=dtype, **dev)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, d)) for x in qkv.split([H * d, G * d, G * d], 1))
        inv, s["mscale"] = _inv_freq(case)
        s["inv_freq"] = inv.cuda()
        # Turns per position as 64-bit binary fractions.
        s["turns"] = (s["inv_freq"] / (2 * math.pi) * 2.0 ** 64).to(torch.int64)
        t = torch.arange(case["ctx"] - case["chunk"], case["ctx"], **dev).expand(R, -1)
        slot = table.long().gather(1, t // page) * page + t % page
        s["slot"], s["positions"] = torch.full((N,), -1, **i32), torch.full((N,), -1, **i32)
        s["slot"][:t.numel()] = slot.flatten().to(torch.int32)
        s["positions"][:t.numel()] = t.flatten().to(torch.int32)
        s["q_out"] = torch.zeros(N, H, d, dtype=dtype, **dev)
        s["k_cache"] = torch.zeros(pages, page, G, d, dtype=dtype, **dev).to(kv)
        s["v_cache"] = torch.zeros(pages, page, G, d, dtype=dtype, **dev).to(kv)
        return s
    s["block_table"] = table
    s["k_cache"] = torch.randn(pages, page, G, d, generator=g, dtype=dtype, **dev).to(kv)
    s["v_cache"] = torch.randn(pages, page, G, d, generator=g, dtype=dtype, **dev).to(kv)
    s["q"] = rows_of(N, H)
    s["cu_new"] = torch.tensor([0] + new, **dev).cumsum(0).to(torch.int32)
    s["seq_lens"] = torch.tensor(lens, **i32)
    s["scale"] = 1.0 / math.sqrt(d)
    s["out"] = torch.zeros(N, H, d, dtype=dtype, **dev)
    s["lse"] = torch.zeros(N, H, **dev)
    s["workspace"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, **dev)
    return s


def run(s):
    c = s["case"]
    if own:
        from sparse_top_kv_gb300 import hs
        if c["op"] == "extend":
            hs.paged_extend(s["new_lens"], s["seq_lens"], s["block_table"], s["free_ring"],
                            s["ring_pos"], c["page"], s["max_tokens"], lens_out=s["lens_out"],
                            attend_lens=s["attend_lens"], ring_out=s["ring_out"],
                            cu_new=s["cu_new"], slot=s["slot"], row_req=s["row_req"],
                            positions=s["positions"], status=s["status"])
            return _extend_outputs(s)
        if c["op"] == "rope":
            hs.rope_append(s["q"], s["k"], s["v"], s["positions"], s["slot"], s["turns"],
                           s["k_cache"], s["v_cache"], interleaved=c["interleaved"],
                           mscale=s["mscale"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                           q_out=s["q_out"], status=s["status"])
            return [s["q_out"], s["k_cache"], s["v_cache"]]
        hs.paged_prefill(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_new"],
                         s["seq_lens"], s["scale"], window=c["window"], num_sinks=c["sinks"],
                         k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"], lse=s["lse"],
                         workspace=s["workspace"], status=s["status"])
        return [s["out"], s["lse"]]
    return {"extend": _plain_extend, "rope": _plain_rope, "prefill": _plain_prefill}[c["op"]](s, c)


def _extend_outputs(s):
    return [s["block_table"], s["free_ring"], s["ring_out"], s["lens_out"], s["attend_lens"],
            s["cu_new"], s["slot"], s["row_req"], s["positions"]]


def _plain_extend(s, c):
    page, (R, blocks) = c["page"], s["block_table"].shape
    held, new = s["seq_lens"].long(), s["new_lens"].long()
    ask, pages = new.clamp_min(0), s["free_ring"].numel()
    cu = torch.cat([ask.new_zeros(1), ask.cumsum(0)])
    full = -(-held // page)
    fits = (held + ask <= blocks * page) & (cu[1:] <= s["max_tokens"])
    need = torch.where(fits, -(-(held + ask) // page) - full, 0)
    upto = need.cumsum(0)
    served = fits & ((need == 0) | (upto <= s["ring_pos"][1] - s["ring_pos"][0]))
    need = torch.where(served, need, 0)
    lens = torch.where(served, (held + new).clamp_min(0), held)
    back = (full - -(-lens // page)).clamp_min(0)
    at, to = need.cumsum(0) - need, back.cumsum(0) - back
    j = torch.arange(blocks, device="cuda")
    # Pages taken, in the order of the requests and their blocks; pages given
    # back, likewise, behind the ring's last one.
    i = j - full[:, None]
    take = (i >= 0) & (i < need[:, None])
    page_at = (s["ring_pos"][0] + at[:, None] + i) % pages
    i = j - (full - back)[:, None]
    give = (i >= 0) & (i < back[:, None])
    to_at = (s["ring_pos"][1] + to[:, None] + i) % pages
    s["free_ring"][to_at[give]] = s["block_table"][give]
    s["block_table"].copy_(torch.where(take, s["free_ring"][page_at], s["block_table"]))
    t = torch.arange(s["max_tokens"], device="cuda")
    row = torch.searchsorted(cu, t, right=True) - 1
    live = row < R
    row = row.clamp_max(R - 1)
    live = live & served[row]
    pos = torch.where(live, held[row] + t - cu[row], 0)
    slot = s["block_table"][row, pos // page] * page + pos % page
    s["ring_out"].copy_(s["ring_pos"] + torch.stack([need.sum(), back.sum()]))
    s["lens_out"].copy_(lens)
    s["attend_lens"].copy_(torch.where(served & (ask > 0), lens, 0))
    s["cu_new"].copy_(cu)
    s["slot"].copy_(torch.where(live, slot, -1))
    s["row_req"].copy_(torch.where(live, row, -1))
    s["positions"].copy_(torch.where(live, pos, -1))
    return _extend_outputs(s)


def _plain_rope(s, c):
    half, live = c["rot"] // 2, s["positions"] >= 0
    angle = s["positions"][live].double()[:, None] * s["inv_freq"]
    cos, sin = (f(angle).float()[:, None] * s["mscale"] for f in (torch.cos, torch.sin))

    def rotate(x):
        x = x[live].float()
        a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if c["interleaved"] else (
            x[..., :half], x[..., half:2 * half])
        y = (a * cos - b * sin, a * sin + b * cos)
        y = torch.stack(y, -1).flatten(-2) if c["interleaved"] else torch.cat(y, -1)
        return torch.cat([y, x[..., 2 * half:]], -1)

    def put(cache, x, scale):
        if scale is not None:
            x = (x / scale[:, None]).clamp(-448.0, 448.0)
        cache.view(-1, c["kv_heads"], c["d"])[s["slot"][live].long()] = x.to(cache.dtype)

    s["q_out"][live] = rotate(s["q"]).to(s["q_out"].dtype)
    put(s["k_cache"], rotate(s["k"]), s["k_scale"])
    put(s["v_cache"], s["v"][live].float(), s["v_scale"])
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _plain_prefill(s, c):
    R, G, d, page = c["rows"], c["kv_heads"], c["d"], c["page"]
    cu, T = s["cu_new"].long(), s["seq_lens"].long()
    new, ctx = cu[1:] - cu[:-1], c["ctx"]
    i = torch.arange(c["chunk"], device="cuda")
    t = torch.arange(ctx, device="cuda")
    live = i < new[:, None]
    at = torch.where(live, cu[:-1, None] + i, 0)
    slot = s["block_table"].long()[:, t // page] * page + t % page
    k, v = s["k_cache"].flatten(0, 1)[slot].float(), s["v_cache"].flatten(0, 1)[slot].float()
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][:, None], v * s["v_scale"][:, None]
    inside = (t < T[:, None])[:, :, None, None]
    k, v = torch.where(inside, k, 0.0), torch.where(inside, v, 0.0)
    q = s["q"][at].float().view(R, c["chunk"], G, -1, d)
    x = torch.einsum("rigud,rtgd->rguit", q, k).mul_(s["scale"])
    pos = (T - new)[:, None, None] + i[:, None]
    see = t <= pos
    if c["window"]:
        see = see & ((t > pos - c["window"]) | (t < c["sinks"]))
    x.masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    l = x.sum(-1, keepdim=True)
    lse = (torch.log(l) + m).squeeze(-1)
    out = torch.einsum("rguit,rtgd->riugd", x, v) / torch.where(l > 0, l, 1.0).permute(0, 3, 2, 1, 4)
    s["out"][at[live]] = out.transpose(2, 3).flatten(2, 3)[live].to(s["out"].dtype)
    s["lse"][at[live]] = lse.permute(0, 3, 1, 2).flatten(2)[live]
    return [s["out"], s["lse"]]


def exact(case, seed):
    """What `run` returns, request by request from the definition in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "extend":
        return _exact_extend(s, case)
    if case["op"] == "rope":
        return _exact_rope(s, case)
    G, d, page = case["kv_heads"], case["d"], case["page"]
    lens, new = _chunk_lens(case)
    out, lse = torch.zeros_like(s["out"], dtype=torch.float64), torch.zeros_like(s["lse"], dtype=torch.float64)
    u = case["heads"] // G
    first = 0
    for r, (T, n) in enumerate(zip(lens, new)):
        where = torch.arange(T, device="cuda")
        pages = s["block_table"][r].long()[torch.div(where, page, rounding_mode="floor")]
        for g in range(G):
            K, V = s["k_cache"][pages, where % page, g].double(), s["v_cache"][pages, where % page, g].double()
            if s["k_scale"] is not None:
                K, V = K * s["k_scale"][g].double(), V * s["v_scale"][g].double()
            for j in range(0, n, 512):
                p = torch.arange(j, min(n, j + 512), device="cuda")
                Q = s["q"][first + p, g * u:(g + 1) * u].double()
                z = torch.einsum("ihd,td->iht", Q, K) / math.sqrt(d)
                ahead = where[None] - (T - n + p)[:, None]
                hidden = ahead > 0
                if case["window"]:
                    hidden |= (ahead <= -case["window"]) & (where[None] >= case["sinks"])
                z[hidden[:, None].expand_as(z)] = -math.inf
                le = torch.logsumexp(z, 2)
                lse[first + p, g * u:(g + 1) * u] = le
                out[first + p, g * u:(g + 1) * u] = torch.exp(z - le[..., None]) @ V
        first += n
    return [out, lse]


def _exact_rope(s, case):
    G, rot, page = case["kv_heads"], case["rot"], case["page"]
    n = case["rows"] * case["chunk"]
    pos, slot = s["positions"][:n].double(), s["slot"][:n].long()
    turn = torch.polar(torch.full((1,), float(s["mscale"]), dtype=torch.float64, device="cuda"),
                       pos[:, None] * s["inv_freq"][None])[:, None]

    def spun(x):
        x = x[:n].double()
        y = x.clone()
        pair = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (
            slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(x[..., pair[0]].contiguous(), x[..., pair[1]].contiguous()) * turn
        y[..., pair[0]], y[..., pair[1]] = z.real, z.imag
        return y

    q = torch.zeros_like(s["q_out"], dtype=torch.float64)
    q[:n] = spun(s["q"])
    caches = []
    for x, scale in ((spun(s["k"]), s["k_scale"]), (s["v"][:n].double(), s["v_scale"])):
        c = torch.zeros(s["k_cache"].shape, dtype=torch.float64, device="cuda")
        if scale is not None:
            x = (x / scale.double()[:, None]).clamp(-448, 448)
        c[torch.div(slot, page, rounding_mode="floor"), slot % page] = x.view(n, G, -1)
        caches.append(c)
    return [q] + caches


def _exact_extend(s, case):
    page, N = case["page"], s["max_tokens"]
    table, ring = s["block_table"].cpu().numpy().copy(), s["free_ring"].cpu().numpy().copy()
    taken, back = (int(x) for x in s["ring_pos"].cpu())
    lens, new = _step_lens(case)
    rows, pages, blocks = case["rows"], len(ring), table.shape[1]
    lens_out, attend = np.array(lens, np.int32), np.zeros(rows, np.int32)
    cu = np.zeros(rows + 1, np.int32)
    slot, req, pos = (np.full(N, -1, np.int32) for _ in range(3))
    free, asked = back - taken, 0
    given = []
    for r, (held, n) in enumerate(zip(lens, new)):
        first = int(cu[r])
        cu[r + 1] = first + max(0, n)
        have = -(-held // page)
        if n < 0:
            lens_out[r] = max(0, held + n)
            given.extend(table[r, -(-int(lens_out[r]) // page):have])
        if n <= 0 or held + n > blocks * page or first + n > N:
            continue
        need = -(-(held + n) // page) - have
        asked += need
        if need and asked > free:
            continue
        for b in range(have, have + need):
            table[r, b] = ring[taken % pages]
            taken += 1
        lens_out[r] = attend[r] = held + n
        for i in range(n):
            p = held + i
            slot[first + i], req[first + i], pos[first + i] = table[r, p // page] * page + p % page, r, p
    for p in given:
        ring[back % pages] = p
        back += 1
    return [table, ring, np.array([taken, back], np.int64), lens_out, attend, cu, slot, req, pos]


def work(case):
    if case["op"] == "extend":
        lens, new = _step_lens(case)
        page = case["page"]
        moved = sum(abs(-(-max(0, n + m) // page) - -(-n // page)) for n, m in zip(lens, new))
        # Lengths in and out, slots, requests and positions of the tokens, and
        # the pages that change hands (and the tail block of each that grows).
        return {"bytes": 20 * len(lens) + 12 * (sum(max(0, m) for m in new) + case["pad"])
                + 8 * moved + 4 * sum(m > 0 for m in new), "flops": 0.0}
    H, G, d = case["heads"], case["kv_heads"], case["d"]
    elt = 1 if case["cache"] == "e4m3" else 2
    lens, new = _chunk_lens(case)
    n = sum(new)
    if case["op"] == "rope":
        return {"bytes": n * ((2 * H + 2 * G) * d * 2 + 2 * G * d * elt + 8),
                "flops": 3.0 * n * (H + G) * case["rot"]}
    window, sinks = case["window"], case["sinks"]
    cells = tokens = 0
    for T, m in zip(lens, new):
        seen = np.arange(T - m + 1, T + 1, dtype=np.int64)
        first = T - m + 1 - window if window else 0  # the first query's oldest token
        if window:
            seen = np.minimum(seen, window) + np.minimum(np.maximum(seen - window, 0), sinks)
        cells += int(seen.sum())
        tokens += T - max(0, first) + (min(sinks, max(0, first)) if window else 0)
    return {"bytes": 2 * tokens * G * d * elt + 2 * n * H * d * 2 + 4 * n * H + 8 * len(lens)
            + 4 * sum(-(-t // case["page"]) for t in lens), "flops": 4.0 * cells * H * d}
