"""Plain 64-bit definitions of the paged-cache operators, request by request,
with the error bounds that follow from the kernels' number formats.  Shares no
code with the package."""
import math

import torch


def visible(T, window, sinks):
    """Positions that a request of T tokens attends to."""
    return [t for t in range(T) if not window or t >= T - window or t < sinks]


def paged_decode(q, k, v, table, lens, scale, *, window=0, sinks=0, max_len=None, k_scale=None,
                 v_scale=None, score=None, decay=1.0):
    """(out, lse, score, tolerances) in float64 on q's device.  k, v
    [pages, page_size, kv_heads, d]; pages outside the cache are skipped.

    Tolerances, with u = 2^-24 and tensor-core sums that may truncate (2 u an
    addition): a logit is off by dx <= (d + 4) 2u scale max_t sum|q_i k_i| +
    4 u max|x| (the sum, the scale and its exp2 form); a weight by a factor 1 +-
    2 (dx + 8 u) (its exponential and the sum's); the carried P by 2^-16 (two
    bf16 parts); the sums over T tokens by 2 u T.  The output then rounds once:
    eps / 2 of its type."""
    R, H, d = q.shape
    P, page, G, _ = k.shape
    group, dev = H // G, q.device
    out = torch.zeros(R, H, d, dtype=torch.float64, device=dev)
    lse = torch.full((R, H), -math.inf, dtype=torch.float64, device=dev)
    tol_out = torch.zeros_like(out)
    tol_lse = torch.zeros_like(lse)
    ref_score = None if score is None else score.double().clone()
    tol_score = None if score is None else torch.zeros_like(ref_score)
    u = 2.0 ** -24
    half = torch.finfo(q.dtype).eps / 2
    pages_of, lens = table.tolist(), lens.tolist()
    for r in range(R):
        T = max(0, lens[r])
        T = T if max_len is None else min(T, max_len)
        if score is not None:
            ref_score[r, :T] = 0.0 if decay == 0 else ref_score[r, :T] * decay
            tol_score[r, :T] = 2 * u * ref_score[r, :T].abs()
        t = [x for x in visible(T, window, sinks) if 0 <= pages_of[r][x // page] < P]
        if not t:
            continue
        t = torch.tensor(t, device=dev)
        pg, at = table[r].to(dev).long()[t // page], t % page
        for g in range(G):
            K, V = k[pg, at, g].double(), v[pg, at, g].double()
            if k_scale is not None:
                K = K * float(k_scale[g])
            if v_scale is not None:
                V = V * float(v_scale[g])
            hh = slice(g * group, (g + 1) * group)
            Q = q[r, hh].double()
            x = Q @ K.T * scale
            m = x.amax(1, keepdim=True)
            e = torch.exp(x - m)
            L = e.sum(1, keepdim=True)
            w = e / L
            out[r, hh] = w @ V
            lse[r, hh] = (m + torch.log(L))[:, 0]
            dx = ((d + 4) * 2 * u * abs(scale) * (Q.abs() @ K.abs().T).amax(1, keepdim=True)
                  + 4 * u * x.abs().amax(1, keepdim=True))
            rel = 2 * (dx + 8 * u) + 2 * u * len(t)
            tol_out[r, hh] = ((rel + 2.0 ** -16) * (w @ V.abs()) * (1 + half)
                              + half * out[r, hh].abs() + (2.0 ** -25 if q.dtype == torch.float16
                                                           else 0.0))
            tol_lse[r, hh] = (rel[:, 0] + 2 * u * lse[r, hh].abs() + 4 * u)
            if score is not None:
                ws = w.sum(0)
                ref_score[r].index_add_(0, t, ws)
                tol_score[r].index_add_(0, t, (w * rel).sum(0) + 2 * u * group * ws)
        if score is not None:
            tol_score[r] += 2 * u * (G + 1) * ref_score[r].abs()
    return out, lse, ref_score, (tol_out, tol_lse, tol_score)


def check(got, ref, tol, what):
    got = got.double()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.where(fin, 0.0, got), torch.where(fin, 0.0, ref)), \
        f"{what}: non-finite values differ"
    over = ((got - ref).abs() - tol)[fin]
    if over.numel():
        worst = float(over.max())
        assert worst <= 0, f"{what}: {worst} over the bound ({float(tol.max())} at most)"
