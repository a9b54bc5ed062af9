"""Plain definitions of the operators of a step of several new tokens per
request (hs.paged_extend, rope_append, paged_prefill), with the error bounds
that follow from the kernels' number formats.  Shares no code with the package."""
import math

import torch


def extend(new, lens, table, ring, ends, page, max_tokens):
    """(table, ring, ends, lens, attend, cu, slot, row, pos, status), lists; a token
    whose page lies outside [0, len(ring)) has no slot."""
    table, ring = [list(r) for r in table], list(ring)
    (taken, back), pages = ends, len(ring)
    rows, room = len(new), (len(table[0]) if table else 0) * page
    free, asked, given = back - taken, 0, []
    out, attend, cu = [], [], [0]
    slot, req, pos = ([-1] * max_tokens for _ in range(3))
    refused = bad = False
    for r in range(rows):
        held, n, first = max(0, lens[r]), new[r], cu[-1]
        cu.append(first + max(0, n))
        have, left = -(-held // page), held
        attend.append(0)
        if n < 0:
            left = max(0, held + n)
            given += table[r][-(-left // page):have]
        elif n > 0:
            fits = held + n <= room and first + n <= max_tokens
            need = -(-(held + n) // page) - have if fits else 0
            asked += need
            if not fits or need and asked > free:
                refused = True
            else:
                for b in range(have, have + need):
                    table[r][b] = ring[taken % pages]
                    taken += 1
                left = attend[-1] = held + n
                for i in range(n):
                    p = held + i
                    at = table[r][p // page]
                    if 0 <= at < pages:
                        slot[first + i] = at * page + p % page
                    else:
                        bad = True
                    req[first + i], pos[first + i] = r, p
        out.append(left)
    for p in given:
        ring[back % pages] = p
        back += 1
    cu = [min(c, max_tokens) for c in cu]
    return table, ring, [taken, back], out, attend, cu, slot, req, pos, 3 if refused else 6 if bad else 0


def rope(x, positions, inv_freq, interleaved, mscale):
    """x [tokens, heads, d] rotated, in float64."""
    x, half = x.double(), len(inv_freq)
    angle = positions.double()[:, None, None] * inv_freq.double()
    cos, sin = angle.cos() * mscale, angle.sin() * mscale
    a = x[..., 0:2 * half:2] if interleaved else x[..., :half]
    b = x[..., 1:2 * half:2] if interleaved else x[..., half:2 * half]
    y = x.clone()
    ya, yb = a * cos - b * sin, a * sin + b * cos
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = ya, yb
    else:
        y[..., :half], y[..., half:2 * half] = ya, yb
    return y


def rope_bound(x, y, inv_freq, interleaved, mscale, dtype, scale=None):
    """Error bound of the rotated x stored as dtype (divided by `scale`): angles
    within 2 pi 2^-26 of a turn and, of inv_freq's own rounding, 2^-52 of
    themselves (positions below 2^21: 2^-31); sinpi, cospi and the products
    within 8 u of a pair's size; then half a step of the type (its smallest step
    where that is more)."""
    u = 2.0 ** -24
    half = len(inv_freq)
    a = x.double().abs()
    pair = torch.zeros_like(a)
    if interleaved:
        s = a[..., 0:2 * half:2] + a[..., 1:2 * half:2]
        pair[..., 0:2 * half:2], pair[..., 1:2 * half:2] = s, s
    else:
        s = a[..., :half] + a[..., half:2 * half]
        pair[..., :half], pair[..., half:2 * half] = s, s
    err = pair * abs(mscale) * (2 * math.pi * 2.0 ** -26 + 2.0 ** -31 + 8 * u)
    y = y.abs()
    if scale is not None:
        y, err = y / scale, err / scale + 2 * u * y / scale
    f = torch.finfo(dtype)
    return err * (1 + f.eps) + f.eps / 2 * y + f.smallest_normal * f.eps / 2


def visible(p, window, sinks):
    """Positions that a query at position p attends to."""
    return [t for t in range(p + 1) if not window or t > p - window or t < sinks]


def prefill(q, k, v, table, cu, lens, scale, *, window=0, sinks=0, max_len=None, k_scale=None,
            v_scale=None):
    """(out, lse, tolerances, rows that are written) in float64 on q's device.

    Tolerances, with u = 2^-24 and tensor-core sums that may truncate (2 u an
    addition): a logit is off by dx <= (d + 4) 2u scale max_t sum|q_i k_i| + 4 u
    max|x|; E4M3 caches: bf16 queries become fp16 of their row's largest
    magnitude 2^14, which adds 2^-38 scale max|q| sum|k_i|.  A weight is off by a
    factor 1 +- 2 (dx + 8 u); rounded for the product by half a step: 2^-8 of
    itself (bf16 caches) or 2^-11 (fp16 and E4M3), there within 2^-35 of the
    query's largest weight where that is more.  The sums over T tokens add 2 u T.
    The output then rounds once: eps / 2 of its type."""
    N, H, d = q.shape
    P, page, G, _ = k.shape
    group, dev = H // G, q.device
    out = torch.zeros(N, H, d, dtype=torch.float64, device=dev)
    lse = torch.full((N, H), -math.inf, dtype=torch.float64, device=dev)
    tol_out, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    written = torch.zeros(N, dtype=torch.bool, device=dev)
    u = 2.0 ** -24
    half = torch.finfo(q.dtype).eps / 2
    wide = k.dtype == torch.bfloat16  # 8 bits of a weight, any exponent
    pages_of, cu, lens = table.tolist(), cu.tolist(), lens.tolist()
    for r in range(len(lens)):
        n = cu[r + 1] - cu[r]
        T = max(0, lens[r])
        T = T if max_len is None else min(T, max_len)
        written[cu[r]:cu[r + 1]] = True
        t = [x for x in range(T) if 0 <= pages_of[r][x // page] < P]
        if not t or n == 0:
            continue
        t = torch.tensor(t, device=dev)
        pg, at = table[r].to(dev).long()[t // page], t % page
        p = torch.arange(T - n, T, device=dev)[:, None]
        see = t <= p
        if window:
            see &= (t > p - window) | (t < sinks)
        for g in range(G):
            K, V = k[pg, at, g].double(), v[pg, at, g].double()
            if k_scale is not None:
                K = K * float(k_scale[g])
            if v_scale is not None:
                V = V * float(v_scale[g])
            hh = slice(g * group, (g + 1) * group)
            Q = q[cu[r]:cu[r + 1], hh].double()
            x = torch.einsum("ihd,td->iht", Q, K) * scale
            x = torch.where(see[:, None], x, -math.inf)
            m = x.amax(2, keepdim=True)
            e = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
            L = e.sum(2, keepdim=True)
            w = e / torch.where(L > 0, L, 1.0)

            def weigh(w, V):
                # What is not attended to has no effect, whatever it holds.
                y = torch.einsum("iht,td->ihd", w, torch.where(torch.isfinite(V), V, 0.0))
                for j in (~torch.isfinite(V)).any(1).nonzero()[:, 0].tolist():
                    y += torch.where(see[:, j, None, None], w[:, :, j, None] * torch.where(
                        torch.isfinite(V[j]), 0.0, V[j]), 0.0)
                return y

            o = weigh(w, V)
            out[cu[r]:cu[r + 1], hh] = o
            lse[cu[r]:cu[r + 1], hh] = (m + torch.log(L))[..., 0]
            size = torch.einsum("ihd,td->iht", Q.abs(), torch.where(torch.isfinite(K), K, 0.0).abs())
            size = torch.where(see[:, None] & torch.isfinite(x), size, 0.0).amax(2, keepdim=True)
            ax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(2, keepdim=True)
            dx = (d + 4) * 2 * u * abs(scale) * size + 4 * u * ax
            if k.dtype == torch.float8_e4m3fn:
                ks = torch.where(torch.isfinite(K), K, 0.0).abs().sum(1).amax()
                dx = dx + 2.0 ** -38 * abs(scale) * Q.abs().amax(2, keepdim=True) * ks
            rel = 2 * (dx + 8 * u) + 2 * u * len(t)
            aV = torch.where(torch.isfinite(V), V.abs(), 0.0)
            small = 0.0 if wide else 2.0 ** -35 * w.amax(2, keepdim=True) * torch.einsum(
                "it,td->id", see.double(), aV)[:, None]
            tol_out[cu[r]:cu[r + 1], hh] = (
                ((rel + (2.0 ** -8 if wide else 2.0 ** -11)) * torch.einsum("iht,td->ihd", w, aV)
                 + small) * (1 + half) + half * torch.nan_to_num(o, 0.0, 0.0, 0.0).abs()
                + (2.0 ** -25 if q.dtype == torch.float16 else 0.0))
            tol_lse[cu[r]:cu[r + 1], hh] = (rel[..., 0] + 2 * u * torch.nan_to_num(
                lse[cu[r]:cu[r + 1], hh], 0.0, 0.0, 0.0).abs() + 4 * u)
    return out, lse, (tol_out, tol_lse), written
