"""hs_paged_decode where one token takes nearly all of the softmax's weight and
has no value (an attention sink with V = 0): the output is then the sum of the
other tokens' small weights, which the kernels have to carry as exactly as
large ones.  Against the 64-bit definition, every cache type, on both kernels
and every way of cutting a call."""
import math

import pytest
import torch

from sparse_top_kv_gb300 import hs

pytestmark = pytest.mark.gpu

KINDS = {"bf16": (torch.bfloat16, torch.bfloat16), "fp16": (torch.float16, torch.float16),
         "e4m3": (torch.bfloat16, torch.float8_e4m3fn),
         "e4m3_fp16": (torch.float16, torch.float8_e4m3fn)}
# lens, heads, kv_heads, d, page: the tcgen05 kernel with its tiles dealt to the
# CTAs and with a cluster to a unit, up to 8 and up to 16 query heads to a KV
# head; the warp-level kernel likewise (odd pages, few heads).
CUTS = {"dealt": ([8192, 3000, 1, 0, 5000], 16, 2, 128, 64),
        "dealt_many_heads": ([4100, 700] + [900] * 20, 64, 8, 128, 16),
        "cluster": ([300, 77], 16, 2, 128, 16),
        "cluster_wide": ([900], 32, 2, 256, 16),
        "dealt_wide": ([6000, 100, 3000], 32, 2, 256, 16),
        "small": ([5000, 33], 8, 2, 128, 64),
        "warps": ([4000, 77], 8, 2, 64, 12),
        "warps_wide": ([4000, 260], 24, 2, 128, 5)}


def inputs(kind, cut, gap, sink_at, seed):
    lens, heads, kvh, d, page = CUTS[cut]
    qt, kt = KINDS[kind]
    g = torch.Generator(device="cuda").manual_seed(seed)
    R, blocks = len(lens), -(-max(lens) // page)
    table = torch.randperm(R * blocks, generator=g, device="cuda").to(torch.int32).view(R, blocks)
    scale = 1 / math.sqrt(d)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    # Dim 0 of the queries is 8 and of the keys 0 but for the sink's, which
    # lies `gap` above 0; the other dims spread the logits by about a half.
    q = rnd(R, heads, d) * 0.5
    k, v = rnd(R * blocks, page, kvh, d), rnd(R * blocks, page, kvh, d)
    q[..., 0], k[..., 0] = 8.0, 0.0
    for r, n in enumerate(lens):
        if n:
            t = min(n - 1, sink_at(n))
            p = int(table[r, t // page])
            k[p, t % page] = 0.0
            k[p, t % page, :, 0] = gap / (8 * scale)
            v[p, t % page] = 0.0
    scales = (None, None)
    if kt is torch.float8_e4m3fn:
        scales = (torch.full((kvh,), 1.25, device="cuda"), torch.full((kvh,), 0.75, device="cuda"))
        k, v = (k / 1.25).to(torch.bfloat16), v.to(torch.bfloat16)
    return dict(q=q.to(qt), k=k.to(kt), v=v.to(kt), table=table, scales=scales, scale=scale,
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def definition(s):
    """(out, bound) in 64 bits.  With u = 2^-24: a logit is off by dx <= (d + 4)
    2u scale max sum |q_i k_i| + 4u max |x|; a weight w by the factor 1 +- (2 (dx +
    8u) + 2u T).  It is carried to 2^-16 of itself (E4M3 parts 2^-19, two bf16 or
    fp16 parts less) or, where that is more, to the smaller of 2^-10 w and 2^-35
    of the largest weight, and to 2^-40 of that where even less is left.  The
    output rounds once."""
    q, k, v = s["q"].double(), s["k"].float().double(), s["v"].float().double()
    R, H, d = q.shape
    page, G = k.shape[1], k.shape[2]
    out, tol = torch.zeros_like(q), torch.zeros_like(q)
    u, half = 2.0 ** -24, torch.finfo(s["q"].dtype).eps / 2
    for r, n in enumerate(s["lens"].tolist()):
        t = torch.arange(n, device="cuda")
        if not n:
            continue
        at = s["table"][r].long()[t // page], t % page
        for g in range(G):
            K, V = k[at][:, g], v[at][:, g]
            if s["scales"][0] is not None:
                K, V = K * s["scales"][0][g].double(), V * s["scales"][1][g].double()
            hh = slice(g * (H // G), (g + 1) * (H // G))
            x = q[r, hh] @ K.T * s["scale"]
            w = torch.softmax(x, 1)
            dx = ((d + 4) * 2 * u * s["scale"] * (q[r, hh].abs() @ K.abs().T).amax(1, keepdim=True)
                  + 4 * u * x.abs().amax(1, keepdim=True))
            top = w.amax(1, keepdim=True)
            dw = (w * (2 * (dx + 8 * u) + 2 * u * n + 2.0 ** -16)
                  + torch.minimum(w * 2.0 ** -10, top * 2.0 ** -35) + top * 2.0 ** -40)
            out[r, hh] = w @ V
            # fp16 values below 2^-14 round to a step of 2^-24.
            tol[r, hh] = (dw @ V.abs() * (1 + half) + half * out[r, hh].abs()
                          + (2.0 ** -25 if s["q"].dtype == torch.float16 else 0.0))
    return out, tol


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("cut", list(CUTS))
@pytest.mark.parametrize("gap", [12, 15, 18, 21])
def test_sink_without_a_value(kind, cut, gap):
    s = inputs(kind, cut, float(gap), lambda n: 0, gap)
    check(s)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("cut", ["dealt", "cluster", "warps"])
def test_sink_behind_other_tokens(kind, cut):
    """The running maximum grows when it comes."""
    check(inputs(kind, cut, 17.0, lambda n: n // 3, 5))


def check(s):
    out, lse = hs.paged_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"],
                               k_scale=s["scales"][0], v_scale=s["scales"][1])
    torch.cuda.synchronize()
    want, tol = definition(s)
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all()
    assert bool((err <= tol).all()), (f"{float((err - tol).max())} over the bound; relative L2 "
                                      f"{float((out.double() - want).norm() / want.norm())}")
