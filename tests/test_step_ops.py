"""Argument checks of hs_paged_extend, hs_rope_append and hs_paged_prefill (each
returns its status before any device work), and the rotary tables (no GPU)."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

from sparse_top_kv_gb300 import hs

BUF = ctypes.create_string_buffer(8192)
P = ctypes.c_void_p(ctypes.addressof(BUF) + (-ctypes.addressof(BUF) % 256))
ODD = ctypes.c_void_p(P.value + 8)
BYTE = ctypes.c_void_p(P.value + 2)

EXTEND = dict(new=P, lens=P, table=P, bt_stride=4, rows=2, max_blocks=4, ring=P, pages=8, ends=P,
              page_size=16, max_tokens=32, lens_out=P, attend=P, ends_out=P, cu=P, slot=P, row=P,
              pos=P, status=None, stream=None)
ROPE = dict(q=P, q_stride=1024, k=P, k_stride=256, v=P, v_stride=256, dtype=0, tokens=2, heads=8,
            kv_heads=2, d=128, pos=P, slot=P, turns=P, rot=128, interleaved=0, mscale=1.0, q_out=P,
            q_out_stride=1024, k_cache=P, v_cache=P, kv_dtype=0, page_stride=4096, row_stride=256,
            head_stride=128, pages=4, page_size=16, k_scale=None, v_scale=None, status=None,
            stream=None)
PREFILL = dict(q=P, q_stride=1024, q_dtype=0, tokens=4, k=P, v=P, kv_dtype=0, page_stride=4096,
               row_stride=256, head_stride=128, num_pages=4, page_size=16, table=P, bt_stride=4,
               max_blocks=4, max_len=64, cu=P, lens=P, k_scale=None, v_scale=None, rows=2, heads=8,
               kv_heads=2, d=128, window=0, sinks=0, scale=1.0, out=P, lse=None, ws=None,
               ws_bytes=0, status=None, stream=None)


@pytest.mark.parametrize("code,kw", [
    (1, dict(rows=-1)), (1, dict(max_blocks=-1)), (1, dict(pages=-1)), (1, dict(page_size=0)),
    (1, dict(max_tokens=-1)), (1, dict(bt_stride=3)), (1, dict(new=None)), (1, dict(lens=None)),
    (1, dict(table=None)), (1, dict(ring=None)), (1, dict(ends=None)), (1, dict(ends_out=None)),
    (1, dict(lens_out=None)), (1, dict(attend=None)), (1, dict(cu=None)), (1, dict(slot=None)),
    (1, dict(row=None)), (1, dict(pos=None)), (2, dict(new=BYTE)), (2, dict(slot=BYTE)),
    (2, dict(ends=ctypes.c_void_p(P.value + 4))), (3, dict(rows=4097)),
    (3, dict(pages=(1 << 30) + 1)), (3, dict(max_tokens=(1 << 30) + 1)),
    (3, dict(pages=1 << 28, page_size=16)), (3, dict(max_blocks=1 << 27, bt_stride=1 << 27))])
def test_extend_checks(code, kw):
    assert hs.lib().hs_paged_extend(*{**EXTEND, **kw}.values()) == code


@pytest.mark.parametrize("code,kw", [
    (1, dict(tokens=-1)), (1, dict(heads=-1)), (1, dict(kv_heads=-2)), (1, dict(d=0)),
    (1, dict(rot=-2)), (1, dict(rot=130)), (1, dict(dtype=2)), (1, dict(kv_dtype=3)),
    (1, dict(q_stride=-8)), (1, dict(pages=-1)), (1, dict(pos=None)), (1, dict(turns=None)),
    (1, dict(q_out=None)), (1, dict(v=None)), (1, dict(slot=None)), (1, dict(k_cache=None)),
    (1, dict(page_size=0)), (2, dict(q=ODD)), (2, dict(k=ODD)), (2, dict(q_out=ODD)),
    (2, dict(v_cache=ODD)), (2, dict(q_stride=1028)), (2, dict(row_stride=260)),
    (2, dict(kv_dtype=2, head_stride=136)), (2, dict(turns=ctypes.c_void_p(P.value + 4))),
    (2, dict(pos=BYTE)), (3, dict(heads=(1 << 20) + 8)), (7, dict(d=100, rot=0)),
    (7, dict(d=1032)), (7, dict(rot=63)), (7, dict(kv_dtype=1)), (7, dict(k_scale=P)),
    (0, dict(tokens=0)), (0, dict(q=None, k=None, v=None))])
def test_rope_checks(code, kw):
    assert hs.lib().hs_rope_append(*{**ROPE, **kw}.values()) == code


@pytest.mark.parametrize("code,kw", [
    (1, dict(rows=-1)), (1, dict(tokens=-1)), (1, dict(heads=9)), (1, dict(kv_heads=0)),
    (1, dict(d=0)), (1, dict(max_len=-1)), (1, dict(max_len=65)), (1, dict(window=-1)),
    (1, dict(sinks=-2)), (1, dict(page_size=0)), (1, dict(num_pages=-1)), (1, dict(q_dtype=2)),
    (1, dict(kv_dtype=3)), (1, dict(page_stride=-8)), (1, dict(q=None)), (1, dict(k=None)),
    (1, dict(v=None)), (1, dict(cu=None)), (1, dict(lens=None)), (1, dict(out=None)),
    (1, dict(table=None)), (2, dict(q=ODD)), (2, dict(k=ODD)), (2, dict(out=ODD)),
    (2, dict(cu=BYTE)), (2, dict(q_stride=1028)), (2, dict(row_stride=260)), (2, dict(ws=ODD)),
    (2, dict(kv_dtype=2, row_stride=264)), (3, dict(rows=4097)), (3, dict(tokens=(1 << 24) + 1)),
    (3, dict(max_blocks=1 << 27, max_len=(1 << 30) + 1)), (7, dict(d=96)), (7, dict(kv_dtype=1)),
    (7, dict(heads=258)), (7, dict(k_scale=P)), (0, dict(rows=0)), (0, dict(tokens=0))])
def test_prefill_checks(code, kw):
    assert hs.lib().hs_paged_prefill(*{**PREFILL, **kw}.values()) == code


def test_prefill_workspace_query():
    f = hs.paged_prefill_workspace_bytes
    assert f(4, 2, 8, 2, 128, 1000) >= 0 and f(0, 0, 8, 2, 128, 0) >= 0
    assert f(-1, 2, 8, 2, 128, 10) == -1 and f(4, 2, 9, 2, 128, 10) == -1
    assert f(4, 4097, 8, 2, 128, 10) == -1


def test_rope_tables():
    inv, m = hs.rope_frequencies(8, 10000.0)
    assert m == 1.0 and torch.allclose(inv, torch.tensor([1, 0.1, 0.01, 0.001], dtype=torch.float64))
    for f, t in zip(inv.tolist(), hs.rope_turns(inv, "cpu").tolist()):
        # float64 of f / 2 pi, times 2^64: relative 2^-52.
        assert abs(t - f / (2 * math.pi) * 2.0 ** 64) <= t * 2.0 ** -52 + 1
    # More than half a turn per position is a negative int64; whole turns drop out.
    t = hs.rope_turns(torch.tensor([2 * math.pi * 0.75, 2 * math.pi * 2.25]), "cpu").tolist()
    assert abs(Fraction(t[0], 2 ** 64) + Fraction(1, 4)) < 1e-6
    assert abs(Fraction(t[1], 2 ** 64) - Fraction(1, 4)) < 1e-6
    lin, _ = hs.rope_frequencies(64, scaling="linear", factor=4.0)
    ntk, _ = hs.rope_frequencies(64, scaling="ntk", factor=4.0)
    yarn, ms = hs.rope_frequencies(64, scaling="yarn", factor=4.0, original_len=2048)
    base, _ = hs.rope_frequencies(64)
    assert torch.allclose(lin * 4, base)
    assert ntk[0] == 1 and torch.isclose(ntk[-1] * 4, base[-1])
    assert yarn[0] == base[0] and torch.isclose(yarn[-1] * 4, base[-1])
    assert abs(ms - (0.1 * math.log(4) + 1)) < 1e-12
    assert hs.rope_frequencies(0)[0].numel() == 0
    for kw in (dict(rot=3), dict(rot=4, factor=0.0), dict(rot=4, scaling="other"),
               dict(rot=4, scaling="yarn"), dict(rot=-2)):
        with pytest.raises(ValueError):
            hs.rope_frequencies(**kw)
