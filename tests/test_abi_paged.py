"""Argument checks of the paged-cache entry points: each returns its status
before any device work (no GPU)."""
import ctypes

import pytest

from sparse_top_kv_gb300 import hs

BUF = ctypes.create_string_buffer(8192)
P = ctypes.c_void_p(ctypes.addressof(BUF) + (-ctypes.addressof(BUF) % 256))
ODD = ctypes.c_void_p(P.value + 8)

DECODE = dict(q=P, q_stride=1024, q_dtype=0, k=P, v=P, kv_dtype=0, page_stride=4096,
              row_stride=256, head_stride=128, num_pages=4, page_size=16, table=P, bt_stride=4,
              max_blocks=4, max_len=64, lens=P, k_scale=None, v_scale=None, rows=2, heads=8,
              kv_heads=2, d=128, window=0, sinks=0, scale=1.0, score=None, score_stride=0,
              decay=1.0, out=P, lse=None, ws=None, ws_bytes=0, status=None, stream=None)


def decode(**kw):
    return hs.lib().hs_paged_decode(*{**DECODE, **kw}.values())


@pytest.mark.parametrize("code,kw", [
    (1, dict(rows=-1)), (1, dict(heads=0)), (1, dict(heads=9)), (1, dict(kv_heads=0)),
    (1, dict(d=0)), (1, dict(max_len=-1)), (1, dict(max_len=65)), (1, dict(window=-1)),
    (1, dict(sinks=-2)), (1, dict(page_size=0)), (1, dict(num_pages=-1)), (1, dict(q_dtype=2)),
    (1, dict(kv_dtype=3)), (1, dict(page_stride=-8)), (1, dict(bt_stride=-1)),
    (1, dict(score=P, score_stride=63)), (1, dict(q=None)), (1, dict(k=None)), (1, dict(v=None)),
    (1, dict(lens=None)), (1, dict(out=None)), (1, dict(table=None)),
    (2, dict(q=ODD)), (2, dict(k=ODD)), (2, dict(v=ODD)), (2, dict(out=ODD)),
    (2, dict(q_stride=1028)), (2, dict(row_stride=260)), (2, dict(head_stride=4)),
    (2, dict(page_stride=4100)), (2, dict(kv_dtype=2, row_stride=264)), (2, dict(ws=ODD)),
    (3, dict()), (3, dict(rows=4097)),
    (3, dict(rows=4096, heads=128, max_blocks=1 << 20, max_len=1 << 24)), (3, dict(ws=P, ws_bytes=100)),
    (7, dict(d=96)), (7, dict(kv_dtype=1)), (7, dict(q_dtype=1)), (7, dict(k_scale=P)),
    (7, dict(v_scale=P)), (0, dict(rows=0))])
def test_paged_decode_checks(code, kw):
    assert decode(**kw) == code


def test_paged_decode_workspace_query():
    f = hs.paged_decode_workspace_bytes
    assert f(2, 8, 2, 128, 1000) > 0
    assert f(2, 8, 2, 128, 1000, with_score=True) >= f(2, 8, 2, 128, 1000) + 2 * 8 * 1000 * 4
    # A window bounds the logits that a scored call keeps.
    assert f(2, 8, 2, 128, 100000, window=64, num_sinks=4, with_score=True) < f(
        2, 8, 2, 128, 100000, with_score=True)
    assert f(-1, 8, 2, 128, 10) == -1 and f(1, 9, 2, 128, 10) == -1 and f(
        4097, 8, 2, 128, 10) == -1 and f(0, 8, 2, 128, 10) == 0


SELECT = dict(score=P, score_stride=64, positions=None, pos_stride=0, lens=P, next_pos=None,
              rows=2, max_len=64, budget=32, recent=4, sinks=2, score_out=P, score_out_stride=64,
              positions_out=None, pos_out_stride=0, lens_out=P, src=P, dst=P, count=P, cap=32,
              status=None, stream=None)
MOVE = dict(k=P, v=None, page_stride=4096, row_stride=256, head_stride=128, kv_heads=2,
            row_bytes=128, num_pages=4, page_size=16, table=P, bt_stride=4, max_blocks=4, src=P,
            dst=P, count=P, rows=2, cap=32, status=None, stream=None)
SELECT_BAD = [
    (1, dict(rows=-1)), (1, dict(max_len=-1)), (1, dict(budget=0)), (1, dict(recent=-1)),
    (1, dict(sinks=-1)), (1, dict(recent=31)), (1, dict(cap=-1)), (3, dict(cap=31)),
    (3, dict(max_len=(1 << 30) + 1)),
    (1, dict(score=None)), (1, dict(lens=None)), (1, dict(score_out=None)),
    (1, dict(lens_out=None)), (1, dict(src=None)), (1, dict(dst=None)), (1, dict(count=None)),
    (1, dict(score_stride=63)), (1, dict(score_out_stride=63)),
    (1, dict(positions=P, pos_stride=10)), (1, dict(positions_out=P, pos_out_stride=10)),
    (1, dict(score_out_stride=80))]
ODD2 = ctypes.c_void_p(P.value + 2)


@pytest.mark.parametrize("code,kw", SELECT_BAD + [(2, dict(score=ODD2, score_out=ODD2)),
                                                  (2, dict(lens=ODD2)), (0, dict(rows=0))])
def test_evict_select_checks(code, kw):
    assert hs.lib().hs_evict_select(*{**SELECT, **kw}.values()) == code


MOVE_BAD = [
    (1, dict(rows=-1)), (1, dict(kv_heads=0)), (1, dict(row_bytes=0)), (1, dict(page_size=0)),
    (1, dict(num_pages=-1)), (1, dict(max_blocks=-1)), (1, dict(page_stride=-16)),
    (1, dict(k=None)), (1, dict(table=None)), (1, dict(v=P)), (2, dict(row_bytes=100)),
    (2, dict(head_stride=100)), (2, dict(row_stride=264)), (2, dict(k=ODD)), (2, dict(v=ODD)),
    (1, dict(kv_heads=1 << 20, row_bytes=4096))]


@pytest.mark.parametrize("code,kw", MOVE_BAD + [(1, dict(src=None)), (1, dict(count=None)),
                                                (0, dict(rows=0)), (0, dict(cap=0))])
def test_evict_move_checks(code, kw):
    assert hs.lib().hs_evict_move(*{**MOVE, **kw}.values()) == code


@pytest.mark.parametrize("code,kw", SELECT_BAD + MOVE_BAD + [(1, dict(max_blocks=3)),
                                                             (0, dict(rows=0))])
def test_evict_checks(code, kw):
    a = {k: v for k, v in SELECT.items() if k not in ("status", "stream")}
    b = {k: v for k, v in MOVE.items() if k not in ("src", "dst", "count", "rows", "cap")}
    assert hs.lib().hs_evict(*{**a, **b, **kw}.values()) == code


def test_paged_decode_head_limit():
    kw = dict(heads=65537, kv_heads=1, ws=P, ws_bytes=1 << 60)
    assert decode(**kw) == 3
    assert hs.paged_decode_workspace_bytes(2, 65537, 1, 128, 64) == -1
    assert hs.paged_decode_workspace_bytes(2, 65536, 1, 128, 64) > 0


@pytest.mark.parametrize("kw", [dict(window=1 << 32), dict(num_sinks=1 << 31),
                                dict(max_len=(1 << 32) + 5), dict(rows=-(1 << 31) - 1)])
def test_sizes_past_32_bits_are_refused(kw):
    """ctypes would wrap them around."""
    with pytest.raises(ValueError):
        hs.paged_decode_workspace_bytes(**{**dict(rows=2, heads=8, kv_heads=2, d=128,
                                                  max_len=64), **kw})
