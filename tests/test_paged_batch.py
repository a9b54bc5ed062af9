"""PagedBatch: set-ups that do not fit are refused before anything is allocated."""
import pytest
import torch

from sparse_top_kv_gb300.pipeline import PagedBatch

SHAPE = dict(num_reqs=3, heads=8, kv_heads=2, d=64, page_size=16, max_len=100, max_tokens=24,
             scale=0.125, device="cpu")


@pytest.mark.parametrize("bad", [
    dict(num_reqs=0), dict(num_reqs=4097), dict(heads=7), dict(heads=0), dict(kv_heads=0),
    dict(d=96), dict(page_size=0), dict(max_len=0), dict(max_tokens=0), dict(layers=0),
    dict(num_pages=0), dict(num_pages=1 << 27), dict(window=-1), dict(num_sinks=-1),
    dict(heads=258, kv_heads=2), dict(k_scale=torch.ones(1, 2)),
    dict(cache_dtype=torch.float8_e4m3fn, v_scale=torch.ones(2)),
    dict(inv_freq=torch.ones(33)), dict(max_len=(1 << 30) + 1, num_pages=9),
    dict(max_tokens=(1 << 24) + 1), dict(max_tokens=1 << 24, heads=128), dict(inv_freq=torch.ones(2, 2))])
def test_bad_values(bad):
    with pytest.raises(ValueError):
        PagedBatch(**{**SHAPE, **bad})


@pytest.mark.parametrize("bad", [dict(dtype=torch.float32), dict(cache_dtype=torch.float16),
                                 dict(dtype=torch.float16, cache_dtype=torch.float8_e5m2)])
def test_bad_types(bad):
    with pytest.raises(TypeError):
        PagedBatch(**{**SHAPE, **bad})


def test_calls():
    b = PagedBatch(**SHAPE)
    q, k, v = torch.zeros(24, 8, 64), torch.zeros(24, 2, 64), torch.zeros(24, 2, 64)
    q, k, v = (t.to(torch.bfloat16) for t in (q, k, v))
    with pytest.raises(ValueError):
        b.attend(1, q, k, v)
    with pytest.raises(ValueError):
        b.attend(0, q[:5], k, v)
    with pytest.raises(TypeError):
        b.attend(0, q, k.half(), v)
    with pytest.raises(ValueError):
        b.step(b.seq_lens, [q], [k, k], [v])
    with pytest.raises(ValueError):
        b.replay(b.seq_lens, [q], [k], [v])
    with pytest.raises(ValueError):
        b.stop(3)
    b.check()
    assert b.max_len == 112  # whole pages
