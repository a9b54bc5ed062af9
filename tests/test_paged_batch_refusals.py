"""PagedBatch: rows and lengths that do not fit are refused before a step has changed
anything."""
from types import SimpleNamespace

import pytest
import torch

from sparse_top_kv_gb300 import hs
from sparse_top_kv_gb300.pipeline import PagedBatch

SHAPE = dict(num_reqs=3, heads=8, kv_heads=2, d=64, page_size=16, max_len=100, max_tokens=24,
             scale=0.125, layers=2)
BF = torch.bfloat16


def rows(heads, device):
    return torch.zeros(24, heads, 64, dtype=BF, device=device)


def bad_rows(heads, device):
    wide = torch.zeros(24 * 2 * heads * 64 + 64, dtype=BF, device=device)
    yield rows(heads, "meta")                                          # another device
    yield wide[:24 * 64 * heads].view(24, 64, heads).transpose(1, 2)   # elements apart
    yield wide[:24 * 64 * heads].view(heads, 24, 64).transpose(0, 1)   # heads apart
    yield wide[1:1 + 24 * 64 * heads].view(24, heads, 64)              # starts inside 16 bytes
    yield wide.as_strided((24, heads, 64), (64 * heads + 4, 64, 1))    # so do its tokens


def check_step(device, monkeypatch):
    b = PagedBatch(**SHAPE, device=device)
    grown = []
    real = hs.paged_extend
    monkeypatch.setattr(hs, "paged_extend", lambda *a, **kw: grown.append(1) or real(*a, **kw))
    new = torch.ones(3, dtype=torch.int32, device=device)
    for which in range(3):
        for bad in bad_rows((8, 2, 2)[which], device):
            layers = [[rows(h, device) for _ in range(2)] for h in (8, 2, 2)]
            layers[which][1] = bad  # the last layer's
            with pytest.raises(ValueError):
                b.step(new, *layers)
    assert not grown and b.seq_lens.tolist() == [0, 0, 0] and b.ring_pos.tolist() == [0, 21]


def test_step(monkeypatch):
    check_step("cpu", monkeypatch)


@pytest.mark.gpu
def test_step_on_the_gpu(monkeypatch):
    check_step("cuda", monkeypatch)


def test_replay():
    b = PagedBatch(**SHAPE, device="cpu")
    ran = []
    b.graph = SimpleNamespace(replay=lambda: ran.append(1))
    b.graph_new = torch.full((3,), 7, dtype=torch.int32)
    b.graph_q, b.graph_k, b.graph_v = (torch.zeros(2, 24, h, 64, dtype=BF) for h in (8, 2, 2))
    good = [[rows(h, "cpu") for _ in range(2)] for h in (8, 2, 2)]
    for new, error in ((torch.ones(1, dtype=torch.int32), ValueError),
                       (torch.ones(3, 1, dtype=torch.int32), ValueError),
                       (torch.ones((), dtype=torch.int32), ValueError),
                       (torch.ones(4, dtype=torch.int32), ValueError),
                       (torch.ones(3), TypeError), (torch.ones(3, dtype=torch.bool), TypeError)):
        with pytest.raises(error):
            b.replay(new, *good)
    assert not ran and b.graph_new.tolist() == [7, 7, 7]
    # Rows are copied: any layout will do.
    b.replay(torch.ones(3, dtype=torch.int32), *[[list(bad_rows(h, "cpu"))[2]] * 2 for h in (8, 2, 2)])
    assert ran and b.graph_new.tolist() == [1, 1, 1]
