"""The status word of the paged-cache calls has to lie on the call's device (or
in pinned host memory): the kernels write to it."""
import pytest
import torch

from sparse_top_kv_gb300 import hs


class Word:
    """A tensor's facts, so that a second device needs no second GPU."""

    def __init__(self, device, dtype=torch.int32, n=1):
        self.index, self.dtype, self.n = device, dtype, n
        self.is_cuda, self.device = device >= 0, f"cuda:{device}" if device >= 0 else "cpu"

    def get_device(self):
        return self.index

    def numel(self):
        return self.n

    def is_contiguous(self):
        return True

    def is_pinned(self):
        return False

    def data_ptr(self):
        return 4096


def test_devices():
    assert hs._status_ptr(None, 0) is None
    assert hs._status_ptr(Word(1), 1) == 4096
    for word, device in ((Word(1), 0), (Word(0), 1), (Word(-1), 0), (Word(0, n=0), 0)):
        with pytest.raises(ValueError):
            hs._status_ptr(word, device)
    with pytest.raises(TypeError):
        hs._status_ptr(Word(0, torch.int64), 0)


@pytest.mark.gpu
def test_pinned_and_refused():
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 8, 64, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    table, lens = torch.full((1, 4), 9, **i32), torch.tensor([40], **i32)
    ws = torch.empty(hs.paged_decode_workspace_bytes(1, 8, 2, 64, 64), dtype=torch.uint8,
                     device="cuda")
    out, lse = torch.empty_like(q), torch.empty(1, 8, device="cuda")
    for status in (torch.zeros(1, **i32), torch.zeros(1, dtype=torch.int32).pin_memory()):
        hs.paged_decode(q, cache, cache.clone(), table, lens, 0.1, out=out, lse=lse, workspace=ws,
                        status=status)
        torch.cuda.synchronize()
        assert int(status) == 6  # every page lies outside the cache
    for status, error in ((torch.zeros(1, dtype=torch.int32), ValueError),
                          (torch.zeros(0, **i32), ValueError),
                          (torch.zeros(1, device="cuda"), TypeError)):
        with pytest.raises(error):
            hs.paged_decode(q, cache, cache.clone(), table, lens, 0.1, out=out, lse=lse,
                            workspace=ws, status=status)
