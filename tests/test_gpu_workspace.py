"""Workspaces that are not one run of memory are refused before any launch: the
kernels take their bytes from the tensor's start, and an expanded tensor has
next to none there."""
import pytest
import torch

from sparse_top_kv_gb300 import hs

LAYOUTS = {"expanded": lambda n, dev: torch.empty(1, dtype=torch.uint8, device=dev).expand(n),
           "strided": lambda n, dev: torch.empty(2 * n, dtype=torch.uint8, device=dev)[::2],
           "transposed": lambda n, dev: torch.empty(n // 64, 64, device=dev).t()}


@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_check(layout):
    with pytest.raises(ValueError):
        hs._check_workspace(LAYOUTS[layout](4096, "cpu"))
    hs._check_workspace(torch.empty(4096))
    hs._check_workspace(torch.empty(64, 64)[1:])
    hs._check_workspace(None)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_calls(layout):
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    n = 32 << 20  # more than any of these calls asks for
    ws = LAYOUTS[layout](n, "cuda")
    q, cache = torch.zeros(2, 8, 128, **bf16), torch.zeros(8, 16, 2, 128, **bf16)
    table, lens = torch.arange(8, **i32).view(2, 4), torch.tensor([64, 9], **i32)
    for out, lse in ((None, None), (torch.empty_like(q), torch.empty(2, 8, device="cuda"))):
        with pytest.raises(ValueError, match="workspace"):
            hs.paged_decode(q, cache, cache, table, lens, 0.1, out=out, lse=lse, workspace=ws)
    rows, cap = 2, 64
    ids, count = torch.zeros(rows, 2, cap, **i32), torch.full((rows, 2), cap, **i32)
    kv = torch.zeros(128, 2, 128, **bf16)
    with pytest.raises(ValueError, match="workspace"):
        hs.sparse_decode(q, kv, kv, 256, 128, 128, ids, count, 0.1, 128, workspace=ws)
