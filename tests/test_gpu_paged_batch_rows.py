"""PagedBatch: which rows of a step's outputs are written."""
import math

import pytest
import torch

import paged_ref
import step_ref
from sparse_top_kv_gb300 import hs
from sparse_top_kv_gb300.pipeline import PagedBatch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float8_e4m3fn])
def test_rows_of_a_refused_request(cache):
    """Zeros and -inf between the rows of its neighbours, which are as ever."""
    g = torch.Generator().manual_seed(2)
    b = PagedBatch(num_reqs=4, heads=8, kv_heads=2, d=128, page_size=16, max_len=512, num_pages=9,
                   max_tokens=400, scale=0.1, cache_dtype=cache)
    for new, refused in (([30, 5, 0, 40], None), ([1, 300, 0, 3], 1), ([1, 0, 400, 2], 2)):
        x = torch.randn(1, 400, 12, 128, generator=g).to(torch.bfloat16).cuda()
        b.out.fill_(7.0)
        b.lse.fill_(7.0)
        n = torch.tensor(new, dtype=torch.int32, device="cuda")
        out, lse = b.step(n, x[:, :, :8], x[:, :, 8:10], x[:, :, 10:])
        ref, ref_lse, (tol, tol_lse), written = step_ref.prefill(
            b.q_rot, b.k_cache[0], b.v_cache[0], b.block_table, b.cu_new, b.attend_lens, b.scale)
        paged_ref.check(out[0][written].double(), ref[written], tol[written], "out")
        paged_ref.check(lse[0][written].double(), ref_lse[written], tol_lse[written], "lse")
        assert (out[0][~written] == 7).all() and (lse[0][~written] == 7).all()
        if refused is None:
            b.check()
            continue
        with pytest.raises(hs.HSError):
            b.check()
        first, last = b.cu_new[refused].item(), b.cu_new[refused + 1].item()
        assert last > first and b.attend_lens[refused].item() == 0
        assert (out[0, first:last] == 0).all() and (lse[0, first:last] == -math.inf).all()
