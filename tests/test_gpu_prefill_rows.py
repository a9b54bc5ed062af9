"""hs.paged_prefill: which rows of out and lse a call writes."""
import math

import pytest
import torch

from test_gpu_prefill import BF, E4, call, check, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,cache,d", [(BF, BF, 128), (BF, E4, 128), (BF, BF, 256)])
@pytest.mark.parametrize("cu", [[0, 5, 3, 8], [0, 8, 2, 8], [4, 3, 3, 3], [0, 2, 9, 8], [0, 60, 4, 8]])
def test_requests_that_overlap_are_not_computed(cu, dtype, cache, d):
    """Two requests must not write one row: the result would be the later one's."""
    s = setup([5, 0, 3], [40, 90, 300], 8, 2, d, 16, dtype, cache)
    s["cu"].copy_(torch.tensor(cu))
    out, lse = call(s)
    assert s["status"].item() == 6
    assert (out == 7).all() and (lse == 7).all()


def test_descending_among_many_requests():
    s = setup([2] * 300, [10 + i for i in range(300)], 4, 2, 64, 16)
    want = call(s)[0].clone()
    assert s["status"].item() == 0
    for r in (1, 150, 299):
        cu = s["cu"].clone()
        s["cu"][r] = cu[r + 1] + 1
        assert (call(s)[0] == 7).all() and s["status"].item() == 6
        s["cu"].copy_(cu)
        s["status"].zero_()
    assert torch.equal(call(s)[0], want) and s["status"].item() == 0
    # Ends outside the tokens are clipped: what is left is computed.
    s["cu"][0], s["cu"][300] = -3, 10 ** 6
    assert torch.equal(call(s)[0], want) and s["status"].item() == 6


@pytest.mark.parametrize("dtype,cache,heads,kv_heads,d", [
    (BF, BF, 32, 8, 128), (BF, E4, 8, 2, 128), (BF, BF, 4, 1, 256), (BF, BF, 7, 1, 64)])
@pytest.mark.parametrize("window", [0, 100])
def test_a_refused_prompt_among_single_tokens(window, dtype, cache, heads, kv_heads, d):
    """Rows of a request without cached tokens, and queries before position 0, are 0 and
    -inf; they change nothing for the others."""
    new = [1] * 6 + [3000] + [1] * 6 + [700, 5]
    lens = [100 + 300 * i for i in range(6)] + [0] + [90 * i for i in range(1, 7)] + [150, 2]
    s = setup(new, lens, heads, kv_heads, d, 16, dtype, cache, pad=2)
    out, lse = check(s, window=window)
    blind = [range(6, 3006), range(3012, 3012 + 550), range(3712, 3715)]
    for rows in blind:
        assert (out[rows] == 0).all() and (lse[rows] == -math.inf).all()
    assert (out[3000 + 6 + 6 + 550] != 0).any()
