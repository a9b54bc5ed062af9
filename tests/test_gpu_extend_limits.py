"""hs.paged_extend where requests ask for more than any call holds."""
import pytest

from test_gpu_extend_rope import compare

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("huge", [
    [MOST], [MOST] * 2, [MOST] * 4, [2 ** 30] * 2, [2 ** 30] * 4, [2 ** 29] * 4, [2 ** 29] * 8,
    [2 ** 26] * 40, [2 ** 20] * 2048, [MOST] * 1023, [MOST] * 3000])
@pytest.mark.parametrize("max_tokens", [8, 5000])
def test_small_requests_behind_huge_ones(huge, max_tokens):
    """A request is served if its tokens lie below max_tokens, those of refused ones
    ahead of it counted."""
    small = [3, 1, -2, 5]
    lens, n = [2, 1, 4, 0], len(huge)
    held = [0, 1, 2, 3]  # pages of two tokens
    table = [[held[0], -1, -1], [held[1], -1, -1], held[2:] + [-1], [-1] * 3]
    ring, ends = [4, 5, 6, 7, -1, -1, -1, -1], [8, 12]
    compare(huge + small, [0] * n + lens, [[-1] * 3 for _ in range(n)] + table, ring, ends, 2,
            max_tokens)
    compare(small + huge + small, lens + [0] * n + lens, [r[:] for r in table] + [
        [-1] * 3 for _ in range(n)] + [[r if r < 0 else r + 4 for r in row] for row in table],
        [8, 9, 10, 11] + [-1] * 8, [12, 16], 2, max_tokens)
