"""hs.paged_extend over tables and rings with entries that are no pages."""
import pytest

import step_ref
from test_gpu_extend_rope import extend

pytestmark = pytest.mark.gpu

NAMES = "table ring ends lens attend cu slot row pos".split()


def check(new, lens, table, ring, ends, page, max_tokens):
    """All outputs are the definition's, which passes pages on as they stand."""
    for in_place in (False, True):
        got = extend(new, lens, table, ring, ends, page, max_tokens, in_place)
        want = step_ref.extend(new, lens, table, ring, ends, page, max_tokens)
        for name, a, b in zip(NAMES, got, want):
            assert a == b, name
    return dict(zip(NAMES, got)), got[-1]


@pytest.mark.parametrize("bad", [-1, 6, 77, 2 ** 31 - 1, -2 ** 31])
def test_given_back(bad):
    got, status = check([-4], [4], [[bad, 1]], [4, 5, 0, 2, -1, -1], [0, 4], 2, 0)
    assert status == 6
    assert got["lens"] == [0] and got["attend"] == [0] and got["ends"] == [0, 6]
    assert got["ring"] == [4, 5, 0, 2, bad, 1]
    # Only the pages that change hands are looked at.
    got, status = check([-1, -1], [3, 4], [[bad, 1], [2, 3]], [4, 5, 0, -1, -1, -1], [0, 3], 2, 0)
    assert status == 0 and got["lens"] == [2, 3] and got["ends"] == [0, 4]


@pytest.mark.parametrize("bad", [-1, 6, 77, 2 ** 31 - 1, -2 ** 31])
def test_grown_over(bad):
    got, status = check([2, 1], [1, 1], [[bad, -1], [2, -1]], [4, 5, 0, 1, 3, -1], [0, 5], 2, 4)
    assert status == 6
    assert got["lens"] == [3, 2] and got["attend"] == [3, 2] and got["ends"] == [1, 5]
    assert got["slot"] == [-1, 8, 5, -1] and got["row"] == [0, 0, 1, -1] and got["pos"] == [1, 2, 1, -1]
    got, status = check([3], [2], [[3, -1, -1]], [bad, 5, 0, 1, -1, -1], [0, 4], 2, 3)
    assert status == 6
    assert got["lens"] == [5] and got["ends"] == [2, 4] and got["table"] == [[3, bad, 5]]
    assert got["slot"] == [-1, -1, 10] and got["pos"] == [2, 3, 4]


def test_many_pages_by_several_ctas():
    """More new tokens than one CTA takes, and a bad page in each of a cluster's shares."""
    rows, page = 64, 4
    table = [[r * 8 + b for b in range(8)] for r in range(rows)]
    for r in range(0, rows, 5):
        table[r][r % 8] = 9999
    ring = [rows * 8 + i for i in range(rows)] + [-1] * rows * 8
    new = [-32 if r % 2 else 1 for r in range(rows)]
    got, status = check(new, [32 if r % 2 else 31 for r in range(rows)], table, ring, [0, rows], page,
                        4000)
    assert status == 6 and got["ends"] == [0, rows + rows // 2 * 8]


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("rows", [2, 33, 1000, 4096])
@pytest.mark.parametrize("max_tokens", [40, 4000])
def test_one_code_for_several_errors(rows, first, max_tokens):
    """A length past its table, a refused request and a bad page in one call: the
    code does not depend on which thread finds which, or when."""
    def call(at_length, at_refused, at_page):
        table = [[r, -1] for r in range(rows)]
        new, lens = [0] * rows, [1] * rows
        if at_refused is not None:
            new[at_refused] = 9
        if at_page is not None:
            new[at_page], table[at_page][0] = 1, -7
        if at_length is not None:
            lens[at_length] = 5
        ring = [rows, rows + 1] + [-1] * rows
        return extend(new, lens, table, ring, [0, 2], 2, max_tokens, True)[-1]

    a, b = (0, rows - 1) if first else (rows - 1, 0)
    for _ in range(20):
        assert call(a, b, None) == 6 and call(None, a, b) == 3 and call(None, None, a) == 6
        assert call(None, a, None) == 3 and call(None, None, None) == 0
        if rows > 2:
            assert call(a, b, rows // 2) == 6
