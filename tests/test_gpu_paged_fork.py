"""Forks of the cache's rows on the GPU where tables and counts are at odds, or rows are named twice: outcomes written out."""
import pytest
import torch

import video_diffusion_transformer_sage_gb300 as sage

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _fork(refs, table, src, dst, tokens, page=8):
    pool = sage.PagedPool(_i32(refs), _i32(table), page)
    got = sage.sage_paged_fork(pool, _i32(src), _i32(dst), _i32(tokens))
    return [x.tolist() for x in got], pool.refs.tolist(), pool.page_table.tolist(), sage.sage_check_device_status(pool.status)


@pytest.mark.parametrize("again", range(3))
def test_pages_of_the_source_that_nobody_holds(again):
    """Page 0 and 2 are free and -2 means out of use, yet the source's row names them: the children do not share them, the free
    ones go to the children that need a page, and nothing is copied from them."""
    got, refs, table, status = _fork([0, 1, 0, -2, 0, 0], [[0, 1, 3, 2], [-1] * 4, [-1] * 4, [-1] * 4], [0, 0, 0], [1, 2, 3], [28, 28, 12])
    assert got == [[-1, -1, 1], [0, 2, 4], [4, 4, 4], [1, 1, 1]]
    assert table == [[0, 1, 3, 2], [-1, 1, -1, 0], [-1, 1, -1, 2], [-1, 4, -1, -1]]
    assert refs == [1, 3, 1, -2, 1, 0] and status == (1, 24)


def test_a_begun_page_and_a_first_page_that_nobody_holds():
    got, refs, table, status = _fork([2, 0, 0, 0], [[1, 0], [0, 1], [-1, -1], [-1, -1]], [0, 1], [2, 3], [16, 9])
    assert got == [[-1, -1], [-1, 1], [0, 1], [1, 1]]
    assert table == [[1, 0], [0, 1], [-1, 0], [0, 1]] and refs == [4, 1, 0, 0] and status == (1, 24)


def test_many_forks_of_rows_that_name_free_pages():
    """Half of the parents' pages are free pages, which are given out by the same call: whoever comes first, counts are the
    entries that hold a page.  More forks than a CTA has warps."""
    rows, width, page = 500, 9, 16
    n_pages = 2000
    table = [[(r * width + i) % n_pages for i in range(width)] if r < 100 else [-1] * width for r in range(rows)]
    refs = [0] * n_pages
    for r in range(100):
        for i in range(0, width, 2):          # every second page of a parent is counted
            refs[table[r][i]] += 1
    src, dst = [k % 100 for k in range(400)], [100 + k for k in range(400)]
    tokens = [(7 * k) % (width * page) for k in range(400)]
    first = None
    for _ in range(5):
        got, after, tab, status = _fork(refs, table, src, dst, tokens, page)
        assert got[3] == [1] * 400 and status == (1, 24)
        given = [p for p in got[1] if p >= 0]
        assert len(set(given)) == len(given) and all(refs[p] == 0 for p in given) and given == sorted(given)
        want = list(refs)
        for k in range(400):
            full, part = divmod(tokens[k], page)
            parent, child = table[src[k]], [-1] * width
            for i in range(full):
                if refs[parent[i]] > 0:
                    child[i] = parent[i]
                    want[parent[i]] += 1
            if part:
                child[full] = got[1][k]
                want[child[full]] += 1
                assert got[0][k] == (parent[full] if refs[parent[full]] > 0 else -1) and got[2][k] == part
            else:
                assert (got[0][k], got[1][k], got[2][k]) == (-1, -1, 0)
            assert tab[dst[k]] == child
        assert after == want
        first = first or (got, after, tab)
        assert first == (got, after, tab)


def test_forks_that_are_not_possible_by_themselves_stand_in_no_others_way():
    """Row 3 is the dst of a fork with src = dst, row 1 that of one whose src does not exist and that of one whose dst holds a
    page: other forks have row 3 and 2 as src and row 1 as dst all the same."""
    world = [0, 1, 1, 0, 0], [[-1, -1], [-1, -1], [1, -1], [2, -1], [-1, -1]]
    got, refs, table, status = _fork(*world, [3, 3], [3, 4], [8, 8])
    assert got == [[-1, -1], [-1, -1], [0, 0], [0, 1]] and status == (1, 25)
    assert table == [[-1, -1], [-1, -1], [1, -1], [2, -1], [2, -1]] and refs == [0, 1, 2, 0, 0]
    got, refs, table, status = _fork(*world, [9, 2], [1, 1], [8, 8])
    assert got == [[-1, -1], [-1, -1], [0, 0], [0, 1]] and status == (1, 25)
    assert table == [[-1, -1], [1, -1], [1, -1], [2, -1], [-1, -1]] and refs == [0, 2, 1, 0, 0]
    got, refs, table, status = _fork(*world, [3, 2], [2, 1], [8, 8])
    assert got == [[-1, -1], [-1, -1], [0, 0], [0, 1]] and status == (1, 25)
    assert table == [[-1, -1], [1, -1], [1, -1], [2, -1], [-1, -1]] and refs == [0, 2, 1, 0, 0]


def test_forks_possible_by_themselves_stand_in_others_way():
    """The second fork to a row, and a fork of a row that is made in the call."""
    world = [0, 1, 0], [[1, -1], [-1, -1], [-1, -1], [-1, -1]]
    got, refs, table, status = _fork(*world, [0, 0, 1], [1, 1, 2], [8, 8, 8])
    assert got == [[-1] * 3, [-1] * 3, [0] * 3, [1, 0, 0]] and status == (1, 25)
    assert table == [[1, -1], [1, -1], [-1, -1], [-1, -1]] and refs == [0, 2, 0]
