"""Page numbers that the cache has not, in the table or on the stack: reported, and
no row's slot is made of them."""
import pytest
import torch

import speculative_decoding_drafter_markov_gb300 as dsp
from speculative_decoding_drafter_markov_gb300 import _lib
from test_gpu_target import err_word, ints

pytestmark = pytest.mark.gpu

# 2 requests, pages of 4, 10 pages: request 0 holds 3, request 1 holds 2
TABLE = [[7, 2, 5, -1, -1], [1, 0, -1, -1, -1]]
FREE = [3, 4, 6, 8, 9]


def call(lens, rows, held, table=TABLE, free=FREE, **kw):
    t, f, err = ints(table), ints(free + [-1] * (10 - len(free))), err_word()
    out = dsp.page_map(ints(lens), ints(rows), t, ints(held), f, ints([len(free)]), page=4, N=sum(rows), err=err, **kw)
    return {k: v.tolist() for k, v in out.items()}, t.tolist(), f.tolist(), int(err)


def test_good_pages_are_not_reported():
    out, table, free, err = call([9, 6], [3, 4], [3, 2])
    assert err == 0
    assert out["slot"] == [5 * 4 + 1, 5 * 4 + 2, 5 * 4 + 3, 2, 3, 9 * 4, 9 * 4 + 1]
    assert table[1][2] == 9 and out["n_free"] == [4]


@pytest.mark.parametrize("bad", [-1, 10, 1 << 30, -(1 << 31)])
def test_held_beyond_the_filled_entries(bad):
    """Rows that fall into an entry that nobody filled."""
    table = [TABLE[0][:3] + [bad, -1], TABLE[1]]
    out, after, free, err = call([9, 6], [6, 2], [4, 2], table)
    assert err == _lib.ERR_RANGE
    assert out["slot"] == [5 * 4 + 1, 5 * 4 + 2, 5 * 4 + 3, -1, -1, -1, 2, 3] and out["pos"] == [9, 10, 11, 12, 13, 14, 6, 7]
    assert after == table and out["held"] == [4, 2] and free[:5] == FREE


@pytest.mark.parametrize("bad", [-1, 10, 1 << 30])
def test_bad_page_given_back(bad):
    """It is reported when it goes to the stack, and again when it is taken."""
    table = [TABLE[0][:3] + [bad, -1], TABLE[1]]
    out, after, free, err = call([9, 6], [1, 2], [4, 2], table)
    assert err == _lib.ERR_RANGE and out["slot"] == [5 * 4 + 1, 2, 3] and out["n_free"] == [6] and free[:6] == FREE + [bad]
    out, after, free, err = call([9, 6], [1, 5], [3, 2], after, free[:6])
    assert err == _lib.ERR_RANGE and out["slot"] == [5 * 4 + 1, 2, 3, -1, -1, -1]
    assert after[1][2] == bad and out["n_free"] == [5]
    # given back and taken in one call
    out, after, free, err = call([9, 6], [1, 5], [4, 2], table)
    assert err == _lib.ERR_RANGE and out["slot"] == [5 * 4 + 1, 2, 3, -1, -1, -1] and after[1][2] == bad


@pytest.mark.parametrize("bad", [-1, 10, 1 << 30])
@pytest.mark.parametrize("tree", [False, True])
def test_bad_entry_of_the_stack(bad, tree):
    more = dict(parents=ints([-1, -1, 0, 1, 1, 2]), max_rows=5) if tree else {}
    out, after, free, err = call([9, 6], [1, 5], [3, 2], free=FREE[:4] + [bad], **more)
    assert err == _lib.ERR_RANGE and out["slot"] == [5 * 4 + 1, 2, 3, -1, -1, -1] and after[1][2] == bad
    # not taken: not looked at
    out, after, free, err = call([9, 6], [1, 2], [3, 2], free=FREE[:4] + [bad])
    assert err == 0


def test_page_numbers_of_the_last_page():
    out, table, free, err = call([9, 6], [3, 3], [3, 2], free=FREE[:4] + [9])
    assert err == 0 and out["slot"][-1] == 9 * 4


@pytest.mark.parametrize("R", [4000, 4077, 4078, 4079, 4090, 4095, 4096, 8192])
def test_any_number_of_requests(R):
    """Around the sums' 48 KB of shared memory, where a launch has to ask for more."""
    table, free = torch.full((R, 1), -1, dtype=torch.int32, device="cuda"), torch.arange(R, dtype=torch.int32, device="cuda")
    one, err = torch.ones(R, dtype=torch.int32, device="cuda"), err_word()
    out = dsp.page_map(one - 1, one, table, one - 1, free, ints([R]), page=4, N=R, err=err)
    assert int(err) == 0 and int(out["n_free"]) == 0
    assert table.flatten().tolist() == list(range(R - 1, -1, -1)) and out["row_start"].tolist() == list(range(R + 1))
    assert torch.equal(out["slot"], 4 * table.flatten())
