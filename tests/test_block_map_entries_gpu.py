"""np_block_map where a row gives back table entries that are no blocks."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _step(npg, tables, lens, new, free, count, bs, tokens, kept=None):
    i32 = dict(dtype=torch.int32, device="cuda")
    t = [torch.tensor(x, **i32) for x in (tables, lens, new, free, [count])]
    starts, err = torch.zeros(len(lens) + 1, **i32), torch.zeros(1, **i32)
    slots = torch.zeros(tokens, dtype=torch.int64, device="cuda") if tokens else None
    npg.np_block_map(t[0], t[1], t[2], t[3], t[4], starts, slots, None, bs, err_word=err,
                     kept_lens=None if kept is None else torch.tensor(kept, **i32))
    return (t[0].tolist(), t[1].tolist(), t[3].tolist()[:int(t[4])], int(t[4]),
            None if slots is None else slots.tolist(), int(err))


def test_entries_that_are_no_blocks_do_not_reach_the_free_list(nplib):
    # two rows end; the first one's second entry and the last one's first are no blocks of the pool's 8
    tables = [[3, -1, 5, -1], [1, 2, -1, -1], [99, 6, -1, -1]]
    got = _step(nplib, tables, [6, 4, 3], [0, 0, 0], [7, 0, 9, 9, 9, 9, 9, 9], 2, 2, 0, [0, 4, 0])
    assert got[0] == [[-1] * 4, [1, 2, -1, -1], [-1] * 4] and got[1] == [0, 4, 0]
    assert got[2] == [7, 0, 6, 5, 3] and got[3] == 5
    assert got[5] == nplib.NP_FLAG_BLOCK_ID


def test_the_same_step_takes_what_is_left(nplib):
    """One row ends with an entry that is no block, another takes more than the rest."""
    got = _step(nplib, [[4, -7, -1, -1], [-1] * 4], [2, 0], [0, 4], [2, 0, 0, 0, 0], 2, 1, 5, [0, 0])
    # counted on: 0, 2, 4 and the lost one; there are three
    assert got[0] == [[-1] * 4, [4, 0, 2, -1]] and got[4] == [4, 0, 2, -1, -1]
    assert got[2] == [] and got[3] == 0 and got[5] == nplib.NP_FLAG_BLOCK_ID


@pytest.mark.parametrize("rows,mb", [(1, 3000), (4096, 3), (300, 33)])
def test_many_entries(nplib, rows, mb):
    """Every third entry of all rows is no block: the others go back in the documented order."""
    nb = rows * mb + 10
    ids = torch.randperm(nb, generator=torch.Generator().manual_seed(rows)).to(torch.int32)
    tables, free = ids[:rows * mb].view(rows, mb).clone(), ids[rows * mb:].tolist()
    flat = tables.view(-1)
    flat[::3] = torch.tensor([-1, nb, -2**31, 2**31 - 1], dtype=torch.int32).repeat(rows * mb)[:len(flat[::3])]
    want = free + [b for b in reversed(flat.tolist()) if 0 <= b < nb]
    got = _step(nplib, tables.tolist(), [mb] * rows, [0] * rows, free + [-9] * (nb - 10), 10, 1, 0, [0] * rows)
    assert got[2] == want and got[5] == nplib.NP_FLAG_BLOCK_ID
    assert (torch.tensor(got[0]) == -1).all()


def test_a_lost_block_is_nobodys(nplib):
    """A bad list entry goes into a row's table as -1; the row's end does not put it back."""
    i32 = dict(dtype=torch.int32, device="cuda")
    tables, lens, free = torch.full((1, 2), -1, **i32), torch.zeros(1, **i32), torch.tensor([1, 0, 77, 3], **i32)
    count, starts, err = torch.tensor([4], **i32), torch.zeros(2, **i32), torch.zeros(1, **i32)
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    nplib.np_block_map(tables, lens, torch.tensor([2], **i32), free, count, starts, slots, None, 1, err_word=err)
    assert tables.tolist() == [[3, -1]] and slots.tolist() == [3, -1] and int(err) == nplib.NP_FLAG_BLOCK_ID
    err.zero_()
    nplib.np_block_map(tables, lens, torch.zeros(1, **i32), free, count, starts, None, None, 1,
                       kept_lens=torch.zeros(1, **i32), err_word=err)
    assert int(err) == nplib.NP_FLAG_BLOCK_ID and int(count) == 3 and free[:3].tolist() == [1, 0, 3]
