"""np_block_map against a request-by-request implementation on the host."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def host_step(tables, lens, new, kept, free, count, bs, tokens, mb):
    """One step; lists in, lists out: (tables, lens, free, count, starts, slots, positions, flags)."""
    tables, free = [list(t) for t in tables], list(free)
    rows, flags = len(lens), 0
    keep, get = [], []
    for r in range(rows):
        c, n, k = lens[r], new[r], lens[r] if kept is None else kept[r]
        if not 0 <= c <= mb * bs:
            flags |= 0x2
            c = min(max(c, 0), mb * bs)
        if n < 0 or (kept is not None and k < 0):
            flags |= 0x40
        n, k = max(n, 0), min(max(k, 0), c)
        if k + n > mb * bs:
            flags |= 0x2
            n = 0
        lens[r] = c
        keep.append(k)
        get.append(n)

    def blocks(x):
        return -(-x // bs)

    back = sum(max(0, blocks(lens[r]) - blocks(keep[r] + get[r])) for r in range(rows))
    tok = take = 0
    stop = False
    for r in range(rows):
        tok += get[r]
        take += max(0, blocks(keep[r] + get[r]) - blocks(lens[r]))
        no, out = tokens is not None and tok > tokens, take > count + back
        if no or out:
            if get[r] > 0:
                flags |= (0x40 if no else 0) | (0x100 if out else 0)
            stop = True
        if stop:
            get[r] = get[r] if not (no or out) else 0
    for r in reversed(range(rows)):
        need = blocks(keep[r] + get[r])
        for j in reversed(range(need, blocks(lens[r]))):
            if count < len(free):
                free[count] = tables[r][j]
                count += 1
            else:  # the list holds blocks that tables hold too: dropped
                flags |= 0x100
            tables[r][j] = -1
    starts, slots, positions = [0], [], []
    for r in range(rows):
        for j in range(blocks(lens[r]), blocks(keep[r] + get[r])):
            count -= 1
            tables[r][j] = free[count]
        for t in range(keep[r], keep[r] + get[r]):
            slots.append(tables[r][t // bs] * bs + t % bs)
            positions.append(t)
        starts.append(len(positions))
        lens[r] = keep[r] + get[r]
    if tokens is not None:
        slots += [-1] * (tokens - len(slots))
        positions += [0] * (tokens - len(positions))
    return tables, lens, free, count, starts, slots, positions, flags


class State:
    def __init__(self, rows, mb, bs, nb, lens, seed=0):
        gen = torch.Generator().manual_seed(seed)
        ids = torch.randperm(nb, generator=gen).tolist()
        self.bs, self.mb, self.nb = bs, mb, nb
        self.lens = list(lens)
        self.tables = [[-1] * mb for _ in range(rows)]
        for r, c in enumerate(lens):
            for j in range(-(-c // bs)):
                self.tables[r][j] = ids.pop()
        self.count = len(ids)
        self.free = ids + [-7] * (nb - len(ids))
        self.dev = [torch.tensor(x, dtype=torch.int32, device="cuda").view(s) for x, s in
                    ((self.tables, (rows, mb)), (self.lens, (rows,)), (self.free, (nb,)), ([self.count], (1,)))]

    def step(self, npg, new, kept=None, tokens=None, positions=True):
        rows = len(self.lens)
        i32 = dict(dtype=torch.int32, device="cuda")
        starts = torch.full((rows + 1,), 99, **i32)
        slots = None if tokens is None else torch.full((tokens,), 99, dtype=torch.int64, device="cuda")
        pos = torch.full((tokens,), 99, **i32) if tokens is not None and positions else None
        err = torch.zeros(1, **i32)
        tables, lens, free, count = self.dev
        npg.np_block_map(tables, lens, torch.tensor(new, **i32), free, count, starts, slots, pos, self.bs,
                         kept_lens=None if kept is None else torch.tensor(kept, **i32), err_word=err)
        want = host_step(self.tables, self.lens, new, kept, self.free, self.count, self.bs, tokens, self.mb)
        self.tables, self.lens, self.free, self.count = want[:4]
        assert lens.tolist() == self.lens
        assert starts.tolist() == want[4]
        assert tables.tolist() == self.tables
        assert int(count) == self.count and free.tolist() == self.free
        if slots is not None:
            assert slots.tolist() == want[5]
            if pos is not None:
                assert pos.tolist() == want[6]
        return int(err), want[7]


@pytest.mark.parametrize("bs", [1, 5, 16, 64])
@pytest.mark.parametrize("rows", [1, 33, 700, 1025, 4096])
def test_decode_steps(nplib, rows, bs):
    gen = torch.Generator().manual_seed(rows)
    lens = torch.randint(0, 100, (rows,), generator=gen).tolist()
    st = State(rows, 130 // bs + 2, bs, rows * (130 // bs + 2) + 5, lens)
    for k in range(3):
        got, want = st.step(nplib, [1] * rows, tokens=rows + k)
        assert got == want == 0


@pytest.mark.parametrize("bs", [1, 16])
def test_prompts_rollback_and_release(nplib, bs):
    gen = torch.Generator().manual_seed(bs)
    rows, mb = 40, 4000 // bs
    st = State(rows, mb, bs, rows * mb, [0] * rows)
    for k in range(6):
        new = torch.randint(0, 300, (rows,), generator=gen).tolist()
        kept = [max(0, c - int(x)) for c, x in zip(st.lens, torch.randint(0, 200, (rows,), generator=gen))]
        if k == 3:
            kept = [0 if r % 3 == 0 else c for r, c in enumerate(st.lens)]
            new = [0 if r % 3 == 0 else n for r, n in enumerate(new)]
        got, want = st.step(nplib, new, kept if k else None, tokens=sum(new) + 17 * (k % 2))
        assert got == want == 0
    st.step(nplib, [0] * rows, [0] * rows)  # everything goes back
    assert st.count == rows * mb and sorted(st.free) == list(range(rows * mb))


def test_a_step_taken_back_leaves_the_list_as_it_was(nplib):
    st = State(20, 40, 16, 500, [7 * r for r in range(20)])
    before, lens = list(st.free), list(st.lens)
    st.step(nplib, [40 + r for r in range(20)], tokens=2000)
    st.step(nplib, [0] * 20, lens)
    assert st.free[:st.count] == before[:st.count] and st.lens == lens


def test_free_list_runs_out(nplib):
    st = State(10, 20, 16, 12, [0] * 10)
    got, want = st.step(nplib, [40] * 10, tokens=400)  # three blocks each: four rows fit
    assert got == want == nplib.NP_FLAG_BLOCKS
    assert st.lens == [40] * 4 + [0] * 6
    # freed blocks serve the same step; rows refused still give back what they do not keep
    got, want = st.step(nplib, [0, 0, 100, 0, 50, 9, 0, 0, 0, 0], [3, 0, 40, 33, 0, 0, 0, 0, 0, 0], tokens=300)
    assert got == want


def test_no_room_for_tokens_or_in_tables(nplib):
    st = State(6, 4, 8, 60, [0, 5, 8, 31, 32, 1])
    got, want = st.step(nplib, [1, 1, 1, 2, 1, 31], tokens=100)  # rows 3 and 4: past their tables
    assert got == want == nplib.NP_FLAG_CONTEXT
    got, want = st.step(nplib, [2, 2, 2, 0, 0, 0], [0, 0, 4, 9, 9, 9], tokens=4)
    assert got == want == nplib.NP_FLAG_QUERY
    assert st.lens == [2, 2, 4, 9, 9, 9]


def test_bad_lengths_and_entries(nplib):
    st = State(4, 4, 8, 60, [3, 9, 0, 0])
    st.dev[1][2:] = torch.tensor([-4, 99], dtype=torch.int32, device="cuda")
    st.lens[2:] = [-4, 99]
    st.tables[3] = [50, 51, 52, 53]
    st.dev[0][3] = torch.tensor(st.tables[3], dtype=torch.int32, device="cuda")
    got, want = st.step(nplib, [-3, 1, 1, 0], [2, -1, 0, 8], tokens=8)
    # (row 3's blocks are in the list already, which has no room for all of them again)
    assert got == want == nplib.NP_FLAG_CONTEXT | nplib.NP_FLAG_QUERY | nplib.NP_FLAG_BLOCKS


def test_a_list_entry_outside_the_pool(nplib):
    i32 = dict(dtype=torch.int32, device="cuda")
    tables, lens, free = torch.full((2, 3), -1, **i32), torch.zeros(2, **i32), torch.tensor([0, 1, 9, -2], **i32)
    count, starts, err = torch.tensor([4], **i32), torch.zeros(3, **i32), torch.zeros(1, **i32)
    slots, pos = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, **i32)
    nplib.np_block_map(tables, lens, torch.tensor([1, 3], **i32), free, count, starts, slots, pos, 2, err_word=err)
    # taken: -2 and 9 (of a pool of four blocks: neither is one), then 1
    assert tables.tolist() == [[-1, -1, -1], [-1, 1, -1]] and slots.tolist() == [-1, -1, -1, 2]
    assert int(err) == nplib.NP_FLAG_BLOCK_ID and int(count) == 1


def test_bad_counts(nplib):
    for bad, lens in ((-1, [0, 0]), (5, [0, 0])):
        i32 = dict(dtype=torch.int32, device="cuda")
        tables, free = torch.full((2, 3), -1, **i32), torch.arange(4, **i32)
        count, starts, err = torch.tensor([bad], **i32), torch.zeros(3, **i32), torch.zeros(1, **i32)
        slots = torch.zeros(2, dtype=torch.int64, device="cuda")
        nplib.np_block_map(tables, torch.tensor(lens, **i32), torch.ones(2, **i32), free, count, starts, slots,
                           None, 2, err_word=err)
        assert int(err) == nplib.NP_FLAG_BLOCKS
        assert slots.tolist() == ([-1, -1] if bad < 0 else [6, 4]) and int(count) == (0 if bad < 0 else 2)


def test_kept_lens_may_be_context_lens_and_no_rows(nplib):
    i32 = dict(dtype=torch.int32, device="cuda")
    tables, lens, free = torch.full((1, 3), -1, **i32), torch.zeros(1, **i32), torch.arange(4, **i32)
    count, starts = torch.tensor([4], **i32), torch.zeros(2, **i32)
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    nplib.np_block_map(tables, lens, torch.full((1,), 3, **i32), free, count, starts, slots, None, 2, kept_lens=lens)
    assert slots.tolist() == [6, 7, 4] and lens.tolist() == [3]
    empty = torch.zeros(0, **i32)
    nplib.np_block_map(torch.zeros(0, 3, **i32), empty, empty, free, count, starts[:1], slots, None, 2)
    assert slots.tolist() == [-1] * 3 and int(count) == 2
