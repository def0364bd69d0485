"""The prompt attention's division of work, on the CPU: a line-by-line Python
model of the plan kernel's arithmetic (prefix sums of kv tiles in closed form and
a fixed cost per unit, equal shares, ends moved to unit starts, the list of cut units) and of the
blocks' walk, against brute force over random chunks and contexts: every kv
tile of every unit is read exactly once, every cut unit is named once with all
the blocks that hold its pieces, and every other unit lies whole in one block.
"""
import random

import pytest


def floor_sum(n, m, a, b):
    s = 0
    while n > 0:
        s += n * (n - 1) // 2 * (a // m) + n * (b // m)
        a %= m
        b %= m
        y = a * n + b
        if y < m:
            break
        n, b, m, a = y // m, y % m, a, m
    return s


def kv_tiles(n, c, bn, tok):
    e = max(0, c - n + min(tok, n))
    return max(1, -(-e // bn))


def units_of(n, U):
    return -(-n // U)


def tile_cost(n, T, mt, costs, a):
    full, single, _ = costs
    return single if (a * mt + 1) * T >= n else full


def row_prefix(n, c, T, mt, bn, costs, units, k):
    """Cost of a row's first k units, of mt tiles of T chunk tokens each."""
    if k <= 0:
        return 0
    U = T * mt
    full, _, unit = costs
    cost = k * unit
    if k == units:
        k -= 1
        cost += kv_tiles(n, c, bn, n) * tile_cost(n, T, mt, costs, k)
    base = c - n
    z0 = (-base) // U if base < 0 else 0
    z = min(z0, k)
    return cost + (z + floor_sum(k - z, bn, U, base + (z + 1) * U + bn - 1)) * full


def plan(rows, heads, T, mt, bn, ctas, costs, min_share):
    """rows: [(n, c)]; returns where each block's share begins (and the end), and the cut units."""
    U = T * mt
    pre = [0]
    for n, c in rows:
        u = units_of(n, U)
        pre.append(pre[-1] + row_prefix(n, c, T, mt, bn, costs, u, u) * heads)
    W = pre[-1]
    pe = min(ctas, max(1, -(-W // min_share)))
    pos = []
    for b in range(ctas + 1):
        share = W // pe
        x = W if b >= pe else share * b + (W % pe) * b // pe
        q = (len(rows), 0, 0, 0)
        if x < W:
            lo, hi = 0, len(rows)
            while hi - lo > 1:
                mid = (lo + hi) // 2
                if pre[mid] <= x:
                    lo = mid
                else:
                    hi = mid
            n, c = rows[lo]
            u = units_of(n, U)
            wh = (pre[lo + 1] - pre[lo]) // heads
            kvh = (x - pre[lo]) // wh
            inn = (x - pre[lo]) - kvh * wh
            a, e = 0, u
            while e - a > 1:
                mid = (a + e) // 2
                if row_prefix(n, c, T, mt, bn, costs, u, mid) <= inn:
                    a = mid
                else:
                    e = mid
            s0 = row_prefix(n, c, T, mt, bn, costs, u, a)
            cost = tile_cost(n, T, mt, costs, a)
            nk = kv_tiles(n, c, bn, (a + 1) * U)
            off = (inn - s0 - costs[2]) // cost
            if off <= 0 or off * cost * 16 <= share:
                off = 0
            elif (nk - off) * cost * 16 <= share:
                off, a = 0, a + 1
                if a >= u:
                    a, kvh = 0, kvh + 1
                    if kvh >= heads:
                        kvh, lo = 0, lo + 1
            q = (lo, kvh, a, off)
        pos.append(q)
    cuts = []
    for b in range(ctas):
        cut, s, e = None, pos[b], pos[b + 1]
        if e[3] > 0 and (s[:3] != e[:3] or s[3] == 0):
            last = b + 1
            while last + 1 <= ctas and pos[last + 1][:3] == e[:3]:
                last += 1
            cut = (e[0], e[1], e[2], last)
        cuts.append(cut)
    return pos, cuts


def walk(rows, heads, U, bn, pos, end):
    """The segments (row, head, unit, kv0, kv1, nk) of one block."""
    r, kvh, m, off = pos
    while r < len(rows):
        u = units_of(rows[r][0], U)
        while m >= u:
            m = 0
            kvh += 1
            if kvh < heads and u > 0:
                break
            kvh = 0
            r += 1
            if r >= len(rows):
                return
            u = units_of(rows[r][0], U)
        last = (r, kvh, m) == end[:3]
        if off >= end[3] if last else (r, kvh, m) > end[:3]:
            return
        nk = kv_tiles(*rows[r], bn, (m + 1) * U)
        yield r, kvh, m, off, end[3] if last else nk, nk
        off = 0
        m += 1


def check(rows, heads, T, mt, bn, ctas, costs, min_share):
    U = T * mt
    pos, cuts = plan(rows, heads, T, mt, bn, ctas, costs, min_share)
    assert all(x <= y for x, y in zip(pos, pos[1:]))
    pieces = {}
    for b in range(ctas):
        segs = list(walk(rows, heads, U, bn, pos[b], pos[b + 1]))
        # a block cuts at most its first and its last unit: one slot each
        slots = [0 if kv0 > 0 else 1 for _, _, _, kv0, kv1, nk in segs if kv0 > 0 or kv1 < nk]
        assert len(slots) == len(set(slots))
        for r, k, m, kv0, kv1, nk in segs:
            assert 0 <= kv0 < kv1 <= nk
            pieces.setdefault((r, k, m), []).append((kv0, kv1, nk, b))
    want = {(r, k, m): kv_tiles(n, c, bn, (m + 1) * U) for r, (n, c) in enumerate(rows)
            for k in range(heads) for m in range(units_of(n, U))}
    assert pieces.keys() == want.keys()
    named = {cut[:3]: (b, cut[3]) for b, cut in enumerate(cuts) if cut}
    assert len(named) == sum(c is not None for c in cuts)
    for key, ps in pieces.items():
        assert ps[0][0] == 0 and ps[-1][1] == want[key] == ps[0][2]
        assert all(x[1] == y[0] for x, y in zip(ps, ps[1:]))
        blocks = [x[3] for x in ps]
        if len(ps) == 1:
            assert key not in named
        else:
            # the blocks from the first to the one named last, but for empty shares (which begin
            # where the next one does: the join skips them)
            first, last = named[key]
            assert blocks == [b for b in range(first, last + 1) if pos[b] != pos[b + 1]]
            assert first == blocks[0]
    assert named.keys() == {k for k, v in pieces.items() if len(v) > 1}


@pytest.mark.parametrize("seed", range(8))
def test_shares_cover_every_tile_once(seed):
    rnd = random.Random(seed)
    for _ in range(120):
        G = rnd.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        tile, mt, bn = rnd.choice([(64, 1, 64), (128, 2, 128), (128, 1, 64), (128, 2, 64)])
        rows = []
        for _ in range(rnd.choice([1, 1, 2, 5, 30])):
            n = rnd.choice([0, 1, rnd.randint(1, 40), rnd.randint(1, 2000)])
            c = rnd.choice([n, n, rnd.randint(0, 3 * n + 1), n + rnd.randint(0, 9000)])
            rows.append((n, c))
        check(rows, rnd.choice([1, 2, 3, 8]), tile // G, mt, bn, rnd.choice([1, 4, 148, 152, 160]),
              rnd.choice([(1, 1, 0), (1, 1, 2), (3, 2, 4), (3, 2, 9)]), rnd.choice([1, 2, 4, 8]))


def test_prefix_in_closed_form():
    rnd = random.Random(99)
    for _ in range(300):
        n, T, bn = rnd.randint(1, 700), rnd.choice([8, 14, 25, 42, 64, 128]), rnd.choice([64, 128])
        mt, costs = rnd.choice([1, 2]), rnd.choice([(1, 1, 0), (3, 2, 4)])
        c = rnd.randint(0, 2 * n + 300)
        u = units_of(n, T * mt)
        run = 0
        for k in range(u + 1):
            assert row_prefix(n, c, T, mt, bn, costs, u, k) == run
            run += kv_tiles(n, c, bn, (k + 1) * T * mt) * tile_cost(n, T, mt, costs, k) + costs[2]


def test_far_positions_stay_exact():
    # tiles of a 2^31-token table are counted in 64 bits
    n, c, T, bn = 5000, 2**31 - 300, 16, 128
    u = units_of(n, 2 * T)
    assert row_prefix(n, c, T, 2, bn, (1, 1, 0), u, u) == \
        sum(kv_tiles(n, c, bn, (k + 1) * 2 * T) for k in range(u))
