"""The prompt attention's division of work, on the CPU: a line-by-line Python
model of the plan kernel's arithmetic (prefix sums of kv tiles in closed form,
equal shares, ends moved to unit starts, the list of cut units) and of the
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


def row_prefix(n, c, U, bn, units, k):
    if k <= 0:
        return 0
    last = 0
    if k == units:
        last = kv_tiles(n, c, bn, n)
        k -= 1
    base = c - n
    z0 = (-base) // U if base < 0 else 0
    z = min(z0, k)
    return z + floor_sum(k - z, bn, U, base + (z + 1) * U + bn - 1) + last


def plan(rows, heads, U, bn, ctas, min_tiles):
    """rows: [(n, c)]; returns (pos, length, cuts) per block."""
    pre = [0]
    for n, c in rows:
        u = units_of(n, U)
        pre.append(pre[-1] + row_prefix(n, c, U, bn, u, u) * heads)
    W = pre[-1]
    pe = min(ctas, max(1, -(-W // min_tiles)))
    at, unit_end, pos = [], [], []
    for b in range(ctas + 1):
        share = W // pe
        t = W if b >= pe else share * b + (W % pe) * b // pe
        q, end = (len(rows), 0, 0, 0), W
        if t < W:
            lo, hi = 0, len(rows)
            while hi - lo > 1:
                mid = (lo + hi) // 2
                if pre[mid] <= t:
                    lo = mid
                else:
                    hi = mid
            n, c = rows[lo]
            u = units_of(n, U)
            wh = (pre[lo + 1] - pre[lo]) // heads
            rem = t - pre[lo]
            kvh, inn = rem // wh, rem % wh
            a, e = 0, u
            while e - a > 1:
                mid = (a + e) // 2
                if row_prefix(n, c, U, bn, u, mid) <= inn:
                    a = mid
                else:
                    e = mid
            s0 = row_prefix(n, c, U, bn, u, a)
            s1 = row_prefix(n, c, U, bn, u, a + 1)
            ustart = t - (inn - s0)
            end = ustart + s1 - s0
            off = inn - s0
            if off > 0 and off * 16 <= share:
                t, off = ustart, 0
            elif off > 0 and (end - t) * 16 <= share:
                t, off = end, 0
                r2, k2, a2 = lo, kvh, a + 1
                if a2 >= u:
                    a2, k2 = 0, k2 + 1
                    if k2 >= heads:
                        k2, r2 = 0, r2 + 1
                q, end = (r2, k2, a2, 0), t
            if q[0] == len(rows) and t < W:
                q = (lo, kvh, a, off)
        at.append(t)
        unit_end.append(end)
        pos.append(q)
    cuts = []
    for b in range(ctas):
        cut = None
        e = pos[b + 1]
        if at[b + 1] > at[b] and at[b + 1] < W and e[3] > 0 and at[b + 1] - e[3] >= at[b]:
            last = b + 1
            while last + 1 < ctas and at[last + 1] < unit_end[b + 1]:
                last += 1
            cut = (e[0], e[1], e[2], last)
        cuts.append(cut)
    return pos[:ctas], [at[b + 1] - at[b] for b in range(ctas)], cuts


def walk(rows, heads, U, bn, pos, left):
    """The segments (row, head, unit, kv0, kv1, nk) of one block."""
    r, kvh, m, off = pos
    while left > 0:
        u = units_of(rows[r][0], U)
        while m >= u:
            m = 0
            kvh += 1
            if kvh < heads and u > 0:
                break
            kvh = 0
            r += 1
            assert r < len(rows)
            u = units_of(rows[r][0], U)
        nk = kv_tiles(*rows[r], bn, (m + 1) * U)
        kv1 = off + left if left < nk - off else nk
        yield r, kvh, m, off, kv1, nk
        left -= kv1 - off
        off = 0
        m += 1


def check(rows, heads, U, bn, ctas, min_tiles):
    pos, length, cuts = plan(rows, heads, U, bn, ctas, min_tiles)
    assert all(x >= 0 for x in length)
    pieces = {}
    for b in range(ctas):
        segs = list(walk(rows, heads, U, bn, pos[b], length[b]))
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
            assert blocks == list(range(blocks[0], blocks[-1] + 1))
            assert named[key] == (blocks[0], blocks[-1])
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
        check(rows, rnd.choice([1, 2, 3, 8]), tile // G * mt, bn, rnd.choice([1, 4, 148, 152, 160]),
              rnd.choice([1, 2, 4, 7]))


def test_prefix_in_closed_form():
    rnd = random.Random(99)
    for _ in range(300):
        n, U, bn = rnd.randint(1, 700), rnd.choice([8, 14, 50, 64, 85, 256]), rnd.choice([64, 128])
        c = rnd.randint(0, 2 * n + 300)
        u = units_of(n, U)
        run = 0
        for k in range(u + 1):
            assert row_prefix(n, c, U, bn, u, k) == run
            run += kv_tiles(n, c, bn, (k + 1) * U)


def test_far_positions_stay_exact():
    # tiles of a 2^31-token table are counted in 64 bits
    n, c, U, bn = 5000, 2**31 - 300, 32, 128
    u = units_of(n, U)
    assert row_prefix(n, c, U, bn, u, u) == sum(kv_tiles(n, c, bn, (k + 1) * U) for k in range(u))
