"""A model of the paged attention's division of work (extend_prepare_kernel in csrc/swska_extend.cu), in the kernel's integer
arithmetic (32-bit unsigned where it has that) and its blocks of 256 sequences, checked on the CPU: the units of a query tile
cover its key tiles once, in the columns' order; units, parts and counters stay inside the workspace and no two share one; the
units that a column's range names are those that were written."""
import math
import random

import pytest

NT, U32 = 256, 2 ** 32 - 1
SMS = 148


class Route:
    def __init__(self, rows, tile, groups, ctas, min_chunk, rows_div, split_cost, items, M):
        self.rows, self.tile, self.min_chunk, self.rows_div, self.split_cost = rows, tile, min_chunk, rows_div, split_cost
        self.cols = max(1, ctas // groups)
        self.cap_items = min(items, M)


def plan(M, N, H, max_len, tensor):
    """extend_plan: (routes, short_len)."""
    max_len = min(max_len, M)
    if tensor:
        heads = 8 if N * -(-H // 8) >= 48 else 4
        groups = -(-H // heads)
        few = Route(16, 32, groups, (2 if -(-H // groups) <= 4 else 1) * SMS, 2, 16, 6, N, M)
        many = Route(128, 128, (H + 1) // 2, SMS, 4, 0, 12, M // 128 + N, M) if max_len > 16 else None
        return [few, many], 16
    rows = 16 if max_len <= 16 else 64
    return [Route(rows, 64, H, (4 if rows == 16 else 2) * SMS, 1, 0, 1, M // rows + N, M), None], 0


def key_tiles(ctx, length, q0, rows, tile, W, S):
    p0 = ctx + q0
    p1 = ctx + min(q0 + rows, length) - 1
    lo = max(p0 - W + 1, 0) // tile
    sink = min(-(-S // tile), lo)
    return sink + p1 // tile - lo + 1


def division(routes, short_len, i, seqs, W, S, guard=True):
    """(units: {index: dict}, range: [(first, last)] per column) of route i; None where it gives up."""
    r = routes[i]
    N = len(seqs)
    div = lambda a, b: a // b

    def work(n, shift):
        ctx, length = seqs[n]
        if length == 0:
            return 0, 0
        is_short = length <= short_len or routes[1] is None
        if is_short != (i == 0):
            return 0, 0
        span = min(W, ctx + length) + min(length, r.rows)
        most = -(-span // r.tile) + 1 + -(-S // r.tile)
        t = min(most, (ctx + length - 1) // r.tile + 1)
        return -(-length // r.rows), (t >> shift) + (shift > 0)

    shift = 0
    while True:
        ws = [work(n, shift) for n in range(N)]
        items, v = sum(w for w, _ in ws), sum(w * t for w, t in ws)
        if v < 2 ** 31 - 1:
            break
        shift += 1
    none = [(1, 0)] * r.cols
    if items > r.cap_items or (guard and items == 0):
        return {}, none
    t_max = max(t for _, t in ws)
    s_rows = max(t * min(seqs[n][1], r.rows) for n, (_, t) in enumerate(ws))
    assert s_rows <= U32
    even, rounds = div(v + r.cols - 1, r.cols), div(items + r.cols - 1, r.cols)
    Q = max(even, r.min_chunk)
    if r.rows_div:
        Q = max(Q, math.ceil(math.sqrt(s_rows / r.rows_div)))
    whole = rounds * t_max <= Q + r.split_cost
    V = v
    if whole:
        Q, V = rounds * t_max, items * t_max
        ws = [(w, t_max if w else 0) for w, _ in ws]
    assert V <= U32 and Q <= U32
    units, ranges = {}, [[None, None] for _ in range(r.cols)]
    v_done = i_done = 0
    for base in range(0, N, NT):
        block = range(base, min(base + NT, N))
        s_item, s_v, s_at = [], [], []
        it, vv = i_done, v_done
        for n in block:
            s_item.append(it)
            s_v.append(vv)
            s_at.append(it + div(vv, Q))
            it += ws[n][0]
            vv += ws[n][0] * ws[n][1]
        find = lambda first, x: max((k for k in range(len(block)) if first[k] <= x), default=0)
        vb, ve, tot_items = v_done, vv, it - i_done
        for c in range(r.cols):
            if c * Q >= V:
                ranges[c] = [1, 0]
                continue
            b, e = c * Q, min(V, c * Q + Q) - 1
            for side, x in enumerate((b, e)):
                if vb <= x < ve:
                    k = find(s_v, x)
                    ranges[c][side] = s_item[k] + div(x - s_v[k], ws[base + k][1])
        end = i_done + tot_items - 1 + div(ve - 1, Q) if tot_items else -1
        for uid in range(s_at[0], end + 1):
            k = find(s_at, uid)
            n = base + k
            ctx, length = seqs[n]
            t2, vs = ws[n][1], s_v[k]
            if t2 == 0:
                continue
            lo, hi = 0, -(-length // r.rows) - 1
            while lo < hi:
                m = (lo + hi + 1) >> 1
                if s_item[k] + m + div(vs + m * t2, Q) <= uid:
                    lo = m
                else:
                    hi = m - 1
            b = vs + lo * t2
            e, c = b + t2 - 1, uid - s_item[k] - lo
            c0, c1 = div(b, Q), div(e, Q)
            if not c0 <= c <= c1:
                continue
            kn = key_tiles(ctx, length, lo * r.rows, r.rows, r.tile, W, S)
            x0, x1 = max(c * Q - b, 0), min(t2, (c + 1) * Q - b)
            first = 2 * c0 + (c0 * Q != b)
            assert uid not in units
            units[uid] = dict(n=n, q0=lo * r.rows, kt=(x0 * kn // t2, x1 * kn // t2), col=c, c0=c0, c1=c1, kn=kn, item=s_item[k] + lo,
                              part=(first if c == c0 else 2 * c) if c0 != c1 else -1)
        v_done, i_done = ve, it
    return units, [tuple(x) for x in ranges]


def check(seqs, H, W, S, max_len, tensor, M=None):
    M = max(1, sum(m for _, m in seqs)) if M is None else M
    routes, short_len = plan(M, len(seqs), H, max_len, tensor)
    seqs = [(c, min(m, max_len)) for c, m in seqs]
    seen = set()
    for i, r in enumerate(routes):
        if r is None:
            continue
        units, ranges = division(routes, short_len, i, seqs, W, S)
        assert all(0 <= u < r.cap_items + r.cols for u in units)
        tiles, parts, counters = {}, set(), {}
        for u in units.values():
            tiles.setdefault((u["n"], u["q0"]), []).append(u)
            if u["part"] >= 0:
                assert u["part"] < 2 * r.cols and u["part"] not in parts
                parts.add(u["part"])
                assert u["c1"] < r.cols and counters.setdefault(u["c1"], (u["n"], u["q0"])) == (u["n"], u["q0"])
        for key, us in tiles.items():
            assert key not in seen
            seen.add(key)
            us.sort(key=lambda u: u["col"])
            assert [u["col"] for u in us] == list(range(us[0]["c0"], us[0]["c1"] + 1))
            # parts after the first are two numbers apart, as the adding code counts them
            assert all(u["part"] == 2 * (us[0]["c0"] + k) for k, u in enumerate(us) if k)
            at = 0
            for u in us:
                assert u["kt"][0] == at and u["kt"][1] >= at
                at = u["kt"][1]
            assert at == us[0]["kn"]
        read = set()
        for c, (lo, hi) in enumerate(ranges):
            for item in range(lo, hi + 1):
                u = units[item + c]
                assert u["col"] == c and u["item"] == item
                read.add(item + c)
        assert read == set(units)
    assert seen == {(n, q0) for n, (c, m) in enumerate(seqs) for r in [routes[0] if routes[1] is None or m <= short_len else routes[1]]
                    for q0 in range(0, m, r.rows)}


@pytest.mark.parametrize("seed", range(40))
def test_division_of_random_batches(seed):
    r = random.Random(seed)
    N = r.choice([1, 2, 9, 60, 255, 256, 257, 300, 600, 900])
    idle, ones, top = r.choice([0, 0.2, 0.9]), r.choice([0, 0.5, 1]), r.choice([1, 3, 16, 17, 300, 2000 if N < 20 else 40])
    far = r.choice([0, 100, 40000, 2 ** 31 - 3000])
    seqs = []
    for _ in range(N):
        m = 1 if r.random() < ones else r.randint(1, top)
        seqs.append((r.randint(0, far), 0 if r.random() < idle else m))
    W, S, H = r.choice([1, 33, 1000, 4096, 2 ** 31 - 1]), r.choice([0, 4, 128]), r.randint(1, 64)
    most = max(m for _, m in seqs)
    for max_len in {max(1, most), 10 ** 6, max(1, most // 2)}:
        for tensor in (True, False):
            check(seqs, H, W, S, max_len, tensor)


@pytest.mark.parametrize("N", [257, 512, 513, 3000])
def test_division_across_blocks_of_sequences(N):
    """Idle runs over the edges of the 256-sequence blocks, whole blocks without a token, both routes."""
    for pattern in (lambda n: 1 if 200 <= n % 256 <= 255 else 0, lambda n: 0 if n < 256 else n % 3, lambda n: (0, 40, 3)[n % 3],
                    lambda n: 300 if n == N - 1 else 0, lambda n: 17 if n % 256 == 0 else 1):
        check([(50 + n % 700, pattern(n)) for n in range(N)], 5, 300, 4, 10 ** 6, True)


def test_a_route_without_work():
    """Only short sequences while the chunks' route is there, and the other way round: nothing is divided by the chunk length
    of 0 that no work has."""
    for seqs in ([(10, 3), (0, 16), (5, 1)], [(10, 40), (0, 17)], [(0, 0)] * 300):
        check(seqs, 4, 100, 4, 10 ** 6, True)
    routes, short_len = plan(20, 3, 4, 20, True)
    with pytest.raises(ZeroDivisionError):
        division(routes, short_len, 1, [(10, 3), (0, 16), (5, 1)], 100, 4, guard=False)


def test_rows_claimed_more_than_once():
    """cu_seqlens that claims more query tiles than there are rows for: nothing is computed."""
    routes, short_len = plan(40, 9, 2, 40, True)
    units, ranges = division(routes, short_len, 1, [(100, 40)] * 9, 60, 4)
    assert routes[1].cap_items == 9 and units  # 9 tiles fit
    routes[1].cap_items = 8
    assert division(routes, short_len, 1, [(100, 40)] * 9, 60, 4) == ({}, [(1, 0)] * routes[1].cols)
