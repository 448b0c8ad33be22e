"""Edges of the SW-SKA operators with first tokens that stay visible, of the paged attention of new tokens and of the page
tables."""
import pytest
import torch

import sliding_window_attention_chunked_b200 as rod
from sliding_window_attention_chunked_b200 import workloads as wl

from . import row_norms as rn
from . import sink_ref as ref
from .test_gpu_sink_paged import DEV, DT, _check_step, _step

pytestmark = pytest.mark.gpu


# ---- rows that see one key --------------------------------------------------------------------------------
ONE_KEY = [  # B, H, T, dk, dv, W, S: every row sees its own key alone
    (2, 3, 1, 64, 128, 5, 3), (1, 1, 1, 128, 128, 1, 0), (3, 2, 1, 16, 16, 1, 128), (1, 2, 300, 16, 32, 1, 0), (2, 1, 130, 32, 128, 1, 0),
    (1, 3, 129, 128, 128, 1, 0), (2, 2, 77, 128, 64, 1, 0), (1, 2, 65, 64, 64, 1, 0), (1, 2, 1000, 128, 16, 1, 0)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,H,T,dk,dv,W,S", ONE_KEY)
def test_gradients_of_rows_that_see_one_key(B, H, T, dk, dv, W, S, dtype):
    """The softmax of one score is 1 whatever the score: dq = dk = 0 exactly, o = v, and dv = dO."""
    q, k, v = wl.swska_inputs(B, H, T, dk, dv, seed=T + dv, dtype=dtype, device=DEV)
    dO = torch.randn(B, H, T, dv, device=DEV).to(DT[dtype])
    got = _step(q, k, v, dO, W, S)
    rod.check()
    assert (got["dq"] == 0).all() and (got["dk"] == 0).all()
    assert torch.equal(got["o"], v)
    _check_step(got, ref.train(q, k, v, dO, W, S), q, k, W, S, what=f"{dtype} T{T}")


@pytest.mark.parametrize("T,dk,dv,W,S", [(40, 64, 128, 30, 2), (200, 128, 128, 70, 0), (333, 32, 64, 333, 5), (70, 16, 32, 9, 128), (150, 32, 128, 20, 1)])
def test_first_row_in_fp32(T, dk, dv, W, S):
    """The first token of every sequence sees itself alone; in fp32 dP and D are the same sums of the same terms, so their
    difference is 0 and not a rounding."""
    q, k, v = wl.swska_inputs(2, 3, T, dk, dv, seed=T, dtype="fp32", device=DEV)
    dO = torch.randn(2, 3, T, dv, device=DEV)
    got = _step(q, k, v, dO, W, S)
    rod.check()
    assert (got["dq"][:, :, 0] == 0).all() and not (got["dq"][:, :, 1:] == 0).all(-1).any()
    _check_step(got, ref.train(q, k, v, dO, W, S), q, k, W, S, what=f"T{T}")


# ---- many sequences -----------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_training_step_of_many_short_sequences(dtype):
    """More than 65535 sequences: the backward takes every batch that the forward takes."""
    B, H, T, d, W, S = 65537, 1, 2, 16, 2, 1
    q, k, v = wl.swska_inputs(B, H, T, d, d, seed=9, dtype=dtype, device=DEV)
    dO = torch.randn(B, H, T, d, device=DEV).to(DT[dtype])
    got = _step(q, k, v, dO, W, S)
    rod.check()
    at = torch.tensor([0, 1, 32768, 65534, 65535, 65536], device=DEV)
    part = lambda x: x[at]
    _check_step({n: part(x) for n, x in got.items()}, ref.train(*map(part, (q, k, v, dO)), W, S), part(q), part(k), W, S, what="many")
    same = _step(*(x[:9000].contiguous() for x in (q, k, v, dO)), W, S)
    assert all(torch.equal(same[n], got[n][:9000]) for n in same)


# ---- page tables: first tokens beyond every page ------------------------------------------------------------
@pytest.mark.parametrize("S", [5 * 64, 10 ** 9, 2 ** 31 - 64, 2 ** 31 - 63, 2 ** 31 - 1])
@pytest.mark.parametrize("ps", [64, 1, 24])
def test_page_tables_keep_all_first_tokens(S, ps):
    """`sinks` past every position keeps every page of a running sequence, however large it is."""
    N, mp, P, W, M = 3, 8, 30, 16, 200
    ctx, new = [5 * ps, 3 * ps + ps // 2, 7 * ps], [ps, 1, -1]
    table, free = [[-1] * mp for _ in range(N)], list(range(P))
    for n in range(N):
        for p in range(-(-ctx[n] // ps)):
            table[n][p] = free.pop()
    top = len(free)
    args = (ctx, new, table, [0] * N, free + [-1] * (P - top), top, ps, W, S, M)
    dev = lambda x, dt=torch.int32: torch.tensor(x, dtype=dt, device=DEV)
    t, f, fl, fc = dev(table), dev([0] * N), dev(args[4]), dev([top])
    cu, slot = rod.swska_page_tables(dev(ctx, torch.int64), dev(new), t, f, fl, fc, ps, W, S, M)
    rod.check()
    for x, y in zip((t.tolist(), f.tolist(), fl.tolist(), int(fc), cu.tolist(), slot.tolist()), ref.page_tables(*args)):
        assert x == (y if isinstance(y, int) else list(y))


@pytest.mark.parametrize("N,M", [(2000, 1700), (16384, 14000)])
def test_page_tables_of_the_most_sequences(N, M):
    """A step of thousands of sequences: a few tokens, one, none, finished ones, and fewer tokens than are wanted."""
    r = torch.Generator().manual_seed(N)
    rand = lambda hi, *s: torch.randint(0, hi, s, generator=r)
    ps, W, S, mp = 16, 40, 4, 6
    ctx = rand(mp * ps - 20, N).tolist()
    new = [(-1, 0, 1, 1, 1, 3)[x] for x in rand(6, N).tolist()]
    free = torch.randperm(6 * N, generator=r).tolist()
    table = [[free.pop() if p * ps < c and (p == 0 or (p + 1) * ps > c - W) else -1 for p in range(mp)] for c in ctx]
    top = len(free) // 60
    args = (ctx, new, table, [0] * N, free[:top] + [-1] * (6 * N - top), top, ps, W, S, M)
    dev = lambda x, dt=torch.int32: torch.tensor(x, dtype=dt, device=DEV)
    t, f, fl, fc = dev(table), dev([0] * N), dev(args[4]), dev([top])
    cu, slot = rod.swska_page_tables(dev(ctx, torch.int64), dev(new), t, f, fl, fc, ps, W, S, M)
    rod.check()
    want = ref.page_tables(*args)
    assert 0 < want[4][-1] < sum(max(x, 0) for x in new)
    for x, y in zip((t.tolist(), f.tolist(), fl.tolist(), int(fc), cu.tolist(), slot.tolist()), want):
        assert x == (y if isinstance(y, int) else list(y))


def test_page_tables_largest_slot_map():
    """A slot map of 2^31 - 1 tokens is filled to its end and no further."""
    M, i32 = 2 ** 31 - 1, lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    buf = torch.full((M + 5,), 7, dtype=torch.int32, device=DEV)
    table, free, count = torch.full((1, 4), -1, dtype=torch.int32, device=DEV), i32(3, 1, 0, 2), i32(4)
    cu, slot = rod.swska_page_tables(torch.zeros(1, dtype=torch.int64, device=DEV), i32(20), table, i32(0), free, count, 16, 8, 0, M, slot_map=buf[:M])
    rod.check()
    assert cu.tolist() == [0, 20] and slot[:20].tolist() == [*range(32, 48), *range(0, 4)]
    assert (buf[M:] == 7).all()
    # everything past the tokens is -1 (in pieces: a comparison of the whole takes as much memory again)
    assert all(int((x != -1).sum()) == 0 for x in slot[20:].split(2 ** 28))


# ---- paged attention: many sequences, routes without work --------------------------------------------------------
def _paged(b, **kw):
    args, o = b.args(DEV), b.o.to(DEV)
    rod.swska_extend_paged(*args, b.W, sinks=b.S, o=o, **kw)
    return o, args


def _check_paged(b, what, **kw):
    """Rows, the padding behind them and the cache against the 64-bit reference."""
    o, args = _paged(b, **kw)
    rod.check()
    r, ra, kr, vr = b.reference()
    ref.check(o.cpu(), r, ra, b.terms(), b.dk, ref.amp(b.q, torch.nan_to_num(b.k_pool)), what)
    rows = int(b.cu[-1])
    assert torch.equal(o[rows:].cpu(), b.o[rows:]), f"{what}: padding"
    for x, y in ((args[3], kr), (args[4], vr)):
        assert torch.equal(torch.nan_to_num(x.float().cpu(), 1234.5), torch.nan_to_num(y.float(), 1234.5)), f"{what}: cache"


@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 128, 128), ("fp32", 16, 32)])
@pytest.mark.parametrize("N,pattern", [(257, "ends"), (600, "idle block"), (513, "mixed"), (1030, "last"), (300, "none long")])
def test_extend_many_sequences(N, pattern, dtype, dk, dv):
    """More sequences than the 256 that are divided at a time: idle runs over the edges of such blocks, a block without a token,
    short and long sequences side by side."""
    lens = {"ends": lambda n: 1 if 200 <= n % 256 else 0, "idle block": lambda n: 0 if n < 256 else n % 3, "mixed": lambda n: (0, 20, 3)[n % 3],
            "last": lambda n: 60 if n == N - 1 else 0, "none long": lambda n: 1 + n % 2}[pattern]
    b = ref.Batch(dtype, 2, dk, dv, 40, 4, 16, [(37 * n) % 90 for n in range(N)], [lens(n) for n in range(N)], pad=3, seed=N)
    _check_paged(b, f"{N} {pattern}")
    _check_paged(b, f"{N} {pattern} bounded", max_len=b.max_len)


@pytest.mark.parametrize("lens", [[3, 16, 1, 0], [40, 0, 17], [0, 0, 0]])
def test_extend_a_route_without_work(lens):
    """The bound on the lengths allows both kernels, the lengths give one of them nothing (or neither anything)."""
    b = ref.Batch("bf16", 5, 128, 128, 70, 4, 24, [100, 7, 300, 0][:len(lens)], lens, pad=25, seed=sum(lens))
    _check_paged(b, f"{lens}")
    _check_paged(b, f"{lens} bounded", max_len=40)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_extend_missing_pages_and_rows_behind(dtype):
    """Pages that the table lacks are left out, the rows of the sequences around them are right, the padding keeps what it holds."""
    b = ref.Batch(dtype, 3, 128, 128, 60, 4, 16, [100, 40, 0, 20], [1, 20, 5, 2], pad=4, seed=1)
    b.table[1, 1], b.table[0, 0] = -1, b.P
    b.k_pool.nan_to_num_(0.5)
    b.v_pool.nan_to_num_(0.25)
    _check_paged(b, "missing")


def test_extend_bound_of_zero_is_no_bound():
    """max_len = 0 stands for M, as at the C entry: the new tokens are written and attended to."""
    b = ref.Batch("bf16", 3, 128, 128, 60, 4, 16, [100, 3], [2, 20], pad=3, seed=8)
    _check_paged(b, "max_len 0", max_len=0)
    none = ref.Batch("bf16", 3, 128, 128, 60, 4, 16, [100, 3], [0, 0], pad=2, seed=8)
    _check_paged(none, "no tokens", max_len=0)
    args = none.args(DEV)
    assert rod.swska_extend_paged(args[0][:0], *(a[:0] for a in args[1:3]), *args[3:6], args[6][:0], *args[7:], 60, max_len=0).shape == (0, 3, 128)


@pytest.mark.parametrize("dtype,bound", [("bf16", 1), ("bf16", None), ("fp32", 1)])
def test_extend_the_most_sequences(dtype, bound):
    """16384 sequences of one token, each in a page of its own; every third one idle."""
    N, H, d, ps = 16384, 2, 128, 8
    g = torch.Generator(DEV).manual_seed(3)
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g).to(DT[dtype])
    n = torch.arange(N, device=DEV)
    ctx, lens = (n * 5) % ps, (n % 3 != 2).to(torch.int32)
    table = torch.randperm(N, device=DEV, generator=g).to(torch.int32)[:, None]
    cu = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32)
    who = n[lens == 1]
    M, page = len(who), table[who, 0]
    slot = page * ps + ctx[who].to(torch.int32)
    kp, vp, q, kn, vn = rnd(N, ps, d), rnd(N, H, ps, d), rnd(M, H, d), rnd(M, d), rnd(M, H, d)
    o = rod.swska_extend_paged(q, kn, vn, kp, vp, table, slot, cu, ctx, 5, sinks=1, max_len=bound)
    rod.check()
    assert torch.equal(kp[page.long(), ctx[who]], kn) and torch.equal(vp[page.long(), :, ctx[who]], vn)
    j = torch.arange(ps, device=DEV)
    see = (j <= ctx[who, None]) & ((j > ctx[who, None] - 5) | (j < 1))
    K, V = kp[page.long()].double(), vp[page.long()].double()
    s = torch.where(see[:, None], torch.einsum("mhd,mjd->mhj", q.double(), K) * d ** -0.5, -torch.inf)
    p = torch.softmax(s, -1)
    ref.check(o, torch.einsum("mhj,mhjd->mhd", p, V), torch.einsum("mhj,mhjd->mhd", p, V.abs()), 6, d, ref.amp(q, kp), f"most {dtype}")


# ---- wide windows, row by row ---------------------------------------------------------------------------------
WIDE = [("bf16", 128, 5000, 4096, 4), ("bf16", 128, 4800, 4096, 0), ("bf16", 64, 4500, 3000, 5), ("fp32", 64, 4500, 4000, 4), ("fp32", 128, 4300, 4096, 1)]


@pytest.mark.parametrize("dtype,d,T,W,S", WIDE)
def test_training_step_rows_of_a_wide_window(dtype, d, T, W, S):
    """Flat attention over thousands of keys, each row's error by its norm (row_norms.py): a lost or an extra key shows."""
    H = 2
    q, k, v = wl.swska_inputs(1, H, T, d, d, seed=T + d, dtype="fp32", device=DEV)
    dO = torch.randn(1, H, T, d, device=DEV, generator=torch.Generator(DEV).manual_seed(T))
    q, k, v, dO = ((0.1 * x if n == "q" else x).to(DT[dtype]) for n, x in (("q", q / q.std()), ("k", k / k.std()), ("v", v), ("dO", dO)))
    got = _step(q, k, v, dO, W, S)
    rod.check()
    t = torch.arange(T, device=DEV)
    see, a = ref.visible(t, t, W, S), ref.amp(q, k)
    dk, dk_tol = 0, 0
    many = slice(300, None)  # rows that see hundreds of keys; keys that hundreds of queries see are those before T - 300
    seen = slice(None, T - 300)
    for h in range(H):
        want = rn.gradients(*(x.double() for x in (q[0, h], k[0], v[0, h], dO[0, h])), see, d ** -0.5, DT[dtype], a)
        for name, rows in (("o", many), ("dq", many), ("dv", seen)):
            bad = rn.off(got[name][0, h][rows], want[name][0][rows], want[name][1][rows])
            assert not bad.any(), f"{name} head {h}: {int(bad.sum())} rows, first {bad.nonzero()[0].tolist()}"
        dk, dk_tol = dk + want["dk"][0], dk_tol + want["dk"][1]
    assert not rn.off(got["dk"][0][seen], dk[seen], dk_tol[seen]).any()


@pytest.mark.parametrize("dtype,lens", [("bf16", [1, 1, 1, 1]), ("bf16", [5, 1, 16, 2]), ("bf16", [200, 30, 129, 1]), ("fp32", [1, 20, 3, 70])])
def test_extend_rows_of_a_wide_window(dtype, lens):
    """The paged form: every kernel, W 4096, each row's error by its norm."""
    H, W, S, ps, d = 3, 4096, 4, 64, 128
    b = ref.Batch(dtype, H, d, d, W, S, ps, [4100, 9000, 4500, 6001], lens, seed=sum(lens))
    b.q = (0.05 * b.q.float()).to(DT[dtype])  # made with spread 2
    o, args = _paged(b, max_len=b.max_len)
    rod.check()
    kp, vp, a = args[3], args[4], ref.amp(b.q, torch.nan_to_num(b.k_pool))
    for n, (c, m) in enumerate(zip(b.ctx.tolist(), lens)):
        pos = torch.arange(c, c + m)
        j = torch.cat([torch.arange(S), torch.arange(c - W + 1, c + m)])
        pg = b.table[n, j // ps].long()
        K, V = kp[pg, j % ps].double(), vp[pg, :, j % ps].double()
        r0 = int(b.cu[n])
        for h in range(H):
            want, tol = rn.forward(args[0][r0:r0 + m, h].double(), K, V[:, h], ref.visible(pos, j, W, S).to(DEV), d ** -0.5, DT[dtype], a)
            bad = rn.off(o[r0:r0 + m, h], want, tol)
            assert not bad.any(), f"sequence {n} head {h}: {int(bad.sum())} rows"


# ---- gradients where the first tokens draw attention ------------------------------------------------------------
@pytest.mark.parametrize("B,H,T,d,W,S", [(2, 2, 1500, 64, 300, 8), (1, 2, 1999, 128, 500, 13), (1, 2, 900, 128, 700, 60), (1, 2, 1200, 64, 90, 128),
                                         (2, 2, 700, 32, 100, 100), (1, 2, 1000, 128, 200, 128), (1, 3, 127, 128, 40, 20)])
def test_query_gradients_where_the_first_tokens_draw_attention(B, H, T, d, W, S):
    """The first tokens' keys share a direction that draws the queries to them. sum_j dS_j = 0, so that direction cancels in dq =
    sum_j dS_j k_j, and roundings of those dS would be left of it. Held by the norm of the whole dq: its own rounding and those of the dS of
    the other keys, each at most 2^-8 / sqrt(3) of its term on average (row_norms.py), D from the rounded o for those keys, and 2^-13
    (the cubic of the exponentials) of the first tokens' terms. Rounding their dS too would be 2.5e-3 to 2.8e-3 of |dq|."""
    g = torch.Generator(DEV).manual_seed(T + d)
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g)
    u = rnd(d)
    u /= u.norm()
    q, k = rnd(B, H, T, d) + 4 * u, rnd(B, T, d)
    k[:, :S] += 8 * u
    q, k, v, dO = (x.bfloat16() for x in (q, k, rnd(B, H, T, d), rnd(B, H, T, d)))
    got = _step(q, k, v, dO, W, S)
    rod.check()
    t = torch.arange(T, device=DEV)
    see, scale = ref.visible(t, t, W, S), d ** -0.5
    err = size = terms = first = err_D = 0.0
    for b in range(B):
        for h in range(H):
            Q, K, V, G = (x.double() for x in (q[b, h], k[b], v[b, h], dO[b, h]))
            o, _, p, _ = ref.attend(Q, K, V, see, scale)
            D = (G * o).sum(1, keepdim=True)
            dS = p * (G @ V.T - D) * scale
            dq, k2 = dS @ K, (K * K).sum(1)
            err += float(((got["dq"][b, h].double() - dq) ** 2).sum())
            size += float((dq * dq).sum())
            terms += float((dS[:, S:] ** 2 @ k2[S:]).sum())
            first += float((dS[:, :S] ** 2 @ k2[:S]).sum())
            rest = ((p[:, S:] @ K[S:]) ** 2).sum(1)
            err_D += float((((G * o) ** 2).sum(1) * rest).sum()) * scale ** 2
    step = 2.0 ** -8 / 3 ** 0.5
    tol = step * (size + terms + err_D) ** 0.5 * 1.01 + 2.0 ** -13 * first ** 0.5
    assert err ** 0.5 <= tol, f"{(err / size) ** 0.5:.2e} of |dq|, allowed {tol / size ** 0.5:.2e}"


@pytest.mark.parametrize("T,dk,dv,W,S", [(2, 16, 16, 36, 1), (2, 32, 128, 1, 1), (5, 16, 16, 153, 1), (33, 64, 64, 40, 2), (64, 128, 128, 64, 1), (60, 32, 64, 9, 0)])
def test_fp32_gradients_where_attention_is_peaked_in_one_tile(T, dk, dv, W, S):
    """fp32 rows whose keys lie in one key tile and that give one of them nearly everything: dS = p (dP - D) is a small difference of
    large sums. An error of D is taken out (sum_j dS_j = 0 as computed), which leaves, with A_j = |dO| . |v_j| and u = 2^-23 for 32 bits:
    the relative errors of p and dP - D, and those of the dP_j, d u A_j, which enter dS_j as p_j (err_j - sum_k p_k err_k) and so only with
    the weights of the others, (1 - p_j) A_j + sum_{k != j} p_k A_k; the sum e of the differences, rounded to 4 u of its terms; and the
    roundings of dP and D in the 64-bit reference, dv 2^-52 of A_j and of sum_k p_k A_k (a row that sees one key has nothing else)."""
    B, H = 2, 3
    q, k, v = wl.swska_inputs(B, H, T, dk, dv, seed=T + dk, dtype="fp32", device=DEV)
    g = torch.Generator(DEV).manual_seed(T)
    dO, w = torch.randn(B, H, T, dv, device=DEV, generator=g), torch.randn(dk, device=DEV, generator=g)
    w /= w.norm()
    q = q + dk ** 0.5 * w
    k[:, ::max(W, 2) if S == 0 else T] += 11 * w
    got = _step(q, k, v, dO, W, S)
    rod.check()
    t = torch.arange(T, device=DEV)
    see, scale, u = ref.visible(t, t, W, S), dk ** -0.5, 2.0 ** -23
    inner = (T + dk + dv) * u * (1 + ref.amp(q, k)) + 2.0 ** -20
    dk_want, dk_tol, peaked = torch.zeros_like(k, dtype=torch.float64), torch.zeros_like(k, dtype=torch.float64), 0
    for b in range(B):
        for h in range(H):
            Q, K, V, G = (x.double() for x in (q[b, h], k[b], v[b, h], dO[b, h]))
            o, _, p, _ = ref.attend(Q, K, V, see, scale)
            dP = G @ V.T - (G * o).sum(1, keepdim=True)
            A, a = G.abs() @ V.abs().T, (p * dP.abs()).sum(1, keepdim=True)
            err = inner * p * (dP.abs() + a) + dv * u * p * ((1 - p) * A + (p * A).sum(1, keepdim=True) - p * A) + 4 * u * p * a
            err = err + dv * 2.0 ** -52 * p * (A + (p * A).sum(1, keepdim=True))
            want, tol = (p * dP) @ K * scale, err @ K.abs() * scale
            bad = (got["dq"][b, h].double() - want).abs() > tol + u * want.abs() + 1e-30
            assert not bad.any(), f"dq {b} {h}: {int(bad.sum())} off at {bad.nonzero()[0].tolist()}"
            dk_want[b] += (p * dP).T @ Q * scale
            dk_tol[b] += err.T @ Q.abs() * scale
            peaked += int(((p.max(1).values > 0.99) & (see.sum(1) > 1)).sum())
    bad = (got["dk"].double() - dk_want).abs() > dk_tol + H * u * dk_want.abs() + 1e-30
    assert not bad.any(), f"dk: {int(bad.sum())} off at {bad.nonzero()[0].tolist()}"
    assert peaked > 0


# ---- a stream given by the caller -----------------------------------------------------------------------------
def _late(stream, ms=20):
    """Work that keeps a stream busy for some milliseconds, so that a call on it has not begun when it returns."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(int(ms * 1.5e6))


def _overwrite(sizes):
    """Blocks of these sizes on the current stream, as any later work there may take them, filled with NaN bits."""
    return [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]


def test_training_step_on_a_stream_keeps_its_workspace():
    """Without a workspace the call takes one from the stream it runs on: work that the current stream starts after the call
    has returned does not get that block, nor that of an output which the caller has dropped."""
    B, H, T, W, S = 1, 4, 1500, 300, 4
    q, k, v = wl.swska_inputs(B, H, T, 128, 128, seed=31, device=DEV)
    dO = torch.randn_like(v)
    want = _step(q, k, v, dO, W, S)
    n = rod.load_library().rod_swska_sink_backward_workspace_size(B, H, T, 128, 128, W, S)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        _late(side)
        got = _step(q, k, v, dO, W, S, stream=side)
        _overwrite([n, n // 2, v.numel() * 2, q.numel() * 2, k.numel() * 2, B * H * T * 4])
        torch.cuda.synchronize()
        assert all(torch.equal(got[x], want[x]) for x in got)
    o, lse = rod.swska_prefill_lse(q, k, v, W)
    old = rod.swska_backward_lse(q, k, v, o, lse, dO, W)
    n = rod.load_library().rod_swska_backward_workspace_size(B, H, T)
    torch.cuda.synchronize()
    _late(side)
    got = rod.swska_backward_lse(q, k, v, o, lse, dO, W, stream=side)
    _overwrite([n, n // 2, v.numel() * 2])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, old))


def test_extend_on_two_streams_with_workspaces_of_their_own():
    """Two calls at once on two streams, each without a workspace, and work on the current stream behind them."""
    a = ref.Batch("bf16", 6, 128, 128, 200, 4, 16, [50, 700, 0, 333], [1, 300, 2, 90], seed=1)
    b = ref.Batch("bf16", 6, 128, 128, 200, 4, 16, [500, 70, 9, 33], [200, 1, 0, 16], seed=2)
    batches = []
    for x in (a, b):
        args = x.args(DEV)
        o = x.o.to(DEV)
        rod.swska_extend_paged(*args, x.W, sinks=x.S, o=o)
        n = rod.load_library().rod_swska_extend_paged_workspace_size(x.q.shape[0], len(x.ctx), x.H, 128, 128, x.q.shape[0], rod.ROD_BF16)
        batches.append((x, args, o, n, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        outs = []
        for x, args, o, n, s in batches:
            _late(s)
            outs.append(rod.swska_extend_paged(*args, x.W, sinks=x.S, stream=s))
        _overwrite([n for _, _, _, n, _ in batches] + [o.numel() * 2 for _, _, o, _, _ in batches])
        torch.cuda.synchronize()
        rod.check()
        for (x, args, o, n, s), got in zip(batches, outs):
            assert torch.equal(got, o)
