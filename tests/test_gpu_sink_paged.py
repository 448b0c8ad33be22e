"""SW-SKA with first tokens that stay visible, the paged attention of new tokens and the page tables on the GPU, against
the 64-bit references of sink_ref.py with the tolerances counted there."""
import math

import numpy as np
import pytest
import torch

import sliding_window_attention_chunked_b200 as rod
from sliding_window_attention_chunked_b200 import workloads as wl

from . import sink_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _step(q, k, v, dO, W, S, **kw):
    o, lse = rod.swska_sink_prefill(q, k, v, W, S, **kw)
    return dict(zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *rod.swska_sink_backward(q, k, v, o, lse, dO, W, S, **kw))))


def _check_step(got, r, q, k, W, S, scale=None, what=""):
    T, d, H = q.shape[2], q.shape[3], q.shape[1]
    a = ref.amp(q, k, scale)
    seen = min(W + S, T)
    for name in ("o", "dq"):
        ref.check(got[name], *r[name], seen, d, a, f"{what} {name}")
    # the key side sums over every query that sees the key (all of them for the first tokens), dk over the heads too
    ref.check(got["dv"], *r["dv"], T, d, a, f"{what} dv")
    ref.check(got["dk"], *r["dk"], T * H, d, a, f"{what} dk")
    # the log-sum-exp: a score's error and a sum of terms in fp32 (absolute), and one rounding of the result
    lse = r["lse"][0]
    tol = (seen + d) * 2.0 ** -23 * (1 + a) + 2.0 ** -12 * (q.dtype == torch.bfloat16) + 2.0 ** -21 + 2.0 ** -23 * lse.abs()
    assert ((got["lse"].double() - lse).abs() <= tol).all(), f"{what} lse"


SMALL = [  # B, H, T, dk, dv, W, S
    (1, 1, 1, 128, 128, 1, 0), (1, 2, 2, 16, 32, 1, 1), (2, 3, 63, 64, 64, 7, 5), (1, 2, 65, 128, 64, 64, 1),
    (1, 5, 127, 128, 128, 30, 4), (2, 2, 128, 128, 128, 1, 3), (1, 3, 129, 128, 128, 1000, 128), (2, 3, 300, 128, 128, 40, 64),
    (1, 2, 513, 128, 128, 128, 65), (1, 4, 700, 128, 128, 129, 128), (1, 1, 1300, 128, 128, 100, 1), (3, 2, 200, 32, 16, 50, 128),
    (1, 2, 400, 16, 128, 3, 0), (1, 2, 390, 64, 128, 65, 70), (1, 3, 640, 128, 128, 500, 127), (1, 2, 1030, 128, 128, 2, 0)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,H,T,dk,dv,W,S", SMALL)
def test_training_step(B, H, T, dk, dv, W, S, dtype):
    q, k, v = wl.swska_inputs(B, H, T, dk, dv, seed=T + W, dtype=dtype, device=DEV)
    dO = torch.randn(B, H, T, dv, device=DEV).to(DT[dtype])
    got = _step(q, k, v, dO, W, S)
    rod.check()
    _check_step(got, ref.train(q, k, v, dO, W, S), q, k, W, S, what=f"{dtype} T{T} W{W} S{S}")


@pytest.mark.parametrize("B,H,T,W,S", [(3, 11, 300, 100, 5), (1, 40, 260, 129, 128), (17, 1, 500, 64, 2), (2, 16, 129, 200, 0), (9, 7, 130, 1, 1)])
def test_training_step_many_heads(B, H, T, W, S):
    """More (sequence, head) pairs than the 16 that go side by side, and a last set that is not full."""
    q, k, v = wl.swska_inputs(B, H, T, 128, 128, seed=T + H, dtype="bf16", device=DEV)
    dO = torch.randn_like(v)
    got = _step(q, k, v, dO, W, S)
    rod.check()
    _check_step(got, ref.train(q, k, v, dO, W, S), q, k, W, S, what=f"B{B} H{H} T{T}")


@pytest.mark.parametrize("dtype,T,W,S", [("bf16", 5000, 300, 4), ("bf16", 4100, 4096, 128), ("fp32", 1700, 90, 100), ("bf16", 20000, 64, 2)])
def test_training_step_long(dtype, T, W, S):
    """Many far segments of the first tokens, and a window that ends just before the sequence does."""
    q, k, v = wl.swska_inputs(1, 1, T, 128, 128, seed=T, dtype=dtype, device=DEV)
    dO = torch.randn_like(v)
    got = _step(q, k, v, dO, W, S)
    rod.check()
    _check_step(got, ref.train(q, k, v, dO, W, S), q, k, W, S, what=f"long {dtype} T{T}")


@pytest.mark.parametrize("dtype,d,T,W,S,where", [("bf16", 128, 900, 300, 4, "first"), ("bf16", 128, 900, 300, 0, "window"), ("bf16", 128, 400, 1, 1, "first"),
                                                 ("bf16", 64, 500, 100, 2, "first"), ("bf16", 32, 300, 90, 0, "window"), ("fp32", 64, 300, 90, 3, "first")])
def test_gradients_where_attention_is_peaked(dtype, d, T, W, S, where):
    """Rows that give one key nearly everything (a first token, or one in the window): dS = p (dP - D) is a small
    difference there, so dq is held to the roundings of dS itself, with no allowance for an error of D beyond that of the
    exponentials (2^-13 each): tolerance H |dq| + (2^-8 + 2^-13) sum p |dP - D| |k| scale + 2^-12 (sum p |dP - D|) (sum p |k|) scale, and
    D's own sums in fp32, d 2^-22 (sum p |dO| |v|) (sum p |k|) scale. The tcgen05 kernel takes D from the rounded o (off by 2^-8 of
    |dO| |o|) for the keys other than the peak: 2^-8 (|dO| |o|) (sum of p |k| without the largest p) scale more."""
    H = 2
    q, k, v = wl.swska_inputs(1, H, T, d, d, seed=T, dtype=dtype, device=DEV)
    torch.manual_seed(T + W)
    u = torch.randn(d, device=DEV)
    u /= u.norm()
    at = torch.arange(T, device=DEV) % (T if where == "first" else W) == (0 if where == "first" else 7)
    q = (q.float() + math.sqrt(d) * u).to(DT[dtype])
    k = torch.where(at[None, :, None], k.float() + 11 * u, k.float()).to(DT[dtype])
    dO = torch.randn_like(v)
    got = _step(q, k, v, dO, W, S)
    rod.check()
    t = torch.arange(T, device=DEV)
    see, scale, half = ref.visible(t, t, W, S), d ** -0.5, torch.finfo(DT[dtype]).eps / 2
    peaked = 0
    for h in range(H):
        Q, K, V, G = q[0, h].double(), k[0].double(), v[0, h].double(), dO[0, h].double()
        o, _, p, _ = ref.attend(Q, K, V, see, scale)
        dP = G @ V.T - (G * o).sum(1, keepdim=True)
        want, a = (p * dP) @ K * scale, (p * dP.abs())
        inner = (T + d) * 2.0 ** -23 * (1 + ref.amp(q, k)) + (2.0 ** -8 + 2.0 ** -13) * (dtype == "bf16")
        tol = half * want.abs() * 1.01 + inner * (a @ K.abs()) * scale + (2.0 ** -12 if dtype == "bf16" else 2.0 ** -15) * a.sum(1, keepdim=True) * (p @ K.abs()) * scale + 1e-30
        # D itself, the difference dP - D and the sums they come from are fp32: that error adds to the roundings of dS (a row that
        # sees one key has dq = 0, and all that stands there is this)
        tol += (d * 2.0 ** -22) * (G.abs() @ V.abs().T * p).sum(1, keepdim=True) * (p @ K.abs()) * scale
        if dtype == "bf16" and d == 128:
            rest = torch.where(p == p.max(1, keepdim=True).values, 0, p)
            tol += 2.0 ** -8 * (G * o).abs().sum(1, keepdim=True) * (rest @ K.abs()) * scale
        bad = (got["dq"][0, h].double() - want).abs() > tol
        assert not bad.any(), f"head {h}: {int(bad.sum())} off at {bad.nonzero()[0].tolist()}"
        peaked += int((p.max(1).values > 0.9).sum())
    assert peaked > T // 4


def test_training_step_scale_graph_and_streams():
    """An explicit scale; the step captured in a graph and replayed on new inputs equals the eager step bit for bit; so does
    one on a side stream, and a repeated one (no order of additions depends on timing)."""
    B, H, T, W, S = 1, 3, 600, 100, 4
    mk = lambda s: [*wl.swska_inputs(B, H, T, 128, 128, seed=s, device=DEV), torch.randn(B, H, T, 128, device=DEV).bfloat16()]
    a, b = mk(1), mk(2)
    eager = {}
    for name, x in (("a", a), ("b", b)):
        eager[name] = _step(*x, W, S, scale=0.3)
        _check_step(eager[name], ref.train(*x, W, S, scale=0.3), x[0], x[1], W, S, scale=0.3, what="scale")
    again = _step(*a, W, S, scale=0.3)
    assert all(torch.equal(again[n], eager["a"][n]) for n in again)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = _step(*a, W, S, scale=0.3, stream=side)
    side.synchronize()
    assert all(torch.equal(on_side[n], eager["a"][n]) for n in on_side)
    buf = [t.clone() for t in a]
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = _step(*buf, W, S, scale=0.3)
    for name, x in (("b", b), ("a", a)):
        for t, n in zip(buf, x):
            t.copy_(n)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], eager[name][n]) for n in out)
    rod.check()


def test_training_step_zero_first_tokens_is_the_window():
    q, k, v = wl.swska_inputs(2, 4, 500, 128, 128, seed=5, device=DEV)
    o, lse = rod.swska_sink_prefill(q, k, v, 90, 0)
    o2, lse2 = rod.swska_prefill_lse(q, k, v, 90)
    rod.check()
    see = ref.train(q, k, v, torch.zeros_like(v), 90, 0)
    for x, l in ((o, lse), (o2, lse2)):
        ref.check(x, *see["o"], 90, 128, ref.amp(q, k), "o")
        assert (l.double() - see["lse"][0]).abs().max() < 1e-3


# ---- paged attention of new tokens ----------------------------------------------------------------------
def _run(b, **kw):
    args = b.args(DEV)
    o = b.o.to(DEV)
    rod.swska_extend_paged(*args, b.W, sinks=b.S, o=o, **kw)
    return o, args[3], args[4]


def _check_run(b, got, what, **kw):
    o, kp, vp = got
    r, ra, kr, vr = b.reference(**kw)
    ref.check(o.cpu(), r, ra, b.terms(), b.dk, ref.amp(b.q, torch.nan_to_num(b.k_pool)), what)
    for x, y in ((kp, kr), (vp, vr)):
        assert torch.equal(torch.nan_to_num(x.float().cpu(), 1234.5), torch.nan_to_num(y.float(), 1234.5)), f"{what}: cache"


CASES = [  # H, W, S, page, ctx, lens, pad
    (1, 1, 0, 8, [0], [1], 0),
    (16, 100, 4, 16, [0, 5, 99, 100, 333], [1, 1, 1, 1, 1], 3),
    (5, 64, 3, 24, [0, 7, 200, 64, 1000], [3, 16, 0, 1, 12], 5),
    (3, 50, 128, 8, [300, 0, 127, 128], [1, 2, 5, 16], 0),
    (2, 200, 5, 64, [0, 10, 500], [17, 130, 260], 7),
    (4, 1000, 4, 40, [0, 129, 0], [300, 128, 0], 0),
    (16, 33, 1, 8, [77], [129], 1),
    (7, 4096, 4, 128, [0, 4000], [400, 250], 0),
    (10, 300, 20, 200, [450, 0, 900, 30], [1, 40, 0, 513], 9),
    (1, 130, 128, 256, [1000, 20], [70, 1], 0),
    (64, 40, 2, 16, [90, 3], [1, 20], 2),
    (9, 700, 7, 8, [5000, 64, 63, 65, 128, 2], [1, 1, 2, 3, 4, 5], 0)]


@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 128, 128), ("fp32", 128, 128), ("fp32", 16, 64), ("bf16", 64, 32)])
@pytest.mark.parametrize("H,W,S,page,ctx,lens,pad", CASES)
def test_extend(H, W, S, page, ctx, lens, pad, dtype, dk, dv):
    b = ref.Batch(dtype, H, dk, dv, W, S, page, ctx, lens, pad=pad, seed=H + W)
    got = _run(b, max_len=b.max_len)
    rod.check()
    _check_run(b, got, f"{dtype} {dk} H{H} W{W}")
    if H <= 16:  # without the bound on the lengths the other kernels may run
        _check_run(b, _run(b), f"{dtype} {dk} H{H} W{W} no max_len")


@pytest.mark.parametrize("lens", [[2], [3], [4], [5], [8], [9], [15], [16], [16, 1, 2], [7, 0, 13]])
def test_extend_few_tokens_over_a_long_window(lens):
    """Few rows over many keys: every tile is cut, and rows of two, four, eight and more are added together."""
    b = ref.Batch("bf16", 5, 128, 128, 2500, 4, 64, [2600 + 900 * i for i in range(len(lens))], lens, pad=2, seed=sum(lens))
    got = _run(b, max_len=b.max_len)
    rod.check()
    _check_run(b, got, f"few {lens}")
    again = _run(b, max_len=16)[0]
    assert torch.equal(_run(b, max_len=16)[0].view(torch.int16), again.view(torch.int16))  # no order depends on timing


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_extend_hostile_tables(dtype):
    """Entries and slots outside the pool, positions past the table, bad ctx, a bound below a length: nothing outside is
    touched, what is missing is left out, a row that sees no key is 0 and one at an impossible position NaN."""
    b = ref.Batch(dtype, 3, 128, 128, 60, 4, 16, [100, 40, 30, 50, 20, 0], [1, 20, 3, 2, 4, 5], pad=2, seed=1)
    b.table[0, 5], b.table[1, 0], b.table[2, :] = b.P, -7, 2 ** 31 - 1
    b.slot[2], b.slot[5], b.slot[6] = -5, b.P * b.ps, 2 ** 31 - 1
    b.ctx[3], b.ctx[4] = -1, 2 ** 31 - 2
    b.table[5, 0] = -1
    # keys whose slot was not written hold NaN: give those rows numbers, the reference reads them too
    b.k_pool.nan_to_num_(0.5)
    b.v_pool.nan_to_num_(0.25)
    got = _run(b, max_len=7)
    rod.check()
    _check_run(b, got, "hostile", max_len=7)
    assert torch.isnan(got[0][24:26].float()).all() and (got[0][21:24] == 0).all() and (got[0][30:] != got[0][30:] + 1).all()


def test_extend_bad_cumulative_lengths_stay_inside():
    """cu_seqlens that fall, start late or run past M are cut to the rows there are."""
    b = ref.Batch("bf16", 2, 128, 128, 60, 4, 16, [100, 40, 30], [3, 20, 3], seed=2)
    keep = b.o.clone()
    b.cu = torch.tensor([-9, 3, 2, 1000], dtype=torch.int32)
    o, _, _ = _run(b)
    rod.check()
    # rows 0 .. 2 are sequence 0's, rows 2 .. 25 sequence 2's (3, 2 is empty, 1000 is cut to M = 26): row 2 is either's
    assert o.shape == keep.shape and torch.isfinite(o.float()[:2]).all()


def test_extend_overlapping_sequences_stay_inside():
    """cu_seqlens that claims the same rows many times over asks for more query tiles than the workspace holds: nothing is
    written out of place (the rows are left as they are), and the next call is right."""
    b = ref.Batch("bf16", 2, 128, 128, 60, 4, 16, [100] * 9, [40] + [0] * 8, seed=6)
    args = b.args(DEV)
    cu = torch.tensor([0, 40] * 5, dtype=torch.int32, device=DEV)
    o = b.o.to(DEV)
    work = torch.zeros(rod.load_library().rod_swska_extend_paged_workspace_size(40, 9, 2, 128, 128, 40, 1) + 4096, dtype=torch.uint8, device=DEV)
    rod.swska_extend_paged(args[0], None, None, args[3], args[4], args[5], None, cu, args[8], 60, sinks=4, o=o, workspace=work[:-4096])
    rod.check()
    assert int(work[-4096:].sum()) == 0
    _check_run(b, _run(b), "after")


def test_extend_reads_only_and_negative_zero_lengths():
    """Without new keys and values the cache is read as it is; a batch without tokens does nothing."""
    b = ref.Batch("bf16", 4, 128, 128, 100, 4, 32, [300, 20], [5, 30], seed=3)
    o1, kp, vp = _run(b, max_len=30)
    args = b.args(DEV)
    o2 = rod.swska_extend_paged(args[0], None, None, kp, vp, args[5], None, args[7], args[8], b.W, sinks=b.S, max_len=30)
    rod.check()
    assert torch.equal(o1[:35], o2[:35])
    zero = torch.zeros(3, dtype=torch.int32, device=DEV)
    o3 = rod.swska_extend_paged(*args[:3], kp, vp, args[5], torch.full_like(args[6], -1), zero, args[8], b.W, o=b.o.to(DEV))
    rod.check()
    assert torch.equal(o3.cpu(), b.o)


def test_extend_far_positions_and_large_pools():
    """Positions near 2^31 and pool offsets past 2^31 elements."""
    ps, H = 256, 16
    mp, W = (2 ** 31 - 1) // ps, 300
    ctx = mp * ps - 60
    P = 4700  # 4700 * 16 * 256 * 128 = 2.46e9 elements of values
    table = torch.full((1, mp), -1, dtype=torch.int32, device=DEV)
    lo = (ctx - W + 1) // ps
    table[0, lo:] = torch.arange(P - (mp - lo), P, dtype=torch.int32, device=DEV)
    k_pool = torch.zeros(P, ps, 128, device=DEV, dtype=torch.bfloat16)
    v_pool = torch.zeros(P, H, ps, 128, device=DEV, dtype=torch.bfloat16)
    k_pool[-8:].normal_()
    v_pool[-8:].normal_()
    n = mp * ps - ctx
    q = torch.randn(n, H, 128, device=DEV).bfloat16()
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    c = torch.tensor([ctx], dtype=torch.int64, device=DEV)
    for m in (1, n):  # one token, and a chunk
        cu[1] = m
        o = rod.swska_extend_paged(q[:m].contiguous(), None, None, k_pool, v_pool, table, None, cu, c, W, sinks=4, max_len=m)
        rod.check()
        j = torch.arange(ctx - W + 1, ctx + m, device=DEV)
        pg, off = table[0, j // ps].long(), j % ps
        K, V = k_pool[pg, off].double(), v_pool[pg, :, off].double()
        for h in range(H):
            r, _, _, ra = ref.attend(q[:m, h].double(), K, V[:, h], ref.visible(torch.arange(ctx, ctx + m, device=DEV), j, W, 0), 128 ** -0.5)
            ref.check(o[:, h], r, ra, W + m, 128, ref.amp(q, K), f"far {m} head {h}")


def test_extend_graph_streams_and_repeats():
    """A captured call replayed on other lengths, tables and inputs equals the eager call bit for bit (the lengths live on the
    device); two calls at once with a workspace each; a repeat gives the same bits."""
    mk = lambda lens, s: ref.Batch("bf16", 6, 128, 128, 200, 4, 16, [50, 700, 0, 333], lens, pad=400 - sum(lens), seed=s, slack=40)
    a, b = mk([1, 300, 2, 90], 1), mk([200, 1, 0, 16], 2)
    P = max(a.P, b.P)
    for x in (a, b):  # one pool size and table width for both
        x.k_pool = torch.cat([x.k_pool, x.k_pool[:1].expand(P - x.P, -1, -1)])
        x.v_pool = torch.cat([x.v_pool, x.v_pool[:1].expand(P - x.P, -1, -1, -1)])
        x.P = P
    width = max(a.max_pages, b.max_pages)
    for x in (a, b):
        x.table = torch.nn.functional.pad(x.table, (0, width - x.max_pages), value=-1)
        x.max_pages = width
    eager = [_run(x, max_len=400) for x in (a, b)]
    again = _run(a, max_len=400)
    for x, got in ((a, eager[0]), (b, eager[1]), (a, again)):
        _check_run(x, got, "eager")
    assert torch.equal(again[0], eager[0][0])
    buf, o = a.args(DEV), a.o.to(DEV)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            rod.swska_extend_paged(*buf, a.W, sinks=a.S, max_len=400, o=o)
    for x, want in ((b, eager[1]), (a, eager[0])):
        for t, n in zip(buf, x.args(DEV)):
            t.copy_(n)
        o.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0])
    xa, xb, oa, ob = a.args(DEV), b.args(DEV), a.o.to(DEV), b.o.to(DEV)
    torch.cuda.synchronize()
    for _ in range(5):
        rod.swska_extend_paged(*xa, a.W, sinks=a.S, max_len=400, o=oa, stream=side,
                               workspace=_workspace(a, 400, "a"))
        rod.swska_extend_paged(*xb, b.W, sinks=b.S, max_len=400, o=ob, stream=other,
                               workspace=_workspace(b, 400, "b"))
    torch.cuda.synchronize()
    rod.check()
    assert torch.equal(oa, eager[0][0]) and torch.equal(ob, eager[1][0])


_spaces = {}


def _workspace(b, max_len, key):
    n = rod.load_library().rod_swska_extend_paged_workspace_size(b.q.shape[0], len(b.ctx), b.H, b.dk, b.dv, max_len, 1)
    if key not in _spaces:
        _spaces[key] = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
    return _spaces[key]


# ---- page tables --------------------------------------------------------------------------------------------
def _tables_once(ctx, new, table, first, stack, top, ps, W, S, M):
    dev = lambda x, dt=torch.int32: torch.tensor(x, dtype=dt, device=DEV)
    t, f, fl, fc = dev(table), dev(first), dev(stack), dev([top])
    c, m = dev(ctx, torch.int64), dev(new)
    cu, slot = rod.swska_page_tables(c, m, t, f, fl, fc, ps, W, S, M)
    rod.check()
    assert c.tolist() == [int(x) for x in ctx] and m.tolist() == [int(x) for x in new]
    return t.tolist(), f.tolist(), fl.tolist(), int(fc), cu.tolist(), slot.tolist()


@pytest.mark.parametrize("N,mp,P,ps,W,S,M", [(1, 10, 12, 8, 20, 3, 30), (5, 40, 60, 8, 37, 9, 100), (33, 30, 200, 16, 64, 0, 500),
                                             (70, 25, 500, 24, 100, 30, 5001), (3, 1500, 900, 1, 300, 2, 1000), (300, 12, 700, 64, 128, 4, 4099),
                                             (2, 4, 3, 256, 4096, 128, 600)])
def test_page_tables(N, mp, P, ps, W, S, M):
    """A random run of steps: chunks, single tokens, idle and finished sequences, rows that are full, memory that runs out."""
    r = np.random.RandomState(N)
    state = ([[-1] * mp for _ in range(N)], [0] * N, r.permutation(P).tolist(), P)
    ctx = [0] * N
    for step in range(12):
        new = [int(r.choice([0, 1, 1, 1, 5, 2 * ps, mp * ps // 4])) if r.rand() > 0.08 else -1 for _ in range(N)]
        want = ref.page_tables(ctx, new, *state, ps, W, S, M)
        got = _tables_once(ctx, new, *state, ps, W, S, M)
        for name, x, y in zip(("table", "first", "free list", "free count", "cu", "slot"), got, want):
            assert x == (y if isinstance(y, int) else list(y)), f"step {step}: {name}"
        state, cu = want[:4], want[4]
        for n in range(N):
            ctx[n] = 0 if new[n] < 0 else ctx[n] + cu[n + 1] - cu[n]


def test_page_tables_hostile():
    """Entries outside the pool are no pages; a free count outside the list is cut to it; ctx < 0 is left alone; a repeated
    call takes nothing more; wants past 2^31 in sum are refused, not wrapped."""
    args = ([40, -3, 7, 10 ** 12, 0, 0], [9, 4, -1, 5, 2 ** 31 - 1, 2 ** 31 - 1],
            [[3, 99, -8, 5, 2 ** 31 - 1, -1, -1, -1], [1] * 8, [4, -1, 7, 0, 0, 0, 0, 0], [2] * 8, [-1] * 8, [-1] * 8],
            [1, 0, 0, 3, 0, 0], [11, 12, 13, 14, 15, 8, 9, 10, 6, 2] + [0] * 10, 25, 8, 16, 4, 40)
    want = ref.page_tables(*args)
    got = _tables_once(*args)
    for x, y in zip(got, want):
        assert x == (y if isinstance(y, int) else list(y))
    # a free list that holds 10 and 11 for a pool of 10 pages: they are handed out, and are no pages the next time
    odd = ([40, 3], [9, 4], [[-1] * 8, [1] + [-1] * 7], [0, 0], list(range(2, 12)), 10, 8, 100, 4, 40)
    one = _tables_once(*odd)
    assert list(one) == list(ref.page_tables(*odd))
    assert list(_tables_once(*odd[:2], *one[:4], *odd[6:])) == list(ref.page_tables(*odd[:2], *one[:4], *odd[6:]))
    ok = ([40, 3], [9, 4], [[-1] * 8, [1] + [-1] * 7], [0, 0], list(range(2, 12)) + [0, 0], 10, 8, 100, 4, 40)
    one = _tables_once(*ok)
    assert _tables_once(*ok[:2], *one[:4], *ok[6:]) == one


def test_page_tables_none():
    dev = lambda n, dt=torch.int32: torch.zeros(n, dtype=dt, device=DEV)
    cu, slot = rod.swska_page_tables(dev(0, torch.int64), dev(0), torch.zeros(0, 4, dtype=torch.int32, device=DEV), dev(0), dev(5), dev(1), 8, 4, 0, 7)
    rod.check()
    assert cu.tolist() == [0] and slot.tolist() == [-1] * 7


# ---- together -------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_serving_run_equals_training_rows(dtype):
    """Three requests served through tables and paged attention -- a prompt in chunks, then single tokens, one idle at times, the
    pool too small for every page ever needed -- give the rows of the whole sequences' forward, and finished requests give all
    pages back. The steps run from one captured graph: lengths and tables stay on the device."""
    H, W, S, ps, d, N = 3, 70, 5, 16, 128, 3
    T = [420, 197, 250]
    seqs = [wl.swska_inputs(1, H, t, d, d, seed=t, dtype=dtype) for t in T]
    whole = [ref.train(q, k, v, torch.zeros_like(v), W, S) for q, k, v in seqs]
    P = 3 * (-(-(W + 90) // ps) + 2)
    assert P * ps < sum(T)
    M, mp = 150, -(-max(T) // ps)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)
    table, first = i32(N, mp) - 1, i32(N)
    free_list, count = torch.randperm(P, device=DEV).to(torch.int32), i32(1) + P
    ctx, n_new = torch.zeros(N, dtype=torch.int64, device=DEV), i32(N)
    kp, vp = torch.full((P, ps, d), math.nan, device=DEV, dtype=DT[dtype]), torch.full((P, H, ps, d), math.nan, device=DEV, dtype=DT[dtype])
    q, kn, vn = (torch.zeros(*s, device=DEV, dtype=DT[dtype]) for s in ((M, H, d), (M, d), (M, H, d)))
    o = torch.zeros(M, H, d, device=DEV, dtype=DT[dtype])
    cu, slot = i32(N + 1), i32(M)

    def step():
        rod.swska_page_tables(ctx, n_new, table, first, free_list, count, ps, W, S, M, cu_seqlens=cu, slot_map=slot)
        rod.swska_extend_paged(q, kn, vn, kp, vp, table, slot, cu, ctx, W, sinks=S, o=o)
        ctx.add_(cu[1:] - cu[:-1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step()  # a step without tokens
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    at, r = [0] * N, np.random.RandomState(0)
    for it in range(400):
        lens = [min(T[n] - at[n], int(r.choice([0, 1, 1, 1, 30, 50])) if at[n] else 40) for n in range(N)]
        if sum(lens) == 0 and all(a == t for a, t in zip(at, T)):
            break
        pos = 0
        for n, m in enumerate(lens):
            sq, sk, sv = seqs[n]
            rows = slice(at[n], at[n] + m)
            q[pos:pos + m] = sq[0, :, rows].transpose(0, 1).to(DEV)
            kn[pos:pos + m] = sk[0, rows].to(DEV)
            vn[pos:pos + m] = sv[0, :, rows].transpose(0, 1).to(DEV)
            pos += m
        n_new.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        assert (cu[1:] - cu[:-1]).tolist() == lens, "the pool is large enough for what a window needs"
        pos = 0
        for n, m in enumerate(lens):
            if m:
                w = whole[n]["o"]
                rows = slice(at[n], at[n] + m)
                ref.check(o[pos:pos + m].cpu(), w[0][0, :, rows].transpose(0, 1), w[1][0, :, rows].transpose(0, 1), W + S, d,
                          ref.amp(seqs[n][0], seqs[n][1]), f"step {it} sequence {n}")
            at[n] += m
            pos += m
    assert at == T
    n_new.fill_(-1)
    rod.swska_page_tables(ctx, n_new, table, first, free_list, count, ps, W, S, M)
    rod.check()
    assert int(count) == P and sorted(free_list.tolist()) == list(range(P)) and (table == -1).all()
