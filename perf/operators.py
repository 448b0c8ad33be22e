"""Cases and plain forms of the SW-SKA operators with first tokens that stay visible, over a paged cache.

Three operators (one key matrix k shared by the H heads, per-head values v, window W, the first S
tokens of a sequence visible to every later query; query at position p sees the keys
j <= p with j > p - W or j < S):

  train   forward (output and row log-sum-exp) and gradients of whole sequences [B,H,T,d];
  extend  a ragged batch of new tokens (one, a few or a long chunk per sequence, some sequences
          idle) is written to a paged cache and attends over it;
  tables  the block tables, the free list and the slot map for such a batch, from each
          sequence's cached and new lengths (pages behind the window go back, pages for the new
          tokens are taken).

``own`` false: the plain forms below; true: the calls of the package."""
import math
import random

import torch

own = False

BF16, FP32 = torch.bfloat16, torch.float32
NEG = float("-inf")


def _dtype(case):
    return BF16 if case["dtype"] == "bf16" else FP32


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _train(name, dtype, B, H, T, dk, dv, W, S):
    c = dict(op="train", dtype=dtype, B=B, H=H, T=T, dk=dk, dv=dv, window=W, sinks=S)
    return dict(c, name=name) if name else c


def _extend(name, dtype, N, H, dk, dv, W, S, page, len_lo, len_hi, ctx_lo, ctx_hi, idle=0.0, ones=0.0, pad=0, mix=0):
    c = dict(op="extend", dtype=dtype, N=N, H=H, dk=dk, dv=dv, window=W, sinks=S, page=page, len_lo=len_lo, len_hi=len_hi,
             ctx_lo=ctx_lo, ctx_hi=ctx_hi, idle=idle, ones=ones, pad=pad, mix=mix)
    return dict(c, name=name) if name else c


def _tables(name, N, W, S, page, len_lo, len_hi, ctx_lo, ctx_hi, idle=0.0, ones=0.0, done=0.0, short=False, pad=0, mix=0):
    c = dict(op="tables", N=N, window=W, sinks=S, page=page, len_lo=len_lo, len_hi=len_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi,
             idle=idle, ones=ones, done=done, short=short, pad=pad, mix=mix)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a training step of one SW-SKA layer of the 16 x 128 configuration at the sequence length of its backward benchmark
        _train("train bf16 t8192", "bf16", 1, 16, 8192, 128, 128, 4096, 4),
        # a batch of ragged documents cut to an odd length, few heads, a short window
        _train("train bf16 t1999", "bf16", 3, 5, 1999, 128, 128, 500, 13),
        # narrow heads in bf16
        _train("train bf16 d64", "bf16", 2, 8, 1500, 64, 64, 300, 8),
        # the tiny fp32 configuration used for correctness runs
        _train("train fp32 tiny", "fp32", 1, 2, 256, 16, 32, 64, 4),
        # fp32 training of a small model
        _train("train fp32 t1000", "fp32", 1, 4, 1000, 64, 128, 256, 5),
        # one token for each of many sequences whose windows are full: a serving batch's decode step
        _extend("decode n128", "bf16", 128, 16, 128, 128, 4096, 4, 64, 1, 1, 4096, 20000),
        # one token of one sequence: latency
        _extend("decode n1", "bf16", 1, 16, 128, 128, 4096, 4, 64, 1, 1, 9000, 9000),
        # a long prompt's next chunk
        _extend("chunk 2048", "bf16", 1, 16, 128, 128, 4096, 4, 64, 2048, 2048, 30000, 30000),
        # chunks beside single tokens and idle rows of a padded batch, pages that end inside a tile
        _extend("mixed n33", "bf16", 33, 5, 128, 128, 1000, 5, 24, 2, 400, 0, 3000, idle=0.2, ones=0.5, pad=37, mix=3),
        # fp32 with narrow heads, a few tokens each
        _extend("few fp32", "fp32", 9, 4, 64, 32, 200, 3, 16, 1, 20, 0, 700, idle=0.1, mix=4),
        # the tables of a decode step of 256 sequences
        _tables("tables n256", 256, 4096, 4, 64, 1, 1, 100, 100000, done=0.02, mix=5),
        # the tables of a large prefill batch, small pages, some sequences waiting for memory
        _tables("tables n512 chunks", 512, 2048, 4, 16, 1, 700, 0, 60000, idle=0.1, ones=0.3, done=0.05, short=True, pad=1000, mix=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["train", "train", "extend", "extend", "extend", "tables"])
    if op == "train":
        fast = rng.random() < 0.6
        dtype = "bf16" if fast or rng.random() < 0.3 else "fp32"
        dk, dv = (128, 128) if fast else (rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128]))
        H, B = rng.randint(1, 16), rng.choice([1, 1, 2, 3, 4])
        most = 6000 if fast else 2500
        T = min(_log(rng, 1, most), int(math.sqrt((4e8 if fast else 5e7) / (H * B))))
        return _train(None, dtype, B, H, max(1, T), dk, dv, _log(rng, 1, 4096), rng.choice([0, 1, 4, rng.randint(1, 128)]))
    shape = rng.choice(["one", "few", "chunk", "mixed"])
    page, W, S = 8 * _log(rng, 1, 32), _log(rng, 16, 4096), rng.choice([0, 1, 4, 4, rng.randint(0, 128)])
    mix = rng.randrange(1 << 20)
    ctx_hi = _log(rng, 1, 40000)
    ctx_lo = rng.choice([0, 0, ctx_hi // 2])
    if op == "tables":
        N = _log(rng, 1, 512)
        lens = {"one": (1, 1), "few": (1, 16), "chunk": (1, 700), "mixed": (1, 300)}[shape]
        return _tables(None, N, W, S, page, lens[0], lens[1], ctx_lo, ctx_hi, idle=rng.choice([0.0, 0.2]), ones=0.6 if shape == "mixed" else 0.0,
                       done=rng.choice([0.0, 0.1]), short=rng.random() < 0.3, pad=rng.randint(0, 200), mix=mix)
    fast = rng.random() < 0.75
    dtype = "bf16" if fast or rng.random() < 0.3 else "fp32"
    dk, dv = (128, 128) if fast else (rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128]))
    H = rng.randint(1, 16)
    if shape == "one":
        N, lens = _log(rng, 1, 128 if fast else 24), (1, 1)
    elif shape == "few":
        N, lens = _log(rng, 1, 64 if fast else 16), (1, rng.randint(2, 20))
    elif shape == "chunk":
        N = rng.randint(1, 3)
        hi = _log(rng, 17, 2000 if fast else 200)
        lens = (max(1, hi // 2), hi)
    else:
        N, lens = rng.randint(2, 24 if fast else 8), (1, _log(rng, 17, 500 if fast else 100))
    if not fast:
        W = min(W, 1000)
    return _extend(None, dtype, N, H, dk, dv, W, S, page, lens[0], lens[1], ctx_lo, ctx_hi, idle=rng.choice([0.0, 0.2]),
                   ones=0.5 if shape == "mixed" else 0.0, pad=rng.choice([0, rng.randint(1, 40)]), mix=mix)


def _lengths(case):
    """(cached, new) tokens of each sequence; new = 0: idle, -1: finished (tables only)."""
    r = random.Random(case["mix"] * 7919 + case["N"])
    ctx, new = [], []
    for _ in range(case["N"]):
        c = r.randint(case["ctx_lo"], case["ctx_hi"])
        m = r.randint(case["len_lo"], case["len_hi"])
        m = 1 if r.random() < case["ones"] else m
        m = 0 if r.random() < case["idle"] else m
        m = -1 if r.random() < case.get("done", 0.0) else m
        ctx.append(c)
        new.append(m)
    if case["op"] == "extend" and not any(new):
        new[0] = case["len_lo"]
    return ctx, new


def _pages(case, ctx, new):
    """Logical pages that each sequence holds before the call: those of the first tokens and those of the last window."""
    ps, S, W = case["page"], case["sinks"], case["window"]
    held, first = [], []
    for c in ctx:
        used, sp = -(-c // ps), -(-S // ps)
        back = c - 1  # the last step left the window of the token before
        f = min(used, max(sp, max(0, back - W + 1) // ps))
        held.append([p for p in range(min(sp, used))] + [p for p in range(max(min(sp, used), f), used)])
        first.append(f if used > sp else 0)
    return held, first


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _queries(shape, u, g, dt):
    return (torch.randn(shape, generator=g, device="cuda") + 4.0 * u).to(dt)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] == "tables":
        return _prepare_tables(st, case, seed)
    dt, dk, dv, H, S = _dtype(case), case["dk"], case["dv"], case["H"], case["sinks"]
    u = torch.randn(dk, generator=g, device="cuda")
    u = u / u.norm()  # the direction in which the first tokens draw attention
    if case["op"] == "train":
        B, T = case["B"], case["T"]
        st["q"] = _queries((B, H, T, dk), u, g, dt)
        k = torch.randn((B, T, dk), generator=g, device="cuda")
        k[:, :S] += 8.0 * u
        st["k"] = k.to(dt)
        st["v"] = torch.randn((B, H, T, dv), generator=g, device="cuda").to(dt)
        st["dO"] = torch.randn((B, H, T, dv), generator=g, device="cuda").to(dt)
        return st
    N, ps = case["N"], case["page"]
    ctx, new = _lengths(case)
    held, _ = _pages(case, ctx, new)
    max_pages = max(-(-(c + m) // ps) for c, m in zip(ctx, new)) + 1
    table = torch.full((N, max_pages), -1, dtype=torch.int32)
    for n in range(N):  # the new tokens' pages are there too: the tables were built before
        held[n] += [p for p in range(-(-ctx[n] // ps), -(-(ctx[n] + new[n]) // ps))]
    P = sum(len(h) for h in held) + 3
    perm = torch.randperm(P, generator=torch.Generator().manual_seed(int(seed)), dtype=torch.int64).to(torch.int32)
    at = 0
    for n in range(N):
        if held[n]:
            table[n, torch.tensor(held[n])] = perm[at:at + len(held[n])]
        at += len(held[n])
    M = sum(new) + case["pad"]
    slot = torch.full((M,), -1, dtype=torch.int32)
    cu = [0]
    for n in range(N):
        p = torch.arange(ctx[n], ctx[n] + new[n])
        slot[cu[-1]:cu[-1] + new[n]] = table[n, p // ps] * ps + (p % ps).to(torch.int32)
        cu.append(cu[-1] + new[n])
    st["block_table"], st["slot_map"] = table.cuda(), slot.cuda()
    st["cu"] = torch.tensor(cu, dtype=torch.int32).cuda()
    st["ctx"] = torch.tensor(ctx, dtype=torch.int64).cuda()
    k_pool = torch.randn((P, ps, dk), generator=g, device="cuda")
    for i in range(-(-S // ps) if S else 0):  # the first tokens' keys
        if i < max_pages:
            have = st["block_table"][:, i]
            k_pool[have[have >= 0].long(), :min(ps, S - i * ps)] += 8.0 * u
    st["k_pool"] = k_pool.to(dt)
    del k_pool
    v_pool = torch.empty((P, H, ps, dv), dtype=dt, device="cuda")
    v_pool.normal_(generator=g)
    st["v_pool"] = v_pool
    st["q"] = _queries((M, H, dk), u, g, dt)
    st["k_new"] = torch.randn((M, dk), generator=g, device="cuda").to(dt)
    st["v_new"] = torch.randn((M, H, dv), generator=g, device="cuda").to(dt)
    st["o"] = torch.zeros((M, H, dv), dtype=dt, device="cuda")
    st["max_len"] = max(new)
    st["span"] = max(c + m - max(0, c - case["window"] + 1) for c, m in zip(ctx, new))
    return st


def _prepare_tables(st, case, seed):
    N, ps = case["N"], case["page"]
    ctx, new = _lengths(case)
    held, first = _pages(case, ctx, new)
    max_pages = max(-(-(c + max(m, 0)) // ps) for c, m in zip(ctx, new)) + 2
    want = sum(max(0, -(-(c + m) // ps) - -(-c // ps)) for c, m in zip(ctx, new) if m > 0)
    have = sum(len(h) for h in held)
    free = want // 2 if case["short"] else want + 5
    P = max(1, have + free)
    perm = torch.randperm(P, generator=torch.Generator().manual_seed(int(seed)), dtype=torch.int64).to(torch.int32)
    table = torch.full((N, max_pages), -1, dtype=torch.int32)
    at = 0
    for n in range(N):
        if held[n]:
            table[n, torch.tensor(held[n])] = perm[at:at + len(held[n])]
        at += len(held[n])
    free_list = torch.full((P,), -1, dtype=torch.int32)
    free_list[:P - have] = perm[have:]
    # one buffer, so that a pass can start from the same state with one copy
    st["held"] = torch.cat([table.reshape(-1), torch.tensor(first, dtype=torch.int32), free_list, torch.tensor([P - have], dtype=torch.int32)]).cuda()
    st["sizes"] = (N, max_pages, P)
    st["ctx"] = torch.tensor(ctx, dtype=torch.int64).cuda()
    st["n_new"] = torch.tensor(new, dtype=torch.int32).cuda()
    st["max_tokens"] = sum(max(m, 0) for m in new) + case["pad"]
    return st


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(st):
    if st["op"] == "train":
        return _run_train(st)
    if st["op"] == "extend":
        return _run_extend(st)
    return _run_tables(st)


def _run_train(st):
    q, k, v, dO, W, S = st["q"], st["k"], st["v"], st["dO"], st["window"], st["sinks"]
    if own:
        import sliding_window_attention_chunked_b200 as rod

        o, lse = rod.swska_sink_prefill(q, k, v, W, S)
        dq, dk, dv = rod.swska_sink_backward(q, k, v, o, lse, dO, W, S)
    else:
        o, lse, dq, dk, dv = _plain_train(q, k, v, dO, W, S)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _visible(p, j, W, S):
    return (j <= p) & ((j > p - W) | (j < S))


def _plain_train(q, k, v, dO, W, S):
    dt, (B, H, T, dk) = q.dtype, q.shape
    q, k, v, dO = q.float(), k.float(), v.float(), dO.float()
    scale = 1.0 / math.sqrt(dk)
    t = torch.arange(T, device=q.device)
    see = _visible(t[:, None], t[None, :], W, S)
    s = torch.matmul(q, k[:, None].transpose(-1, -2)) * scale
    s.masked_fill_(~see, NEG)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    del s
    l = p.sum(-1, keepdim=True)
    p /= l
    o = torch.matmul(p, v)
    lse = (m + torch.log(l)).squeeze(-1)
    D = (dO * o).sum(-1, keepdim=True)
    dv = torch.matmul(p.transpose(-1, -2), dO)
    ds = torch.matmul(dO, v.transpose(-1, -2))
    ds -= D
    ds *= p
    del p
    dq = torch.matmul(ds, k[:, None]) * scale
    dkey = torch.matmul(ds.transpose(-1, -2), q).sum(1) * scale
    return o.to(dt), lse, dq.to(dt), dkey.to(dt), dv.to(dt)


def _run_extend(st):
    args = [st[n] for n in ("q", "k_new", "v_new", "k_pool", "v_pool", "block_table", "slot_map", "cu", "ctx")]
    if own:
        import sliding_window_attention_chunked_b200 as rod

        rod.swska_extend_paged(*args, st["window"], sinks=st["sinks"], max_len=st["max_len"], o=st["o"])
    else:
        _plain_extend(*args, st["window"], st["sinks"], st["max_len"], st["span"], st["o"])
    return {"o": st["o"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def _plain_extend(q, k_new, v_new, k_pool, v_pool, table, slot, cu, ctx, W, S, L, span, o):
    (M, H, dk), (P, ps, _), dv, N, dev = q.shape, k_pool.shape, v_pool.shape[-1], ctx.shape[0], q.device
    # the new tokens into their slots (a padded row, slot -1, repeats the first token's write)
    i = torch.where(slot >= 0, torch.arange(M, device=dev), 0)
    to = slot[i].long()
    k_pool.view(P * ps, dk)[to] = k_new[i]
    v_pool[to // ps, :, to % ps] = v_new[i]
    # the keys that a sequence's new tokens see: its first S tokens, then a span from its first window's start
    lo = (ctx - W + 1).clamp_min(0)[:, None]
    j = torch.cat([torch.arange(S, device=dev)[None].expand(N, S), lo + torch.arange(span, device=dev)[None]], 1)
    there = torch.cat([torch.arange(S, device=dev)[None] < lo, torch.ones((N, span), dtype=torch.bool, device=dev)], 1)
    col = j // ps
    page = torch.where(col < table.shape[1], torch.gather(table, 1, col.clamp_max(table.shape[1] - 1)), -1)
    there &= page >= 0
    page, off = page.clamp_min(0).long(), j % ps
    k, v = k_pool[page, off].float(), v_pool[page, :, off].float()  # [N,K,dk], [N,K,H,dv]
    # queries padded to the longest
    a = torch.arange(L, device=dev)
    row = cu[:-1, None].long() + a
    live = row < cu[1:, None]
    qp = q[row.clamp_max(M - 1)].float().transpose(1, 2)  # [N,H,L,dk]
    pos = ctx[:, None] + a
    s = torch.matmul(qp, k[:, None].transpose(-1, -2)) * (1.0 / math.sqrt(dk))
    see = _visible(pos[:, :, None], j[:, None, :], W, S) & there[:, None, :]
    s.masked_fill_(~see[:, None], NEG)
    m = s.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(s - m)
    del s
    out = torch.matmul(p, v.transpose(1, 2)) / p.sum(-1, keepdim=True).clamp_min(1e-38)
    out = out.transpose(1, 2).to(o.dtype)  # [N,L,H,dv]
    # rows of no sequence keep what they hold
    where = torch.where(live, row, M).reshape(-1)
    wide = torch.cat([o, torch.zeros_like(o[:1])])
    wide[where] = out.reshape(-1, H, dv)
    o.copy_(wide[:M])


def _run_tables(st):
    N, max_pages, P = st["sizes"]
    held = st["held"].clone()
    at = N * max_pages
    table, first, free_list, count = held[:at].view(N, max_pages), held[at:at + N], held[at + N:at + N + P], held[at + N + P:]
    if own:
        import sliding_window_attention_chunked_b200 as rod

        cu, slot = rod.swska_page_tables(st["ctx"], st["n_new"], table, first, free_list, count, st["page"], st["window"], st["sinks"], st["max_tokens"])
    else:
        cu, slot = _plain_tables(st["ctx"], st["n_new"], table, first, free_list, count, st["page"], st["window"], st["sinks"], st["max_tokens"])
    return {"block_table": table, "first": first, "free_list": free_list, "free_count": count, "cu_seqlens": cu, "slot_map": slot}


def _plain_tables(ctx, n_new, table, first, free_list, count, ps, W, S, M):
    N, max_pages = table.shape
    P, dev = free_list.shape[0], table.device
    new = n_new.long()
    active, done = (new > 0) & (ctx >= 0), (new < 0) & (ctx >= 0)
    sp = -(-S // ps)
    used = torch.div(ctx + ps - 1, ps, rounding_mode="floor")
    end = torch.div(ctx + new.clamp_min(0) + ps - 1, ps, rounding_mode="floor")
    low = torch.div((ctx - W + 1).clamp_min(0), ps, rounding_mode="floor").clamp_min(sp).minimum(used)
    # pages behind the window go back, and all of a finished sequence's
    col = torch.arange(max_pages, device=dev)[None]
    gone = active[:, None] & (col >= first[:, None]) & (col >= sp) & (col < low[:, None])
    gone |= done[:, None]
    gone &= table >= 0
    total = gone.sum()
    rank = torch.cumsum(gone.reshape(-1).long(), 0) - 1
    dst = torch.where(gone.reshape(-1), count.long() + rank, P)
    stack = torch.cat([free_list, free_list[:1]])
    stack[dst] = table.reshape(-1)
    # the new tokens' pages, while they last; what a sequence holds already stays
    lack = (active & (end <= max_pages))[:, None] & (col >= used[:, None]) & (col < end[:, None]) & (table < 0)
    need = lack.sum(1)
    upto = torch.cumsum(need, 0)
    fits = active & (end <= max_pages) & (torch.cumsum(new * active, 0) <= M)
    ok = fits & ((need == 0) | (upto <= count + total))
    take = torch.where(ok, need, 0)
    before = torch.cumsum(take, 0) - take
    fresh = ok[:, None] & lack
    src = count.long() + total - (before[:, None] + torch.cumsum(lack, 1))
    got = stack[src.clamp(0, P)]
    table.copy_(torch.where(fresh, got, torch.where(gone, -1, table)))
    first.copy_(torch.where(done, 0, torch.where(active, torch.maximum(first, low.to(torch.int32)), first)))
    free_list.copy_(stack[:P])
    count.copy_(count + total - take.sum())
    # where each new token goes
    served = torch.where(ok, new, 0)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(served, 0)])
    i = torch.arange(M, device=dev)
    n = torch.searchsorted(cu[1:].contiguous(), i, right=True).clamp_max(N - 1)
    pos = (ctx[n] + i - cu[n]).clamp_min(0)
    entry = table[n, torch.div(pos, ps, rounding_mode="floor").clamp_max(max_pages - 1)].long()
    slot = torch.where((i < cu[-1]) & (entry >= 0), entry * ps + pos % ps, -1)
    return cu.to(torch.int32), slot.to(torch.int32)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def _seen(p, W, S):
    """Keys that the query at position p sees."""
    lo = max(0, p - W + 1)
    return p + 1 - lo + min(S, lo)


def work(case):
    W, S = case["window"], case["sinks"]
    if case["op"] == "train":
        B, H, T, dk, dv = (case[n] for n in ("B", "H", "T", "dk", "dv"))
        es = 2 if case["dtype"] == "bf16" else 4
        pairs = B * H * sum(_seen(p, W, S) for p in range(T))
        rows = B * H * T
        return {"bytes": es * (2 * rows * (dk + 2 * dv) + 2 * B * T * dk) + 4 * rows, "flops": pairs * (8 * dk + 6 * dv)}
    ctx, new = _lengths(case)
    ps = case["page"]
    if case["op"] == "extend":
        H, dk, dv = case["H"], case["dk"], case["dv"]
        es = 2 if case["dtype"] == "bf16" else 4
        keys = pairs = 0
        for c, m in zip(ctx, new):
            if m > 0:
                lo = max(0, c - W + 1)
                keys += c - lo + min(S, lo)
                pairs += sum(_seen(p, W, S) for p in range(c, c + m))
        M = sum(new)
        return {"bytes": es * (keys * (dk + H * dv) + M * (H * (dk + dv) + 2 * (dk + H * dv))) + 4 * (keys // ps + M), "flops": pairs * H * 2 * (dk + dv)}
    held, first = _pages(case, ctx, new)
    moved = sum(len(h) if m < 0 else max(0, max(-(-S // ps), max(0, c - W + 1) // ps) - f) if m > 0 else 0 for h, f, c, m in zip(held, first, ctx, new))
    taken = sum(-(-(c + m) // ps) - -(-c // ps) for c, m in zip(ctx, new) if m > 0)
    tokens = sum(max(m, 0) for m in new) + case["pad"]
    return {"bytes": 12 * case["N"] + 8 * case["N"] + 4 * case["N"] + 12 * moved + 8 * taken + 4 * tokens, "flops": 2 * tokens + 10 * case["N"]}


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    st = prepare(case, seed)
    return _exact_train(st) if case["op"] == "train" else _exact_extend(st)


def _softmax64(s, see):
    """Rows of probabilities and their log-sum-exp over the visible entries."""
    top = torch.where(see, s, torch.full_like(s, -1e300)).max(-1, keepdim=True).values
    e = torch.where(see, (s - top).exp(), torch.zeros_like(s))
    z = e.sum(-1, keepdim=True)
    return e / z, (top + z.log()).squeeze(-1)


def _exact_train(st):
    q, k, v, g, W, S = (st[n] for n in ("q", "k", "v", "dO", "window", "sinks"))
    B, H, T, d = q.shape
    r = torch.arange(T, device=q.device)
    age = r[:, None] - r[None, :]
    see = (age >= 0) & ((age < W) | (r[None, :] < S))
    out = {n: torch.empty(x.shape, dtype=torch.float64, device=q.device) for n, x in (("o", v), ("dq", q), ("dv", v))}
    out["lse"] = torch.empty((B, H, T), dtype=torch.float64, device=q.device)
    out["dk"] = torch.zeros(k.shape, dtype=torch.float64, device=q.device)
    c = d ** -0.5
    for b in range(B):
        K = k[b].double()
        for h in range(H):
            Q, V, G = q[b, h].double(), v[b, h].double(), g[b, h].double()
            prob, out["lse"][b, h] = _softmax64(c * (Q @ K.T), see)
            out["o"][b, h] = prob @ V
            out["dv"][b, h] = prob.T @ G
            e = prob * (G @ V.T - (G * out["o"][b, h]).sum(1, keepdim=True)) * c
            out["dq"][b, h] = e @ K
            out["dk"][b] += e.T @ Q
    return out


def _exact_extend(st):
    q, table, slot, W, S, ps = (st[n] for n in ("q", "block_table", "slot_map", "window", "sinks", "page"))
    kp, vp, o = st["k_pool"].clone(), st["v_pool"], st["o"].double()
    H, d = q.shape[1], q.shape[2]
    new = (slot >= 0).nonzero().squeeze(1)
    at = slot[new].long()
    kp[at // ps, at % ps] = st["k_new"][new]
    vp[at // ps, :, at % ps] = st["v_new"][new]
    ctx, lens = _lengths(st)
    r0 = 0
    for n, (c, m) in enumerate(zip(ctx, lens)):
        if m <= 0:
            continue
        end, lo = c + m, max(0, c - W + 1)
        key = torch.tensor([x for x in range(min(S, lo))] + [x for x in range(lo, end)], device=q.device)
        page = table[n, key // ps].long()
        K = kp[page, key % ps].double()
        V = vp[page, :, key % ps].double()
        age = torch.arange(c, end, device=q.device)[:, None] - key[None]
        see = (age >= 0) & ((age < W) | (key[None] < S))
        for h in range(H):
            prob, _ = _softmax64(q[r0:r0 + m, h].double() @ K.T / math.sqrt(d), see)
            o[r0:r0 + m, h] = prob @ V[:, h]
        r0 += m
    return {"o": o, "k_pool": None, "v_pool": None}
