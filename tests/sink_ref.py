"""Plain 64-bit references of the SW-SKA operators with first tokens that stay visible, of the paged
attention of new tokens, and of the page tables (python loops); and the tolerances that go with
them, counted from the roundings of the kernels.

Tolerances. H = finfo(dtype).eps / 2 is the largest relative error of one rounding. Every output is
rounded once: H |ref|. The tensor-core route also rounds each probability p (and each dS) to bf16
before a product, so a sum of terms x_j = p_j v_j is off by at most H sum |x_j|; D is taken from the
stored o, off by H sum |dO o|. fp32 work adds at most (n + d) 2^-23 relative to the sum of absolute
terms for n terms and head dim d: a dot product of d terms in the exponent (times ln 2 scaling, terms
of size |q||k| scale, given as `amp`), a sum of n terms. The kernels' exponentials are good to 2^-13
on the tensor-core route (a cubic on the FMA pipe) and to 2^-21 elsewhere."""
import math

import numpy as np
import torch


def visible(p, j, W, S):
    p, j = torch.as_tensor(p)[:, None], torch.as_tensor(j)[None, :]
    return (j <= p) & ((j > p - W) | (j < S))


def attend(q, k, v, see, scale):
    """One head: q [n,d], k [m,d], v [m,e] in fp64. Rows without a visible key: o = 0, lse = -inf.
    Returns (o, lse, p, sum_j p_j |v_j|)."""
    s = (q @ k.T) * scale
    s = torch.where(see, s, torch.full_like(s, -math.inf))
    m = s.max(1, keepdim=True).values.clamp_min(-1e300)
    e = torch.exp(s - m)
    z = e.sum(1, keepdim=True)
    p = torch.where(z > 0, e / z.clamp_min(1e-300), torch.zeros_like(e))
    lse = torch.where(z[:, 0] > 0, m[:, 0] + torch.log(z[:, 0].clamp_min(1e-300)), torch.full_like(z[:, 0], -math.inf))
    return p @ v, lse, p, p @ v.abs()


def train(q, k, v, dO, W, S, scale=None):
    """Forward and gradients of [B,H,T,d] tensors in fp64, each with the sum of absolute terms that
    its tolerance is relative to. Returns dict name -> (ref, abs_sum)."""
    q, k, v, dO = (x.double() for x in (q, k, v, dO))
    B, H, T, d = q.shape
    scale = scale or 1.0 / math.sqrt(d)
    t = torch.arange(T, device=q.device)
    see = visible(t, t, W, S)
    z = lambda x: torch.zeros_like(x)
    out = {n: (z(x), z(x)) for n, x in (("o", v), ("dq", q), ("dk", k), ("dv", v))}
    lse = torch.zeros(B, H, T, dtype=torch.float64, device=q.device)
    for b in range(B):
        for h in range(H):
            o, l, p, oa = attend(q[b, h], k[b], v[b, h], see, scale)
            out["o"][0][b, h], out["o"][1][b, h], lse[b, h] = o, oa, l
            dP = dO[b, h] @ v[b, h].T
            D = (dO[b, h] * o).sum(1, keepdim=True)
            dS = p * (dP - D)
            dSa = p * (dP.abs() + D.abs() + (dO[b, h] * o).abs().sum(1, keepdim=True))
            out["dq"][0][b, h], out["dq"][1][b, h] = dS @ k[b] * scale, dSa @ k[b].abs() * scale
            out["dk"][0][b] += dS.T @ q[b, h] * scale
            out["dk"][1][b] += dSa.T @ q[b, h].abs() * scale
            out["dv"][0][b, h], out["dv"][1][b, h] = p.T @ dO[b, h], p.T @ dO[b, h].abs()
    out["lse"] = (lse, torch.ones_like(lse))
    return out


def amp(q, k, scale=None):
    """Largest sum of absolute terms of a scaled score."""
    scale = scale or 1.0 / math.sqrt(q.shape[-1])
    return float(q.double().abs().sum(-1).max() * k.double().abs().max() * scale) if q.numel() else 0.0


def check(got, ref, abs_sum, n, d, score_amp, what, rounds=True):
    """|got - ref| <= tolerance element by element (see the module's text). n: terms of the longest
    sum; rounds: whether the dtype's rounding enters the products (bf16 tensor cores)."""
    assert tuple(got.shape) == tuple(ref.shape), f"{what}: shape"
    g = got.double().to(ref.device)
    half = torch.finfo(got.dtype).eps / 2
    inner = (n + d) * 2.0 ** -23 * (1 + score_amp) + 2.0 ** -21
    if got.dtype == torch.bfloat16 and rounds:
        inner += 2.0 ** -8 + 2.0 ** -13
    tol = half * ref.abs() * (1 + 2.0 ** -7) + inner * abs_sum * (1 + 2.0 ** -7) + 1e-30
    same = (g == ref) | (torch.isnan(g) & torch.isnan(ref))
    bad = ~same & ~((g - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off; worst "
                           f"{float(((g - ref).abs() / tol)[bad].max()):.3g} tolerances at {bad.nonzero()[0].tolist()}")


def extend(q, k_new, v_new, k_pool, v_pool, table, slot, cu, ctx, W, S, o, max_len=None, scale=None):
    """Paged attention of new tokens on CPU tensors; returns (o, sum of absolute terms, k_pool, v_pool)."""
    M, H, d = q.shape
    P, ps = k_pool.shape[:2]
    scale = scale or 1.0 / math.sqrt(d)
    k_pool, v_pool = k_pool.clone(), v_pool.clone()
    if k_new is not None:
        for i in range(M):
            s = int(slot[i])
            if 0 <= s < P * ps:
                k_pool[s // ps, s % ps] = k_new[i]
                v_pool[s // ps, :, s % ps] = v_new[i]
    out = o.double().clone()
    oa = torch.zeros_like(out)
    for n in range(len(ctx)):
        r0, r1, c = int(cu[n]), int(cu[n + 1]), int(ctx[n])
        r1 = min(r1, r0 + (max_len or M))
        if r1 <= r0:
            continue
        if c < 0 or c > 2 ** 31 - 1 - (r1 - r0):
            out[r0:r1] = math.nan
            continue
        pos = torch.arange(c, c + r1 - r0)
        keys = sorted(set(range(min(S, c + r1 - r0))) | set(range(max(0, c - W + 1), c + r1 - r0)))
        keys = [j for j in keys if j // ps < table.shape[1] and 0 <= int(table[n, j // ps]) < P]
        if not keys:
            out[r0:r1] = 0
            continue
        j = torch.tensor(keys)
        pg = table[n, j // ps].long()
        K, V = k_pool[pg, j % ps].double(), v_pool[pg, :, j % ps].double()
        see = visible(pos, j, W, S)
        for h in range(H):
            out[r0:r1, h], _, _, oa[r0:r1, h] = attend(q[r0:r1, h].double(), K, V[:, h], see, scale)
    return out, oa, k_pool, v_pool


def page_tables(ctx, n_new, table, first, free_list, free_count, ps, W, S, M):
    """The bookkeeping step with python integers; returns new (table, first, free_list, free_count, cu, slot)."""
    N, mp = len(table), len(table[0])
    P = len(free_list)
    table, first, stack = [list(r) for r in table], list(first), list(free_list)
    top = min(max(int(free_count), 0), P)
    sp = -(-S // ps)
    for n in range(N):
        c, m = int(ctx[n]), int(n_new[n])
        if c < 0 or m == 0:
            continue
        if m < 0:
            back, first_n = range(mp), 0
        else:
            low = min(max(max(0, c - W + 1) // ps, sp), -(-c // ps), mp)
            back, first_n = range(max(first[n], sp), low), max(first[n], low)
        for p in back:
            e = table[n][p]
            if 0 <= e < P and top < P:
                stack[top] = e
                top += 1
            table[n][p] = -1
        first[n] = first_n
    avail, top0 = top, top
    cu, needed, wanted = [0], 0, 0
    for n in range(N):
        c, m = int(ctx[n]), int(n_new[n])
        served = 0
        if c >= 0 and m > 0:
            wanted += m
            lo, hi = -(-c // ps), -(-(c + m) // ps)
            if hi <= mp:
                lack = [p for p in range(lo, hi) if not 0 <= table[n][p] < P]
                needed += len(lack)
                if wanted <= M and (not lack or needed <= avail):
                    served = m
                    for p in lack:
                        top -= 1
                        table[n][p] = stack[top]
        cu.append(cu[-1] + served)
    slot = [-1] * M
    for n in range(N):
        for i in range(cu[n], cu[n + 1]):
            pos = int(ctx[n]) + i - cu[n]
            e = table[n][pos // ps]
            slot[i] = e * ps + pos % ps if 0 <= e < P else -1
    return table, first, stack, top, cu, slot


class Batch:
    """A random paged batch on the CPU: consistent tables, pages of every sequence scattered over the
    pool, and NaN wherever no token of the batch's sequences is stored."""

    def __init__(self, dtype, H, dk, dv, W, S, ps, ctx, lens, pad=0, seed=0, slack=1, keep_behind=False):
        g = torch.Generator().manual_seed(seed)
        dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
        rnd = lambda *s: torch.randn(*s, generator=g).to(dt)
        N = len(ctx)
        self.dt, self.H, self.dk, self.dv, self.W, self.S, self.ps = dt, H, dk, dv, W, S, ps
        self.max_pages = max(-(-(c + m) // ps) for c, m in zip(ctx, lens)) + slack
        held = []
        for c, m in zip(ctx, lens):
            low = 0 if keep_behind else max(0, c - W + 1) // ps
            held.append([p for p in range(-(-(c + m) // ps)) if p >= low or p < -(-S // ps)])
        self.P = sum(map(len, held)) + 2
        perm = torch.randperm(self.P, generator=g).tolist()
        self.table = torch.full((N, self.max_pages), -1, dtype=torch.int32)
        self.k_pool = torch.full((self.P, ps, dk), math.nan, dtype=dt)
        self.v_pool = torch.full((self.P, H, ps, dv), math.nan, dtype=dt)
        M = sum(lens) + pad
        self.slot = torch.full((M,), -1, dtype=torch.int32)
        cu = [0]
        for n, (c, m) in enumerate(zip(ctx, lens)):
            for p in held[n]:
                e = perm.pop()
                self.table[n, p] = e
                have = max(0, min(ps, c - p * ps))  # cached tokens of the page
                self.k_pool[e, :have] = rnd(have, dk)
                self.v_pool[e, :, :have] = rnd(H, have, dv)
            for i in range(m):
                self.slot[cu[-1] + i] = int(self.table[n, (c + i) // ps]) * ps + (c + i) % ps
            cu.append(cu[-1] + m)
        self.cu = torch.tensor(cu, dtype=torch.int32)
        self.ctx = torch.tensor(ctx, dtype=torch.int64)
        self.q, self.k_new, self.v_new = 2 * rnd(M, H, dk), rnd(M, dk), rnd(M, H, dv)
        self.o = torch.full((M, H, dv), 7.0, dtype=dt)
        self.max_len = max(lens)

    def args(self, device):
        return [t.to(device) for t in (self.q, self.k_new, self.v_new, self.k_pool, self.v_pool, self.table, self.slot,
                                       self.cu, self.ctx)]

    def reference(self, **kw):
        return extend(self.q, self.k_new, self.v_new, self.k_pool, self.v_pool, self.table, self.slot, self.cu, self.ctx,
                      self.W, self.S, self.o, **kw)

    def terms(self):
        return min(self.W + self.S, int(self.ctx.max()) + self.max_len) + 1
