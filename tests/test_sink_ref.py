"""The references of sink_ref.py against differences, against the framework's oracle, and their own invariants (CPU)."""
import math

import numpy as np
import pytest
import torch

import oracle

from . import sink_ref as ref


@pytest.mark.parametrize("T,W,S", [(9, 3, 2), (7, 20, 1), (12, 1, 4), (5, 2, 9)])
def test_gradients_against_differences(T, W, S):
    g = torch.Generator().manual_seed(T)
    B, H, d, e = 1, 2, 4, 3
    q, k, v, dO = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((B, H, T, d), (B, T, d), (B, H, T, e), (B, H, T, e)))
    r = ref.train(q, k, v, dO, W, S)
    loss = lambda *a: float((ref.train(*a, dO, W, S)["o"][0] * dO).sum())
    for i, name in enumerate(("dq", "dk", "dv")):
        x = [q, k, v][i]
        for at in [tuple(np.random.RandomState(s).randint(0, n) for n in x.shape) for s in range(6)]:
            h = 1e-5
            up, dn = x.clone(), x.clone()
            up[at] += h
            dn[at] -= h
            a = [q, k, v]
            diff = (loss(*(a[:i] + [up] + a[i + 1:])) - loss(*(a[:i] + [dn] + a[i + 1:]))) / (2 * h)
            # central difference: truncation of order h^2 = 1e-10, rounding 1e-16 / h = 1e-11 of the loss
            assert abs(diff - float(r[name][0][at])) < 1e-7


def test_without_first_tokens_it_is_the_sliding_window():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(*s, generator=g) for s in ((2, 3, 40, 16), (2, 40, 16), (2, 3, 40, 32)))
    o = ref.train(q, k, v, torch.zeros_like(v), 7, 0)["o"][0]
    np.testing.assert_allclose(o.numpy(), oracle.swska_prefill(q, k, v, 7), rtol=1e-12, atol=1e-12)


def test_paged_reference_is_the_contiguous_one():
    """Whole prompts as one chunk, and as chunks of one token, give the contiguous rows."""
    T, W, S, ps, H = 50, 11, 3, 8, 2
    b = ref.Batch("fp32", H, 16, 16, W, S, ps, [0], [T])
    o, _, kp, vp = b.reference()
    see = ref.train(b.q.transpose(0, 1)[None], b.k_new[None], b.v_new.transpose(0, 1)[None], torch.zeros(1, H, T, 16), W, S)["o"][0]
    torch.testing.assert_close(o, see[0].transpose(0, 1), rtol=1e-12, atol=1e-12)
    one, _, _, _ = ref.extend(b.q[-1:], None, None, kp, vp, b.table, None, torch.tensor([0, 1]), torch.tensor([T - 1]), W, S, b.o[-1:])
    torch.testing.assert_close(one[0], o[-1], rtol=1e-12, atol=1e-12)


def test_page_tables_reference_keeps_every_page():
    """Pages are neither lost nor handed out twice over a long random run."""
    r = np.random.RandomState(3)
    N, mp, P, ps, W, S = 5, 40, 60, 8, 37, 9
    table, first, stack, top = [[-1] * mp for _ in range(N)], [0] * N, list(range(P)), P
    ctx = [0] * N
    for _ in range(200):
        new = [int(r.choice([0, 1, 1, 5, 30])) if r.rand() > 0.05 else -1 for _ in range(N)]
        new = [-1 if c > 250 else m for c, m in zip(ctx, new)]
        table, first, stack, top, cu, slot = ref.page_tables(ctx, new, table, first, stack, top, ps, W, S, 100)
        for n in range(N):
            ctx[n] = 0 if new[n] < 0 else ctx[n] + cu[n + 1] - cu[n]
        held = [e for row in table for e in row if e >= 0]
        assert sorted(held + stack[:top]) == list(range(P))
        assert len(set(s for s in slot if s >= 0)) == cu[-1]
        for n in range(N):  # what the next query sees is there
            need = set(range(min(S, ctx[n]))) | set(range(max(0, ctx[n] - W + 1), ctx[n]))
            assert all(table[n][j // ps] >= 0 for j in need)
