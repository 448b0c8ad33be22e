"""What the row-norm tolerances catch: rounded results pass, a key too many or too few in a window of 4096 does not. On the CPU,
with the mistakes in the reference's mask."""
import math

import pytest
import torch

from . import row_norms as rn
from . import sink_ref as ref

W, S, D = 4096, 4, 128


def _head(seed, n_q=6, first=4200):
    g = torch.Generator().manual_seed(seed)
    T = first + n_q
    rnd = lambda *s: torch.randn(*s, generator=g)
    q = (0.1 * rnd(n_q, D)).bfloat16().double()
    k, v, dO = (rnd(n, D).bfloat16().double() for n in (T, T, n_q))
    p, j = torch.arange(first, T), torch.arange(T)
    return q, k, v, dO, p, j


def _rounded(q, k, v, see, scale):
    """The forward with the kernels' roundings: probabilities and the output to bf16."""
    s = torch.where(see, (q @ k.T) * scale, -math.inf)
    e = torch.exp(s - s.max(1, keepdim=True).values)
    return ((e.bfloat16().double() @ v) / e.sum(1, keepdim=True)).bfloat16()


@pytest.mark.parametrize("seed", range(5))
def test_forward_rows(seed):
    q, k, v, _, p, j = _head(seed)
    see, scale = ref.visible(p, j, W, S), D ** -0.5
    o, tol = rn.forward(q, k, v, see, scale, torch.bfloat16, ref.amp(q, k))
    assert not rn.off(_rounded(q, k, v, see, scale), o, tol).any()
    for wrong in ((W - 1, S), (W + 1, S), (W, S - 1), (W, S + 1), (W, 0)):
        assert rn.off(_rounded(q, k, v, ref.visible(p, j, *wrong), scale), o, tol).all(), wrong
    behind = see & (j[None, :] < p[:, None])  # a query that misses its own key
    assert rn.off(_rounded(q, k, v, behind, scale), o, tol).all()


@pytest.mark.parametrize("seed", range(3))
def test_gradient_rows(seed):
    q, k, v, dO, p, j = _head(seed, n_q=40)
    see, scale = ref.visible(p, j, W, S), D ** -0.5
    want = rn.gradients(q, k, v, dO, see, scale, torch.bfloat16, ref.amp(q, k))

    def rounded(see):
        s = torch.where(see, (q @ k.T) * scale, -math.inf)
        pr = torch.softmax(s, 1)
        o = _rounded(q, k, v, see, scale).double()
        dS = (pr * (dO @ v.T - (dO * o).sum(1, keepdim=True))).bfloat16().double()
        return (dS @ k * scale).bfloat16()

    dq, tol = want["dq"]
    assert not rn.off(rounded(see), dq, tol).any()
    for wrong in ((W - 1, S), (W + 1, S), (W, 0)):
        assert rn.off(rounded(ref.visible(p, j, *wrong)), dq, tol).float().mean() > 0.4, wrong  # a key whose dP is near D adds little
