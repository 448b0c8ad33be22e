"""Tolerances for the norm of an output row over wide windows, where the element bounds of sink_ref.py (a worst case: every
rounding at its largest and of one sign) would let a lost or an extra key pass.

A rounding to a type with half step h (bf16 2^-8) is off by a uniformly spread error of at most h 2^e for a value in [2^e,
2^(e+1)): its square is at most h^2 / 3 of the value's on average. Roundings of different terms are independent where many terms
differ by more than a step (scores spread by about 0.1, hundreds of keys), so the squares add: a row x = sum_j w_j y_j with each w_j rounded
and x rounded once is off, in the square of its norm, by (h^2 / 3) r^2 with r^2 = |x|^2 + sum_j w_j^2 |y_j|^2 on average. A row has
at least 64 elements, whose squared errors scatter the norm by less than 10%: 1.5 times the average is five of that. 32-bit
work adds errors of sqrt(n + d) 2^-23 (1 + amp) r + 2^-20 r in the same way (n terms, dots of d, exponentials good to 2^-21;
2^-13 for the cubic of the tensor-core gradients). One key of n with equal weights is |y| / n of a row of |y| / sqrt(n): at n = 4096
1.6e-2, against a tolerance of 1.5 sqrt(2) 2^-8 / sqrt(3) = 4.8e-3 times that row."""
import math

import torch


def _norm2(x):
    return (x * x).sum(-1)


def tolerance(dtype, x, terms2, n, d, amp, poly=False):
    """For rows x [.., e] (64 bits) with terms2 = sum_j w_j^2 |y_j|^2 of each."""
    r = torch.sqrt(_norm2(x) + terms2)
    inner = math.sqrt(n + d) * 2.0 ** -23 * (1 + amp) + (2.0 ** -13 if poly else 2.0 ** -20)
    half = torch.finfo(dtype).eps / 2
    return (1.5 * half / math.sqrt(3) + 1.5 * inner) * r


def forward(q, k, v, see, scale, dtype, amp):
    """One head in 64 bits: (o, tolerance of each row's norm)."""
    s = torch.where(see, (q @ k.T) * scale, -math.inf)
    p = torch.softmax(s, 1)
    o = p @ v
    return o, tolerance(dtype, o, (p * p) @ _norm2(v), k.shape[0], q.shape[1], amp)


def gradients(q, k, v, dO, see, scale, dtype, amp):
    """One head in 64 bits: {name: (rows, tolerance)} for o, dq, dv, and for dk without its sum over the heads. bf16: D = dO . o is
    taken from the rounded o, an error that all dS of a row share."""
    s = torch.where(see, (q @ k.T) * scale, -math.inf)
    p = torch.softmax(s, 1)
    o = p @ v
    dP = dO @ v.T
    D = (dO * o).sum(1, keepdim=True)
    dS = p * (dP - D) * scale
    n, d, bf16 = k.shape[0], q.shape[1], dtype is torch.bfloat16
    err_D = 1.5 * torch.finfo(dtype).eps / 2 / math.sqrt(3) * torch.sqrt(_norm2(dO * o)) * scale  # of D, times the scale
    # 32 bits: dS is the difference of two sums of size |dP|, |D|, so the terms that its errors scale with are those
    big = dS if bf16 else p * (dP.abs() + D.abs()) * scale
    out = {"o": (o, tolerance(dtype, o, (p * p) @ _norm2(v), n, d, amp)),
           "dv": (p.T @ dO, tolerance(dtype, p.T @ dO, (p * p).T @ _norm2(dO), n, d, amp, poly=bf16))}
    dq, dk = dS @ k, dS.T @ q
    out["dq"] = dq, tolerance(dtype, dq, (big * big) @ _norm2(k), n, d, amp, poly=bf16) + err_D * torch.sqrt(_norm2(p @ k))
    out["dk"] = dk, tolerance(dtype, dk, (big * big).T @ _norm2(q), n, d, amp, poly=bf16) + torch.sqrt((p * p).T @ (err_D ** 2 * _norm2(q)))
    return out


def off(got, want, tol):
    """Rows whose error's norm is over the tolerance."""
    return torch.sqrt(_norm2(got.double().to(want.device) - want)) > tol
