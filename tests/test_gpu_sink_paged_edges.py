"""Edges of the SW-SKA operators with first tokens that stay visible, of the paged attention of new tokens and of the page
tables."""
import pytest
import torch

import sliding_window_attention_chunked_b200 as rod
from sliding_window_attention_chunked_b200 import workloads as wl

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
