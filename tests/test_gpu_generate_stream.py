"""The generation loop on a stream of the caller's: states, positions and kernels all run on it."""
import pytest
import torch

from sliding_window_attention_chunked_b200 import workloads as wl
from sliding_window_attention_chunked_b200.generate import MixerStack

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _run(stream):
    L, N, H, T, d, W = 2, 2, 3, 40, 64, 16
    stack = MixerStack(L, N, H, d, W, device=DEV)
    ins = [wl.gla_inputs(N, H, T, d, d, dist="l2", seed=1, device=DEV), wl.swska_inputs(N, H, T, d, d, seed=2, device=DEV)]
    for lay in stack.layers:  # a state that the prefill has to clear, inputs that the steps use
        for n, t in lay.items():
            if n not in ("g",):
                t.copy_(torch.linspace(-1, 1, t.numel(), device=DEV).reshape(t.shape))
    torch.cuda.synchronize()
    if stream is not None:
        with torch.cuda.stream(stream):
            torch.cuda._sleep(30_000_000)
    outs = stack.prefill(ins, stream=stream)
    for _ in range(3):
        stack.step_eager(stream=stream)
    torch.cuda.synchronize()
    return [*outs, stack.pos, *(t for lay in stack.layers for t in lay.values())]


def test_stack_on_a_stream_that_is_late():
    for x, y in zip(_run(None), _run(torch.cuda.Stream())):
        assert torch.equal(x, y)
