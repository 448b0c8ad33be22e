"""Numbers that do not fit the C entries' ints are refused on the host: ctypes would keep their low 32 bits without a word."""
import pytest
import torch

import sliding_window_attention_chunked_b200 as rod
from sliding_window_attention_chunked_b200 import build as rbuild

z = torch.zeros
I32, I64 = torch.int32, torch.int64
FAR = [2 ** 31, 2 ** 32 + 4, -2 ** 32 + 4, 10 ** 15]


@pytest.fixture(scope="module", autouse=True)
def lib():
    rbuild.build()


def prefill(window=4, sinks=2):
    rod.swska_sink_prefill(z(1, 2, 8, 16), z(1, 8, 16), z(1, 2, 8, 32), window, sinks)


def backward(window=4, sinks=2):
    rod.swska_sink_backward(z(1, 2, 8, 16), z(1, 8, 16), z(1, 2, 8, 32), z(1, 2, 8, 32), z(1, 2, 8), z(1, 2, 8, 32), window, sinks)


def extend(window=4, sinks=2):
    rod.swska_extend_paged(z(1, 2, 16), None, None, z(1, 8, 16), z(1, 2, 8, 16), z(1, 1, dtype=I32), None, z(2, dtype=I32), z(1, dtype=I64),
                           window, sinks)


def tables(window=4, sinks=2, page_size=8):
    i = z(1, dtype=I32)
    rod.swska_page_tables(z(1, dtype=I64), i, z(1, 1, dtype=I32), i, i, i, page_size, window, sinks, 1)


@pytest.mark.parametrize("call", [prefill, backward, extend, tables])
def test_sizes_past_32_bits_are_refused(call):
    names = ["window", "sinks"] + ["page_size"] * (call is tables)
    for name in names:
        for x in FAR:
            with pytest.raises(ValueError, match=f"{name} must be below"):
                call(**{name: x})
        with pytest.raises(ValueError, match="CUDA"):  # the largest that fits goes on to the next check
            call(**{name: 2 ** 31 - 1})
