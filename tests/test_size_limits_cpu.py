"""Sizes near the end of 32 bits are refused, not wrapped around."""

import pytest

from sequence_exact_attention_gb300 import binding

TOP = 2 ** 31 - 1
RANGE = 10


def refused(fn, *args, **kw):
    with pytest.raises(binding.RingAttnError) as e:
        fn(*args, **kw)
    assert e.value.status == RANGE


@pytest.mark.parametrize("B,H_q", [(TOP, 8), (TOP, TOP), (2 ** 20, 2 ** 12), (3, 2 ** 30)])
def test_batches_times_heads(lib, B, H_q):
    refused(binding.bwd_workspace_bytes, B, H_q, 100, 128, 1)
    refused(binding.bwd_window_workspace_bytes, B, H_q, H_q, 100, 128, 1, 10, 2)


@pytest.mark.parametrize("P,order", [(1, "contiguous"), (1, "zigzag"), (8, "contiguous"), (2 ** 30, "zigzag"),
                                     (TOP, "contiguous"), (TOP, "zigzag")])
@pytest.mark.parametrize("S", [TOP, TOP - 100, 2 ** 31 - 127])
def test_lengths(lib, S, P, order):
    refused(binding.bwd_workspace_bytes, 1, 1, S, 128, P, order)
    refused(binding.bwd_window_workspace_bytes, 1, 1, 1, S, 64, P, 10, 2, order, varlen=True)


def test_the_largest_that_fit(lib):
    # whole tiles of rows, two floats a row
    for S in (2 ** 31 - 128, 2 ** 31 - 129, 2 ** 31 - 256):
        want = 2 * 4 * -(-S // 128) * 128
        assert binding.bwd_workspace_bytes(1, 1, S, 128, 1) == want
        assert binding.bwd_window_workspace_bytes(1, 1, 1, S, 128, 1, 10) >= want
