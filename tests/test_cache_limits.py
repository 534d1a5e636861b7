"""Sizes at which the cache calls' own arithmetic would end, on the CPU: the calls are refused."""
import pytest
import torch

from test_cache_checks import CUDA, INVALID, _decode, _read, _write

FAR = dict(table=1 << 50, offsets=1 << 51, start=1 << 52, seq=1 << 53)  # no two of these buffers overlap


@pytest.mark.parametrize("call", [_write, _read, _decode])
def test_sequences_are_counted_in_30_bits(call):
    """A warp's search over B sequences rounds B up to a multiple of 32 in 32 bits: from 2^31 - 31 on
    it would have read in front of the offsets."""
    assert call(B=1 << 30, **FAR) == INVALID
    assert call(B=(1 << 31) - 1, **FAR) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="with a GPU the call would launch on fake addresses")
@pytest.mark.parametrize("call", [_read, _decode])
def test_the_most_sequences_pass_the_checks(call):
    assert call(B=(1 << 30) - 1, **FAR) == CUDA  # it ends at the device lookup
