"""Calls of the serving operators that have to be refused before anything is enqueued, on the CPU:
a call that passes validation here ends with MSA_ERR_CUDA (3) instead."""
import pytest

from tests.test_serving_abi import _attn, _call_append, _call_attn, _lib, _rope


@pytest.mark.parametrize("B", [(1 << 31) - 1, (1 << 31) - 255])
def test_append_of_too_many_sequences(B):
    """The check of the call and the search for a token's sequence step through B + 1 offsets in
    32-bit numbers, which would run past 2^31."""
    assert _call_append(_rope(), B=B) == 2
