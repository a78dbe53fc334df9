"""Calls of the serving operators that have to be refused before anything is enqueued, on the CPU:
a call that passes validation here ends with MSA_ERR_CUDA (3) instead."""
import pytest

from tests.test_serving_abi import _attn, _call_append, _call_attn, _lib, _rope


@pytest.mark.parametrize("B", [(1 << 31) - 1, (1 << 31) - 255])
def test_append_of_too_many_sequences(B):
    """The check of the call and the search for a token's sequence step through B + 1 offsets in
    32-bit numbers, which would run past 2^31."""
    assert _call_append(_rope(), B=B) == 2


@pytest.mark.parametrize("paged,name", [(False, "q_stride"), (False, "k_stride"),
                                        (False, "v_stride"), (True, "q_stride")])
def test_token_strides_past_a_tensor_map(paged, name):
    """bf16 tokens 2^40 bytes apart: a tensor map cannot describe them, and nothing may be enqueued
    before that is found.  fp32 reads them with plain loads."""
    for stride in (1 << 39, 1 << 45, 1 << 58):
        p = _attn(tokens=1, key_tokens=1, **{name: stride})
        assert _call_attn(p, paged) == 2
        assert _lib().lib.msa_attn_workspace_size(p, int(paged)) == 0
    p = _attn(tokens=1, key_tokens=1, **{name: (1 << 39) - 8})
    assert _lib().lib.msa_attn_workspace_size(p, int(paged)) > 0
    p = _attn(tokens=1, key_tokens=1, dtype=0, **{name: 1 << 39})
    assert _lib().lib.msa_attn_workspace_size(p, int(paged)) > 0
