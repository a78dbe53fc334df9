"""Calls of the serving operators that have to be refused before anything is enqueued, on the CPU:
a call that passes validation here ends with MSA_ERR_CUDA (3) instead."""
import pytest

from tests.test_serving_abi import _attn, _call_append, _call_attn, _call_rope, _lib, _rope


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


# Memory far apart: every operand 2^36 bytes from the next.
FAR = {name: (k + 1) << 36 for k, name in enumerate(
    ("Q", "K", "V", "a", "b", "c", "O", "lse", "ws", "qo", "ko", "kc", "vc", "xc", "x", "pos", "f",
     "cu"))}
# Slices of one fused tensor [100, 8 + 2 + 2, 128] bf16: token t's queries, keys and values.
FUSED = dict(q_stride=12 * 128, k_stride=12 * 128, v_stride=12 * 128)
AT = FAR["Q"]
SLICES = dict(Q=AT, K=AT + 8 * 256, V=AT + 10 * 256)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("out", ["O", "lse", "ws"])
def test_attention_outputs_inside_other_memory(paged, out):
    """O, lse or the workspace anywhere inside an input or one another, not at equal addresses
    alone: the first and the last bytes, and inside a fused tensor that Q, K and V are slices of."""
    base = {k: FAR[k] for k in ("Q", "K", "V", "a", "b", "c", "O", "lse", "ws")}
    p = _attn()
    need = _lib().lib.msa_attn_workspace_size(p, int(paged))
    size = dict(O=100 * 8 * 256, lse=100 * 8 * 4, ws=need, Q=100 * 8 * 256, K=100 * 2 * 256,
                V=100 * 2 * 256, a=16, b=12, c=3 * 8 * 4)
    if paged:
        size.update(K=64 * 16 * 2 * 256, V=64 * 16 * 2 * 256)
    step = 256                                          # every alignment that is asked for
    for name in base:
        if name == out or (name == "c" and not paged):
            continue
        ends = [-((size[out] - 1) // step * step)]       # out's last bytes on the first of name
        ends += [(size[name] - 1) // step * step, size[name] // 2 // step * step]
        for at in ends:
            assert _call_attn(p, paged, **{**base, out: base[name] + at}) == 1, (name, at)
    if not paged:
        for at in (0, 256, 8 * 256, 11 * 256, 99 * 12 * 256):
            assert _call_attn(_attn(**FUSED), paged, **{**base, **SLICES, out: AT + at}) == 1, at


@pytest.mark.parametrize("kw", [
    dict(qo=FAR["Q"] + 256), dict(qo=FAR["Q"] - 256), dict(qo=FAR["K"]), dict(ko=FAR["Q"]),
    dict(ko=FAR["K"] + 9 * 512), dict(ko=FAR["qo"] + 9 * 2048 + 1536), dict(qo=FAR["pos"]),
    dict(ko=FAR["f"]), dict(qo=FAR["f"] - 256)])
def test_rope_outputs_inside_other_memory(kw):
    base = {k: FAR[k] for k in ("Q", "K", "pos", "f", "qo", "ko")}
    assert _call_rope(_rope(), **{**base, **kw}) == 1
    # fused [10, 12, 128]: in place at the wrong slice, or with another stride
    f = dict(q_stride=12 * 128, k_stride=12 * 128)
    slices = dict(base, Q=AT, K=AT + 8 * 256)
    for p, at in ((_rope(**f, q_out_stride=12 * 128), dict(qo=AT + 256)),
                  (_rope(**f, q_out_stride=12 * 128), dict(qo=AT + 10 * 256)),
                  (_rope(**f, k_out_stride=12 * 128), dict(ko=AT + 7 * 256)),
                  (_rope(**f), dict(qo=AT + 12 * 256)),
                  (_rope(**f, k_out_stride=24 * 128), dict(ko=AT + 8 * 256)),
                  (_rope(**f, q_out_stride=12 * 128, k_out_stride=24 * 128),
                   dict(qo=AT, ko=AT + 12 * 256))):
        assert _call_rope(p, **{**slices, **at}) == 1, at


@pytest.mark.parametrize("kw", [
    dict(qo=FAR["Q"] + 256), dict(qo=FAR["K"]), dict(qo=FAR["V"] + 512), dict(qo=FAR["x"]),
    dict(qo=FAR["kc"] + 99 * 16 * 512), dict(kc=FAR["K"]), dict(vc=FAR["V"] - 256),
    dict(vc=FAR["kc"]), dict(vc=FAR["kc"] + 100 * 16 * 512 - 256), dict(xc=FAR["vc"] + 1024),
    dict(kc=FAR["Q"]), dict(xc=FAR["x"] + 128), dict(ws=FAR["kc"] + 256), dict(ws=FAR["cu"])])
def test_append_outputs_inside_other_memory(kw):
    base = {k: FAR[k] for k in ("Q", "K", "V", "x", "qo", "kc", "vc", "xc", "ws", "cu")}
    assert _call_append(_rope(), **{**base, **kw}) == 1
