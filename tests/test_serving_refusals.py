"""Which check of the serving operators' Python calls refuses a call: each message, and nothing
gets as far as the library (tensors on the CPU would be refused there anyway, by another check)."""
import pytest
import torch

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def calls(monkeypatch):
    """The binding, with the step that hands a call to the library in sight."""
    from block_sparse_long_03_b200 import binding
    seen = []
    monkeypatch.setattr(binding, "_on_device", lambda where, *a: seen.append(where))
    binding.reached = seen
    yield binding
    del binding.reached


def _refused(b, match, call):
    with pytest.raises(b.MsaError, match=match) as e:
        call()
    assert e.value.status == 1 and not b.reached


def _rope(b, **kw):
    a = dict(Q=torch.zeros((4, 2, 64), dtype=BF16), K=torch.zeros((4, 1, 64), dtype=BF16),
             positions=torch.zeros(4, dtype=torch.int32),
             inv_freq=torch.ones(32, dtype=torch.float64))
    a.update(kw)
    return b.rope(a.pop("Q"), a.pop("K"), a.pop("positions"), a.pop("inv_freq"), **a)


def test_rope_reaches_the_library(calls):
    q, k = _rope(calls)
    assert calls.reached == ["rope"] and q.shape == (4, 2, 64) and k.shape == (4, 1, 64)


@pytest.mark.parametrize("kw,match", [
    (dict(Q=None, K=None), "Q and K are both None"),
    (dict(positions=torch.zeros(4, dtype=torch.int64)), "positions must be dense torch.int32"),
    (dict(positions=torch.zeros(3, dtype=torch.int32)), "positions must be dense"),
    (dict(positions=torch.zeros(8, dtype=torch.int32)[::2]), "positions must be dense"),
    (dict(positions=torch.zeros(4, dtype=torch.int32, device="meta")), "positions must be dense"),
    (dict(inv_freq=torch.ones(32)), "inv_freq must be dense float64"),
    (dict(inv_freq=torch.ones((1, 32), dtype=torch.float64)), "inv_freq must be dense"),
    (dict(inv_freq=torch.ones(64, dtype=torch.float64)[::2]), "inv_freq must be dense"),
    (dict(inv_freq=torch.ones(32, dtype=torch.float64, device="meta")), "inv_freq must be dense"),
    (dict(layout="pairs"), "layout 'pairs'"),
    (dict(K=torch.zeros((4, 1, 64))), "K: dtype or device"),
    (dict(K=torch.zeros((4, 1, 64), dtype=BF16, device="meta")), "K: dtype or device"),
    (dict(K=torch.zeros((3, 1, 64), dtype=BF16)), "K: shape"),
    (dict(K=torch.zeros((4, 1, 128), dtype=BF16)), "K: shape"),
    (dict(K=torch.zeros((4, 64), dtype=BF16)), "K must be .tokens, heads, d."),
    (dict(Q=torch.zeros((4, 2, 64), dtype=torch.float16)), "Q: dtype torch.float16"),
    (dict(Q=torch.zeros((1, 2, 64), dtype=BF16).expand(4, 2, 64)), "Q: expanded over tokens"),
    (dict(Q=torch.zeros((4, 64, 2), dtype=BF16).transpose(1, 2)), "a token's heads must be dense"),
    (dict(Q=torch.zeros((4, 4, 64), dtype=BF16)[:, ::2]), "a token's heads must be dense"),
    (dict(Q=torch.zeros((4, 2, 128), dtype=BF16)[..., ::2]), "a token's heads must be dense"),
    (dict(Q_out=torch.zeros((4, 2, 128), dtype=BF16)), "Q_out: shape"),
    (dict(Q_out=torch.zeros((4, 2, 64))), "Q_out: dtype or device"),
    (dict(K_out=torch.zeros((3, 1, 64), dtype=BF16)), "K_out: shape"),
])
def test_rope(calls, kw, match):
    _refused(calls, match, lambda: _rope(calls, **kw))


def _packed(b, **kw):
    a = dict(Q=torch.zeros((4, 2, 64), dtype=BF16), K=torch.zeros((6, 1, 64), dtype=BF16),
             V=torch.zeros((6, 1, 64), dtype=BF16), cu=torch.tensor([0, 4], dtype=torch.int32),
             ck=torch.tensor([0, 6], dtype=torch.int32))
    a.update(kw)
    return b.attn_packed(a.pop("Q"), a.pop("K"), a.pop("V"), a.pop("cu"), a.pop("ck"), **a)


def _paged(b, **kw):
    a = dict(Q=torch.zeros((4, 2, 64), dtype=BF16), K=torch.zeros((2, 16, 1, 64), dtype=BF16),
             V=torch.zeros((2, 16, 1, 64), dtype=BF16), cu=torch.tensor([0, 4], dtype=torch.int32),
             lens=torch.tensor([6], dtype=torch.int32), table=torch.zeros((1, 1), dtype=torch.int32))
    a.update(kw)
    return b.attn_paged(a.pop("Q"), a.pop("K"), a.pop("V"), a.pop("cu"), a.pop("lens"),
                        a.pop("table"), **a)


def test_attention_reaches_the_library(calls):
    O, lse, _ = _packed(calls)
    assert O.shape == (4, 2, 64) and lse.shape == (4, 2)
    _paged(calls)
    assert calls.reached == ["attn_packed", "attn_paged"]


COMMON = [
    (dict(Q=torch.zeros((4, 64), dtype=BF16)), "Q must be .tokens, heads, d."),
    (dict(Q=torch.zeros((4, 4, 64), dtype=BF16)[:, ::2]), "a token's heads must be dense"),
    (dict(Q=torch.zeros((1, 2, 64), dtype=BF16).expand(4, 2, 64)), "Q: expanded over tokens"),
    (dict(cu=torch.tensor([0, 4])), "cu_seqlens must be dense torch.int32"),
    (dict(cu=torch.tensor([[0, 4]], dtype=torch.int32)), "cu_seqlens must be dense"),
    (dict(cu=torch.tensor([0, 9, 4, 9], dtype=torch.int32)[::2]), "cu_seqlens must be dense"),
    (dict(cu=torch.empty(2, dtype=torch.int32, device="meta")), "cu_seqlens must be dense"),
    (dict(out=torch.zeros((4, 2, 64))), "out must be dense"),
    (dict(out=torch.zeros((4, 4, 64), dtype=BF16)[:, :2]), "out must be dense"),
    (dict(out=torch.zeros((4, 2, 64), dtype=BF16, device="meta")), "out must be dense"),
    (dict(lse=torch.zeros((4, 2), dtype=BF16)), "lse must be dense torch.float32"),
    (dict(lse=torch.zeros((2, 4)).t()), "lse must be dense"),
    (dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8, device="meta")), "workspace must be dense"),
    (dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8)[::2]), "workspace must be dense"),
]


@pytest.mark.parametrize("call", [_packed, _paged])
@pytest.mark.parametrize("kw,match", COMMON)
def test_attention(calls, call, kw, match):
    _refused(calls, match, lambda: call(calls, **kw))


@pytest.mark.parametrize("kw,match", [
    (dict(V=torch.zeros((5, 1, 64), dtype=BF16)), "K, V: shape"),
    (dict(K=torch.zeros((6, 1, 128), dtype=BF16), V=torch.zeros((6, 1, 128), dtype=BF16)),
     "K, V: shape"),
    (dict(K=torch.zeros((6, 1, 64))), "K: dtype or device"),
    (dict(V=torch.zeros((6, 1, 64), dtype=BF16, device="meta")), "V: dtype or device"),
    (dict(K=torch.zeros((6, 1, 128), dtype=BF16)[..., ::2]), "K: a token's heads must be dense"),
    (dict(ck=torch.tensor([0], dtype=torch.int32)), "cu_seqlens_k must be dense"),
    (dict(ck=torch.tensor([0, 6])), "cu_seqlens_k must be dense"),
])
def test_packed_attention(calls, kw, match):
    _refused(calls, match, lambda: _packed(calls, **kw))


CACHES = [
    (dict(K=torch.zeros((32, 1, 64), dtype=BF16)), "K_cache must be .num_pages"),
    (dict(K=torch.zeros((2, 16, 2, 64), dtype=BF16)[:, :, ::2]), "K_cache must be dense"),
    (dict(K=torch.zeros((2, 16, 1, 64))), "K_cache must be dense"),
    (dict(V=torch.zeros((2, 8, 1, 64), dtype=BF16)), "V_cache must be dense"),
    (dict(V=torch.zeros((2, 16, 1, 64), dtype=BF16, device="meta")), "V_cache must be dense"),
    (dict(lens=torch.tensor([6])), "seq_lens must be dense torch.int32"),
    (dict(lens=torch.tensor([6, 1], dtype=torch.int32)), "seq_lens must be dense"),
    (dict(table=torch.zeros(1, dtype=torch.int32)), "block_table .B, max_pages."),
    (dict(table=torch.zeros((2, 1), dtype=torch.int32)), "block_table must be dense"),
    (dict(table=torch.zeros((1, 1), dtype=torch.int64)), "block_table must be dense torch.int32"),
]


@pytest.mark.parametrize("kw,match", CACHES + [
    (dict(K=torch.zeros((2, 16, 1, 32), dtype=BF16), V=torch.zeros((2, 16, 1, 32), dtype=BF16)),
     "K_cache: head dimension")])
def test_paged_attention(calls, kw, match):
    _refused(calls, match, lambda: _paged(calls, **kw))


def _append(b, **kw):
    a = dict(q=torch.zeros((4, 2, 64), dtype=BF16), k=torch.zeros((4, 1, 64), dtype=BF16),
             v=torch.zeros((4, 1, 64), dtype=BF16), x=torch.zeros((4, 32), dtype=BF16),
             cu=torch.tensor([0, 4], dtype=torch.int32), lens=torch.tensor([6], dtype=torch.int32),
             table=torch.zeros((1, 1), dtype=torch.int32), f=torch.ones(32, dtype=torch.float64),
             K=torch.zeros((2, 16, 1, 64), dtype=BF16), V=torch.zeros((2, 16, 1, 64), dtype=BF16),
             X=torch.zeros((2, 16, 32), dtype=BF16))
    a.update(kw)
    args = [a.pop(n) for n in ("q", "k", "v", "x", "cu", "lens", "table", "f", "K", "V", "X")]
    return b.rope_append_paged(*args, **a)


def test_append_reaches_the_library(calls):
    _append(calls)
    assert calls.reached == ["rope_append_paged"]


@pytest.mark.parametrize("kw,match", CACHES + [
    (dict(k=None), "K and V are needed"), (dict(v=None), "K and V are needed"),
    (dict(v=torch.zeros((3, 1, 64), dtype=BF16)), "V or the caches: shape"),
    (dict(v=torch.zeros((4, 1, 64))), "V: dtype or device"),
    (dict(K=torch.zeros((2, 16, 2, 64), dtype=BF16), V=torch.zeros((2, 16, 2, 64), dtype=BF16)),
     "V or the caches: shape"),
    (dict(x=None), "k_idx and k_idx_cache go together"), (dict(X=None), "go together"),
    (dict(x=torch.zeros((3, 32), dtype=BF16)), "k_idx must be dense"),
    (dict(x=torch.zeros((4, 64), dtype=BF16)[:, ::2]), "k_idx must be dense"),
    (dict(X=torch.zeros((2, 16, 64), dtype=BF16)), "k_idx_cache must be dense"),
    (dict(cu=torch.tensor([0, 4])), "cu_seqlens must be dense"),
    (dict(Q_out=torch.zeros((4, 2, 128), dtype=BF16)), "Q_out: shape"),
    (dict(workspace=torch.zeros(256, dtype=torch.uint8, device="meta")), "workspace must be dense"),
])
def test_append(calls, kw, match):
    _refused(calls, match, lambda: _append(calls, **kw))


def test_cpu_tensors_are_refused():
    from block_sparse_long_03_b200 import binding as b
    b.reached = []
    for call in (_rope, _packed, _paged, _append):
        _refused(b, "must be on a CUDA device", lambda: call(b))
    del b.reached
