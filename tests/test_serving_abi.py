"""The serving operators' refusals and host-side arithmetic, on the CPU: every call here fails
validation before any CUDA call, and no pointer is dereferenced."""
import ctypes
import math

import pytest
import torch

FAKE = 0x10000
ODD = 0x10008                       # 8-byte aligned only
WS = 0x20000


def _lib():
    from block_sparse_long_03_b200 import binding
    return binding


def _rope(**kw):
    b = _lib()
    base = dict(tokens=10, q_stride=0, k_stride=0, q_out_stride=0, k_out_stride=0, Hq=8, Hkv=2,
                d=128, rot_dim=64, layout=0, inverse=0, dtype=1, mscale=1.0)
    base.update(kw)
    return b.RopeParams(**base)


def _call_rope(p, Q=FAKE, K=FAKE, pos=FAKE, f=FAKE, qo=FAKE, ko=FAKE):
    return _lib().lib.msa_rope(p, Q, K, pos, f, qo, ko, None)


def _call_append(p, B=2, page=16, pages=8, num=100, Q=FAKE, K=FAKE, V=FAKE, vs=0, x=FAKE, d_idx=64,
                 qo=FAKE, kc=FAKE, vc=FAKE, xc=FAKE, ws=WS, n=256, cu=FAKE):
    return _lib().lib.msa_rope_append_paged(p, B, cu, FAKE, FAKE, page, pages, num, Q, K, V, vs, x,
                                            d_idx, FAKE, qo, kc, vc, xc, ws, n, None)


BAD_ROPE = [
    (dict(tokens=-1), 1), (dict(Hq=0), 1), (dict(Hkv=-2), 1), (dict(Hq=2000), 1), (dict(d=0), 1),
    (dict(rot_dim=0), 1), (dict(rot_dim=144), 1), (dict(layout=2), 1), (dict(inverse=2), 1),
    (dict(dtype=2), 1), (dict(mscale=math.nan), 1), (dict(mscale=math.inf), 1),
    (dict(q_stride=1000), 1), (dict(q_stride=1028), 1), (dict(k_out_stride=8), 1),
    (dict(q_stride=-1024), 1), (dict(d=72, rot_dim=64), 2), (dict(rot_dim=24), 2),
    (dict(d=272, rot_dim=64), 2), (dict(tokens=1 << 31), 2), (dict(q_stride=1 << 61), 1),
]


@pytest.mark.parametrize("kw,status", BAD_ROPE)
def test_rope_refusals(kw, status):
    assert _call_rope(_rope(**kw)) == status
    if "k_out_stride" not in kw:
        assert _call_append(_rope(**kw)) == status


def test_rope_pointer_refusals():
    p = _rope()
    assert _call_rope(None) == 1
    assert _call_rope(p, Q=None, K=None, qo=None, ko=None) == 1
    assert _call_rope(p, Q=None) == 1 and _call_rope(p, ko=None) == 1
    assert _call_rope(p, pos=None) == 1 and _call_rope(p, pos=FAKE + 2) == 1
    assert _call_rope(p, f=None) == 1 and _call_rope(p, f=FAKE + 4) == 1
    for name in ("Q", "K", "qo", "ko"):
        assert _call_rope(p, **{name: ODD}) == 1
    # in place needs one stride
    assert _call_rope(_rope(q_stride=2048, q_out_stride=1024), Q=FAKE, qo=FAKE) == 1


def test_append_refusals():
    p = _rope()
    for kw in (dict(B=0), dict(page=0), dict(pages=-1), dict(num=0), dict(K=None), dict(V=None),
               dict(kc=None), dict(vc=None), dict(x=None), dict(xc=None), dict(vs=8), dict(cu=None),
               dict(V=ODD), dict(vc=ODD), dict(x=ODD), dict(xc=ODD), dict(kc=ODD), dict(d_idx=0),
               dict(cu=FAKE + 1), dict(Q=None)):
        assert _call_append(p, **kw) == 1, kw
    assert _call_append(_rope(inverse=1)) == 1
    for kw in (dict(d_idx=24), dict(d_idx=144), dict(page=1 << 20, pages=1 << 20)):
        assert _call_append(p, **kw) == 2, kw
    for kw in (dict(ws=None), dict(n=255), dict(ws=WS + 16)):
        assert _call_append(p, **kw) == 5, kw


def _attn(**kw):
    b = _lib()
    base = dict(tokens=100, key_tokens=100, q_stride=0, k_stride=0, v_stride=0, B=3, Hq=8, Hkv=2,
                d=128, dtype=1, scale=0.0, page_size=16, max_pages=8, num_pages=64)
    base.update(kw)
    return b.AttnParams(**base)


def _call_attn(p, paged, Q=FAKE, K=FAKE, V=FAKE, a=FAKE, b=FAKE, c=FAKE, O=FAKE, lse=FAKE, ws=WS,
               n=1 << 40):
    lib = _lib().lib
    if paged:
        return lib.msa_attn_paged(p, Q, K, V, a, b, c, O, lse, ws, n, None)
    return lib.msa_attn_packed(p, Q, K, V, a, b, O, lse, ws, n, None)


BAD_ATTN = [
    (dict(tokens=-1), 1), (dict(B=0), 1), (dict(Hq=0), 1), (dict(Hq=7), 1), (dict(d=0), 1),
    (dict(dtype=3), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1), (dict(d=96), 2),
    (dict(Hq=130), 2), (dict(Hq=2048, Hkv=512), 2), (dict(B=1 << 21), 2), (dict(tokens=1 << 31), 2),
    (dict(q_stride=1000), 1), (dict(q_stride=1028), 1), (dict(tokens=(1 << 31) - 255), 2),
]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("kw,status", BAD_ATTN)
def test_attention_refusals(kw, status, paged):
    assert _call_attn(_attn(**kw), paged) == status
    assert _lib().lib.msa_attn_workspace_size(_attn(**kw), int(paged)) == 0


def test_attention_refusals_of_one_form():
    for kw, status in ((dict(key_tokens=-1), 1), (dict(key_tokens=1 << 31), 2),
                       (dict(k_stride=8), 1), (dict(v_stride=260), 1)):
        assert _call_attn(_attn(**kw), False) == status
    for kw, status in ((dict(page_size=0), 1), (dict(max_pages=0), 1), (dict(num_pages=-1), 1),
                       (dict(page_size=12), 2), (dict(num_pages=1 << 30), 2),
                       (dict(max_pages=1 << 30), 2)):
        assert _call_attn(_attn(**kw), True) == status
    assert _lib().lib.msa_attn_workspace_size(_attn(page_size=12, dtype=0), 1) > 0


@pytest.mark.parametrize("paged", [False, True])
def test_attention_pointer_and_workspace_refusals(paged):
    p = _attn()
    need = _lib().lib.msa_attn_workspace_size(p, int(paged))
    assert need >= 256
    assert _call_attn(None, paged) == 1
    names = ["Q", "K", "V", "a", "b", "O", "lse"] + (["c"] if paged else [])
    for name in names:
        assert _call_attn(p, paged, **{name: None}) == 1, name
        assert _call_attn(p, paged, **{name: FAKE + 2}) == 1, name
    for kw in (dict(ws=None), dict(ws=WS + 128), dict(n=need - 1)):
        assert _call_attn(p, paged, **kw) == 5, kw


def test_workspace_is_bounded():
    """The partial results of split keys stay within a few hundred MB at every size."""
    b = _lib()
    for tokens in (1, 64, 1000, 4096, 32768, 1 << 20):
        for Hq, Hkv in ((32, 8), (64, 4), (64, 1), (8, 8)):
            for paged in (0, 1):
                p = _attn(tokens=tokens, key_tokens=tokens, Hq=Hq, Hkv=Hkv, B=64, max_pages=1 << 16,
                          num_pages=1 << 20)
                n = b.lib.msa_attn_workspace_size(p, paged)
                assert 0 < n < (1 << 29) + (tokens << 2), (tokens, Hq, Hkv, paged, n)


FREQ = [(dict(rot_dim=0), 1), (dict(rot_dim=7), 1), (dict(base=1.0), 1), (dict(base=math.nan), 1),
        (dict(scaling="linear", factor=0.0), 1), (dict(scaling="base", factor=2.0, rot_dim=2), 1),
        (dict(scaling="parts", factor=4.0, slow=3.0, fast=2.0), 1),
        (dict(scaling="parts", factor=4.0, context=0.0), 1), (dict(scaling="other"), 1)]


@pytest.mark.parametrize("kw,status", FREQ)
def test_frequency_refusals(kw, status):
    b = _lib()
    with pytest.raises(b.MsaError) as e:
        b.rope_frequencies(**{"rot_dim": 64, "device": "cpu", **kw})
    assert e.value.status == status


def test_frequencies():
    """Against the formulas in fp64 (pow is good to an ulp or two)."""
    b = _lib()
    i = torch.arange(0, 64, 2, dtype=torch.float64)
    plain = 10000.0 ** (-i / 64)
    def same(x, y):
        assert bool(((x - y).abs() <= 1e-14 * y.abs()).all())
    same(b.rope_frequencies(64, device="cpu"), plain)
    same(b.rope_frequencies(64, scaling="linear", factor=8.0, device="cpu"), plain / 8)
    same(b.rope_frequencies(64, base=500000.0, scaling="base", factor=4.0, device="cpu"),
         (500000.0 * 4.0 ** (64 / 62)) ** (-i / 64))
    f = b.rope_frequencies(64, scaling="parts", factor=8.0, context=8192.0, slow=1.0, fast=4.0,
                           device="cpu")
    turns = 8192 * plain / (2 * math.pi)
    same(f[turns >= 4], plain[turns >= 4])
    same(f[turns <= 1], plain[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 4)
    assert bool(mid.any())
    w = (turns[mid] - 1) / 3
    assert bool(((f[mid] - (w + (1 - w) / 8) * plain[mid]).abs() <= 1e-12 * plain[mid]).all())


def test_python_refusals():
    """What the Python calls refuse before the library is called: shapes, dtypes, strides and
    devices that would be read wrongly."""
    b = _lib()
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    k = torch.zeros((4, 1, 64), dtype=torch.bfloat16)
    pos = torch.zeros(4, dtype=torch.int32)
    f = torch.ones(32, dtype=torch.float64)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    bad = [
        lambda: b.rope(None, None, pos, f),
        lambda: b.rope(x, k, pos.long(), f),
        lambda: b.rope(x, k, pos[:3], f),
        lambda: b.rope(x, k, pos, f.float()),
        lambda: b.rope(x, k, pos, f, layout="pairs"),
        lambda: b.rope(x, k.float(), pos, f),
        lambda: b.rope(x, k[:3], pos, f),
        lambda: b.rope(x.half(), None, pos, f),
        lambda: b.rope(x[:1].expand(4, 2, 64), None, pos, f),
        lambda: b.rope(x.transpose(1, 2), None, pos, f),
        lambda: b.rope(x, None, pos, f, Q_out=torch.zeros((4, 2, 128), dtype=x.dtype)),
        lambda: b.rope(x, k, pos, f),                               # not on a GPU
        lambda: b.attn_packed(x, k, k[:3], cu),
        lambda: b.attn_packed(x, k, k, cu.long()),
        lambda: b.attn_packed(x, k, k, cu, cu[:1]),
        lambda: b.attn_packed(x, k, k, cu),                         # not on a GPU
        lambda: b.attn_packed(x, k.expand(4, 2, 64)[:, :, ::2], k, cu),
        lambda: b.attn_paged(x, k, k, cu, pos[:1], pos.view(1, 4)),
        lambda: b.attn_paged(x, torch.zeros((2, 16, 1, 32), dtype=x.dtype),
                             torch.zeros((2, 16, 1, 32), dtype=x.dtype), cu, pos[:1],
                             pos.view(1, 4)),
        lambda: b.rope_append_paged(x, k, k, x[:, 0], cu, pos[:1], pos.view(1, 4), f,
                                    torch.zeros((2, 16, 1, 64), dtype=x.dtype),
                                    torch.zeros((2, 16, 1, 64), dtype=x.dtype)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(b.MsaError):
            call()
            raise AssertionError(f"call {i} was not refused")


@pytest.mark.parametrize("paged", [False, True])
def test_attention_output_over_an_input(paged):
    p = _attn()
    for name in ("Q", "K", "V", "lse"):
        kw = {"Q": 0x30000, "K": 0x40000, "V": 0x50000, "lse": 0x60000, "O": 0x70000}
        kw[name] = kw["O"]
        assert _call_attn(p, paged, **kw) == 1, name


def test_python_refuses_foreign_workspaces_and_missing_keys():
    """A workspace of another device or with gaps, and a cache write without K or V."""
    b = _lib()
    for ws in (torch.zeros(4096, dtype=torch.uint8), torch.zeros(4096, dtype=torch.uint8,
                                                                 device="meta")[::2]):
        with pytest.raises(b.MsaError) as e:
            b._workspace("call", ws, torch.device("meta"))
        assert e.value.status == 1
    b._workspace("call", torch.zeros(4096, dtype=torch.uint8, device="meta"),
                 torch.device("meta"))
    k = torch.zeros((4, 1, 64), dtype=torch.bfloat16)
    cache = torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    f = torch.ones(32, dtype=torch.float64)
    for K, V in ((None, k), (k, None)):
        with pytest.raises(b.MsaError):
            b.rope_append_paged(k, K, V, None, i, i[:1], i.view(1, 2), f, cache, cache)
