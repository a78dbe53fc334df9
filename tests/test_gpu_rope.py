"""Rotary positions and the paged cache write against 64-bit references (tests/serving_ref.py:
the bounds are derived there)."""
import math

import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu


def _msa():
    import block_sparse_long_03_b200 as msa
    return msa


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _close(got, want, bound, where=""):
    d = (got.double().cpu() - want).abs()
    assert bool((d <= bound).all()), f"{where}: off by {float((d - bound).max())} over the bound"


SHAPES = [
    # n, Hq, Hkv, d, rot
    (1, 1, 1, 64, 64), (7, 32, 8, 128, 128), (65, 8, 2, 128, 64), (33, 6, 3, 64, 16),
    (5, 2, 2, 16, 16), (9, 3, 1, 256, 256), (130, 64, 4, 128, 32), (4, 5, 7, 48, 48),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,Hq,Hkv,d,rot", SHAPES)
def test_rope_matches_64_bits(n, Hq, Hkv, d, rot, layout, dtype):
    """Positions from negative ones to the far end of 31 bits; both directions."""
    msa, g = _msa(), _gen(n + d)
    Q, K = (torch.randn((n, H, d), generator=g).to(dtype) for H in (Hq, Hkv))
    pos = torch.randint(-5, 1 << 20, (n,), generator=g, dtype=torch.int32)
    pos[0] = (1 << 20) - 1
    f = msa.rope_frequencies(rot, scaling="parts", factor=4.0, device="cpu")
    for inverse, mscale in ((False, 1.0), (True, 1.25)):
        q, k = msa.rope(Q.cuda(), K.cuda(), pos.cuda(), f.cuda(), layout=layout, mscale=mscale,
                        inverse=inverse)
        for got, x in ((q, Q), (k, K)):
            want, bound = ref.rope(x, pos, f, layout, mscale, inverse)
            _close(got, want, bound, f"inverse={inverse}")
            assert torch.equal(got[..., rot:].cpu(), x[..., rot:])


def test_rope_in_place_and_strided():
    """Slices of one fused projection, turned in place: the same bits as dense copies, and the
    values between the slices untouched.  One tensor alone gives the same bits too."""
    msa, g = _msa(), _gen(3)
    n, Hq, Hkv, d = 37, 8, 2, 128
    fused = torch.randn((n, Hq + 2 * Hkv, d), generator=g).to(torch.bfloat16).cuda()
    before = fused.clone()
    Q, K = fused[:, :Hq], fused[:, Hq:Hq + Hkv]
    pos = torch.arange(n, dtype=torch.int32, device="cuda") * 1000
    f = msa.rope_frequencies(64)
    q, k = msa.rope(Q.contiguous(), K.contiguous(), pos, f, layout="interleaved")
    q1, none = msa.rope(Q, None, pos, f, layout="interleaved")
    assert none is None and torch.equal(q1, q)
    got = msa.rope(Q, K, pos, f, layout="interleaved", Q_out=Q, K_out=K)
    assert got[0].data_ptr() == Q.data_ptr()
    assert torch.equal(Q, q) and torch.equal(K, k)
    assert torch.equal(fused[:, Hq + Hkv:], before[:, Hq + Hkv:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient(layout):
    """inverse=True is the gradient: against the formula's (autograd in fp64) within the bound,
    and <R x, w> = <x, R^T w> against finite differences of the library's own forward (the map
    is linear: a difference is exact up to the outputs' rounding)."""
    msa, g = _msa(), _gen(5)
    n, H, d, rot, mscale = 6, 3, 64, 32, 1.5
    x = torch.randn((n, H, d), generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn((n, H, d), generator=g).float()
    pos = torch.randint(0, 5000, (n,), generator=g, dtype=torch.int32)
    f = msa.rope_frequencies(rot, device="cpu")
    ang = pos.double()[:, None, None] * f
    c, s = ang.cos() * mscale, ang.sin() * mscale
    ia = torch.arange(rot // 2) if layout == "half" else torch.arange(0, rot, 2)
    ib = ia + (rot // 2 if layout == "half" else 1)
    y = x.clone()
    y = y.index_copy(2, ia, x[..., ia] * c - x[..., ib] * s)
    y = y.index_copy(2, ib, x[..., ib] * c + x[..., ia] * s)
    (y * w.double()).sum().backward()
    grad, _ = msa.rope(w.cuda(), None, pos.cuda(), f.cuda(), layout=layout, mscale=mscale,
                       inverse=True)
    _, bound = ref.rope(w, pos, f, layout, mscale, True)
    _close(grad, x.grad, bound)
    # differences: 16 random directions; each y is good to its bound, so the sum over entries is
    x32 = x.detach().float()
    for k in range(16):
        v = torch.randn((n, H, d), generator=g).float()
        up, _ = msa.rope((x32 + v).cuda(), None, pos.cuda(), f.cuda(), layout=layout, mscale=mscale)
        dn, _ = msa.rope((x32 - v).cuda(), None, pos.cuda(), f.cuda(), layout=layout, mscale=mscale)
        diff = ((up.double() - dn.double()).cpu() / 2 * w.double()).sum()
        step = ((x32 + v).double() - (x32 - v).double()) / 2
        want = (grad.double().cpu() * step).sum()
        e = sum((ref.rope(z, pos, f, layout, mscale)[1] * w.double().abs()).sum()
                for z in (x32 + v, x32 - v)) / 2 + (bound * step.abs()).sum()
        assert abs(float(diff - want)) <= float(e)


def test_rope_far_positions_keep_their_angles():
    """Turning by p and by p + 1 differ by one more turn of theta, at 2^31 - 2 too, where an
    fp32 angle would be off by hundreds of radians."""
    msa = _msa()
    f = msa.rope_frequencies(64)
    x = torch.ones((2, 1, 64), device="cuda")
    pos = torch.tensor([2 ** 31 - 2, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    y, _ = msa.rope(x, None, pos, f)
    z = torch.complex(y[..., :32].double(), y[..., 32:].double())
    turned = torch.angle(z[1, 0] / z[0, 0])
    d = torch.remainder(turned - f + math.pi, 2 * math.pi) - math.pi
    # each angle: 2^31 theta in fp64 is good to 2^31 2^-52 rad (twice: theta / 2 pi and the
    # product), 1e-6, and 7e-7 from fp32; two of them
    assert float(d.abs().max()) <= 2 * (1e-6 + 7e-7 * math.sqrt(2))


APPEND = [
    # T, L, page, heads, d, rot, d_idx, dtype, layout
    ([1, 1, 1], [1, 64, 1000], 64, (8, 2), 128, 128, 64, torch.bfloat16, "half"),
    ([5, 0, 130, 1], [5, 0, 300, 17], 16, (6, 3), 64, 32, 0, torch.bfloat16, "interleaved"),
    ([33, 1], [40, 4096], 48, (4, 4), 64, 64, 128, torch.float32, "half"),
    ([3], [7], 1, (2, 1), 128, 64, 16, torch.float32, "interleaved"),
]


@pytest.mark.parametrize("T,L,page,heads,d,rot,d_idx,dtype,layout", APPEND)
def test_append_matches_64_bits(T, L, page, heads, d, rot, d_idx, dtype, layout):
    """Every new token's turned K, V and index key in its row; every other row of the caches,
    and the rows of Q_out outside the sequences, bit for bit as before."""
    msa, g = _msa(), _gen(len(T) + page)
    Hq, Hkv = heads
    lead, tail = 2, 3
    cu = ref.offsets(T, lead)
    n = int(cu[-1]) + tail
    _, _, Kc, Vc, table = ref.paginate(L, page, 3, Hkv, d, dtype, g)
    Ic = torch.randn((*Kc.shape[:2], max(d_idx, 16)), generator=g).to(dtype) if d_idx else None
    Q, K, V = (torch.randn((n, H, d), generator=g).to(dtype) for H in (Hq, Hkv, Hkv))
    x = torch.randn((n, d_idx), generator=g).to(dtype) if d_idx else None
    f = msa.rope_frequencies(rot, device="cpu")
    pos, row = [], []
    for b, (t, l) in enumerate(zip(T, L)):
        for p in range(l - t, l):
            pos.append(p)
            row.append(int(table[b, p // page]) * page + p % page)
    mine = slice(lead, n - tail)
    dev = dict(Kc=Kc.cuda(), Vc=Vc.cuda(), Ic=Ic.cuda() if d_idx else None)
    q_out = torch.full((n, Hq, d), 7.0, dtype=dtype, device="cuda")
    fused = torch.cat([K, V], 1).cuda()                      # K and V as slices
    q, ws = msa.rope_append_paged(Q.cuda(), fused[:, :Hkv], fused[:, Hkv:],
                                  x.cuda() if d_idx else None, cu.cuda(),
                                  torch.tensor(L, dtype=torch.int32).cuda(), table.cuda(),
                                  f.cuda(), dev["Kc"], dev["Vc"], dev["Ic"], layout=layout,
                                  mscale=1.1, Q_out=q_out)
    assert msa.msa_get_device_error(ws) == 0
    p = torch.tensor(pos)
    _close(q[mine], *ref.rope(Q[mine], p, f, layout, 1.1), "Q")
    assert bool((q[:lead] == 7).all()) and bool((q[n - tail:] == 7).all())
    flat = dev["Kc"].flatten(0, 1).cpu()
    _close(flat[row], *ref.rope(K[mine], p, f, layout, 1.1), "K")
    rest = torch.ones(flat.shape[0], dtype=torch.bool)
    rest[row] = False
    assert torch.equal(flat[rest], Kc.flatten(0, 1)[rest])
    for got, old, new in ((dev["Vc"], Vc, V), (dev["Ic"], Ic, x)):
        if got is None:
            continue
        want = old.flatten(0, 1).clone()
        want[row] = new[mine]
        assert torch.equal(got.flatten(0, 1).cpu(), want)


def test_append_without_queries_and_bad_sequences():
    """Keys only; a page id past the pool, a length above the table's capacity and a length
    under the new tokens: those tokens are skipped and reported, the others written."""
    msa, g = _msa(), _gen(11)
    T, L, page, Hkv, d = [2, 3, 1, 4], [40, 33, 20, 9], 16, 2, 64
    _, _, Kc, Vc, table = ref.paginate(L, page, 2, Hkv, d, torch.bfloat16, g)
    cu = ref.offsets(T)
    K, V = (torch.randn((sum(T), Hkv, d), generator=g).to(torch.bfloat16) for _ in range(2))
    f = msa.rope_frequencies(64)
    good, _ = table.clone(), None
    table[1, 1:] = Kc.shape[0]                      # tokens 30, 31 on page 1, token 32 on page 2
    lens = torch.tensor([40, 33, page * table.shape[1] + 1, 3], dtype=torch.int32)
    kc, vc = Kc.cuda(), Vc.cuda()
    q, ws = msa.rope_append_paged(None, K.cuda(), V.cuda(), None, cu.cuda(), lens.cuda(),
                                  table.cuda(), f, kc, vc)
    assert q is None and msa.msa_get_device_error(ws) == 7
    row = [int(good[0, p // page]) * page + p % page for p in (38, 39)]
    want = Vc.flatten(0, 1).clone()
    want[row] = V[:2]
    assert torch.equal(vc.flatten(0, 1).cpu(), want)
    _, ws = msa.rope_append_paged(None, K.cuda(), V.cuda(), None, cu.cuda(),
                                  torch.tensor(L, dtype=torch.int32).cuda(), good.cuda(), f, kc, vc,
                                  workspace=ws)
    assert msa.msa_get_device_error(ws) == 0        # the next call starts clean


@pytest.mark.parametrize("B", [33, 257, 1100])
def test_append_of_many_sequences(B):
    """Single tokens, none, and runs over one to ten pages of many sequences; some have a bad page
    among those of their new tokens (its tokens are skipped), some behind or before them."""
    msa, g = _msa(), _gen(B)
    page, Hkv, d = 16, 1, 16
    T = torch.randint(0, 3, (B,), generator=g)
    T[::5] = torch.randint(1, 150, (len(T[::5]),), generator=g)
    L = T + torch.randint(0, 40, (B,), generator=g)
    n_pages = -(-L // page)
    max_pages, total = int(n_pages.max()) + 1, int(n_pages.sum())
    order = torch.randperm(total, generator=g, dtype=torch.int32)
    table = torch.full((B, max_pages), -5, dtype=torch.int32)
    at = 0
    for b in range(B):
        k = int(n_pages[b])
        table[b, :k] = order[at:at + k]
        at += k
        if b % 7 == 3 and k:
            table[b, b % k] = total + B if b % 2 else -1
    cu = ref.offsets(T.tolist())
    K, V = (torch.randn((int(cu[-1]), Hkv, d), generator=g).to(torch.bfloat16) for _ in range(2))
    cache = torch.zeros((total + B, page, Hkv, d), dtype=torch.bfloat16)
    want, skipped = cache.flatten(0, 1).clone(), 0
    for b in range(B):
        for t in range(int(T[b])):
            p = int(L[b] - T[b]) + t
            pg = int(table[b, p // page])
            if 0 <= pg < total + B:
                want[pg * page + p % page] = V[int(cu[b]) + t]
            else:
                skipped += 1
    assert skipped
    kc, vc = cache.cuda(), cache.cuda()
    args = (None, K.cuda(), V.cuda(), None, cu.cuda(), L.int().cuda())
    f = msa.rope_frequencies(16)
    _, ws = msa.rope_append_paged(*args, table.cuda(), f, kc, vc)
    assert msa.msa_get_device_error(ws) == 7
    assert torch.equal(vc.flatten(0, 1).cpu(), want)
    for b in range(B):                                # without new tokens behind them: no error
        if b % 7 == 3:
            lo, hi = int(L[b] - T[b]) // page, int(n_pages[b])
            row = table[b, lo:hi]
            row[(row < 0) | (row >= total)] = total + b
    kc.zero_(), vc.zero_()
    _, ws = msa.rope_append_paged(*args, table.cuda(), f, kc, vc)
    assert msa.msa_get_device_error(ws) == 0


@pytest.mark.parametrize("with_idx", [False, True])
def test_append_of_no_tokens(with_idx):
    """A step in which no sequence has a new token: nothing is written, the error word is
    cleared, and offsets past the (empty) tokens are still found."""
    msa, g = _msa(), _gen(17)
    Kc, Vc = (torch.randn((3, 16, 2, 64), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    Ic = torch.randn((3, 16, 32), generator=g).to(torch.bfloat16).cuda() if with_idx else None
    caches = [x.clone() for x in (Kc, Vc, Ic) if x is not None]
    Q, K, V = (torch.empty((0, h, 64), dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2))
    x = torch.empty((0, 32), dtype=torch.bfloat16, device="cuda") if with_idx else None
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    lens = torch.tensor([5, 0], dtype=torch.int32, device="cuda")
    table = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    ws = torch.full((256,), 9, dtype=torch.uint8, device="cuda")
    f = msa.rope_frequencies(64)
    for q in (Q, None):
        out, _ = msa.rope_append_paged(q, K, V, x, cu, lens, table, f, Kc, Vc, Ic, workspace=ws)
        assert (out is None) == (q is None) and msa.msa_get_device_error(ws) == 0
    cu[2] = 1
    msa.rope_append_paged(Q, K, V, x, cu, lens, table, f, Kc, Vc, Ic, workspace=ws)
    assert msa.msa_get_device_error(ws) == 7
    for got, old in zip((x for x in (Kc, Vc, Ic) if x is not None), caches):
        assert torch.equal(got, old)


def test_rope_on_another_stream_and_in_a_graph():
    msa, g = _msa(), _gen(13)
    Q = torch.randn((50, 4, 128), generator=g).to(torch.bfloat16).cuda()
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    f = msa.rope_frequencies(128)
    want, _ = msa.rope(Q, None, pos, f)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got, _ = msa.rope(Q, None, pos, f)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(Q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.rope(Q, None, pos, f, Q_out=out)
    for k in range(2):
        Q.mul_(2)
        graph.replay()
        assert torch.equal(out, msa.rope(Q, None, pos, f)[0])
