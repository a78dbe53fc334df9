"""The serving operators where large calls run: every number of warps a token takes in the rotary
step and the cache write, every number of key runs in the attention, against 64 bits (bounds as in
tests/serving_ref.py), and keys that cannot be lost or counted twice unseen."""
import math

import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _msa():
    import block_sparse_long_03_b200 as msa
    return msa


# ---------------------------------------------------------------- rotary positions

def _rope_close(got, x, pos, f, layout, mscale, inverse, where):
    """ref.rope's bound, and the angle's rounding at far positions: three fp64 roundings in the
    library (the part of a turn a token, the constant in it, the product) and one in the
    reference, each 2^-53 of the angle p theta."""
    want, bound = ref.rope(x, pos, f, layout, mscale, inverse)
    rot = 2 * f.numel()
    ia = torch.arange(rot // 2) if layout == "half" else torch.arange(0, rot, 2)
    ib = ia + (rot // 2 if layout == "half" else 1)
    far = (pos.double()[:, None, None] * f).abs() * 2.0 ** -51 * abs(mscale)
    far = far * (x.double()[..., ia].abs() + x.double()[..., ib].abs()) * (1 + ref.U[x.dtype])
    bound[..., ia] += far
    bound[..., ib] += far
    over = (got.double() - want).abs() - bound
    assert bool((over <= 0).all()), f"{where}: {float(over.max())} over the bound"
    assert torch.equal(got[..., rot:], x[..., rot:]), where


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("Hq,Hkv,d,rot", [(64, 8, 128, 128), (40, 4, 256, 128), (13, 20, 48, 32)])
@pytest.mark.parametrize("n", [290, 300, 1200, 2400])
def test_rope_of_many_tokens(n, Hq, Hkv, d, rot, layout, dtype):
    """Eight, four, two and one warp a token, several passes over its heads; positions over all 32
    bits; apart and in place in one fused tensor (the same bits)."""
    msa, g = _msa(), torch.Generator().manual_seed(n + d)
    fused = torch.randn((n, Hq + Hkv, d), generator=g).to(dtype).cuda()
    before = fused.clone()
    Q, K = fused[:, :Hq], fused[:, Hq:]
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (n,), generator=g).int()
    pos[:3] = torch.tensor([(1 << 31) - 1, -(1 << 31), 0])
    pos = pos.cuda()
    f = msa.rope_frequencies(rot, scaling="parts", factor=4.0)
    for inverse, mscale in ((False, 1.0), (True, 1.25)):
        q, k = msa.rope(Q, K, pos, f, layout=layout, mscale=mscale, inverse=inverse)
        _rope_close(q, Q, pos, f, layout, mscale, inverse, "Q")
        _rope_close(k, K, pos, f, layout, mscale, inverse, "K")
    assert torch.equal(fused, before)
    msa.rope(Q, K, pos, f, layout=layout, mscale=1.25, inverse=True, Q_out=Q, K_out=K)
    assert torch.equal(Q, q) and torch.equal(K, k)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [[150, 1, 0, 130, 19], [800, 1, 399], [1500, 1, 1, 898, 40]])
def test_append_of_many_tokens(T, dtype):
    """Prompt chunks and single tokens enter the caches, at four, two and one warp a token: Q and
    every row of the three caches."""
    msa, g = _msa(), torch.Generator().manual_seed(sum(T))
    Hq, Hkv, d, d_idx, page, lead, tail = 64, 4, 128, 64, 48, 2, 3
    L = [t + 31 * b + 5 for b, t in enumerate(T)]
    n = lead + sum(T) + tail
    _, _, Kc, Vc, table = ref.paginate(L, page, 3, Hkv, d, dtype, g, "cuda", 7.0)
    Ic = torch.full((*Kc.shape[:2], d_idx), 7.0, dtype=dtype, device="cuda")
    Q, K, V = (torch.randn((n, H, d), generator=g).to(dtype).cuda() for H in (Hq, Hkv, Hkv))
    x = torch.randn((n, d_idx), generator=g).to(dtype).cuda()
    pos = torch.cat([torch.arange(l - t, l) for t, l in zip(T, L)]).cuda()
    seq = torch.repeat_interleave(torch.arange(len(T)), torch.tensor(T)).cuda()
    row = table[seq, pos // page].long() * page + pos % page
    f = msa.rope_frequencies(64)
    out = torch.full_like(Q, 7.0)
    old = [c.flatten(0, 1).clone() for c in (Kc, Vc, Ic)]
    _, ws = msa.rope_append_paged(Q, K, V, x, ref.offsets(T, lead).cuda(),
                                  torch.tensor(L, dtype=torch.int32).cuda(), table, f, Kc, Vc, Ic,
                                  mscale=1.1, Q_out=out)
    assert msa.msa_get_device_error(ws) == 0
    mine = slice(lead, n - tail)
    _rope_close(out[mine], Q[mine], pos.int(), f, "half", 1.1, False, "Q")
    assert bool((out[:lead] == 7).all()) and bool((out[n - tail:] == 7).all())
    _rope_close(Kc.flatten(0, 1)[row], K[mine], pos.int(), f, "half", 1.1, False, "K")
    old[0][row] = Kc.flatten(0, 1)[row]
    old[1][row], old[2][row] = V[mine], x[mine]
    for c, want in zip((Kc, Vc, Ic), old):
        assert torch.equal(c.flatten(0, 1), want)


# ---------------------------------------------------------------- attention

def _attention(Q, K, V):
    """ref.attention for finite values, all rows at once: (O, lse, O bound, lse bound)."""
    (T, Hq, d), (L, Hkv) = Q.shape, K.shape[:2]
    late = torch.arange(L, device="cuda")[None] > torch.arange(L - T, L, device="cuda")[:, None]
    out = [[], [], [], []]
    for h in range(Hq):
        q, k, v = Q[:, h].double(), K[:, h // (Hq // Hkv)].double(), V[:, h // (Hq // Hkv)].double()
        s = (q @ k.T / math.sqrt(d)).masked_fill(late, -math.inf)
        e = ((d + 8) * 2.0 ** -23 / math.sqrt(d) * (q.abs() @ k.abs().T)).masked_fill(late, 0.0)
        em = e.amax(1)
        x = torch.logsumexp(s, 1)
        w = torch.exp(s - x[:, None])
        o, A = w @ v, w @ v.abs()
        tol = 2 * em + 2 * L * 2.0 ** -23 + 2.0 ** -18 + 2.0 ** -8
        for i, y in enumerate((o, x, A * tol[:, None] + ref.U[Q.dtype] * o.abs(),
                               em + L * 2.0 ** -23 + 2.0 ** -18 + 2.0 ** -22 * x.abs())):
            out[i].append(y)
    return [torch.stack(y, 1) for y in out]


def _runs(tokens, Hq, Hkv):
    """Key runs that rows of a bf16 call may have (the rule of the kernel's cut)."""
    unit = 2 * (128 // (Hq // Hkv))
    units = -(-tokens // unit) * Hkv
    return min(64, -(-592 // units))


def _has_runs(ws, runs, tokens, Hq, d):
    """The workspace says which path a call takes: two partial results a run, row and head."""
    part = 2 * runs * tokens * Hq * (d + 1) * 4 if runs > 1 else 0
    return part <= ws.numel() < part + (1 << 20)


SIZES = [
    # lengths, (Hq, Hkv), runs: one (direct output), two, three
    ([1, 15, 16, 17, 33, 0, 2430], (64, 8), 1), ([700, 31, 1, 650, 32, 64, 1], (64, 8), 2),
    ([900, 5], (64, 8), 3), ([2431, 1, 3], (8, 8), 8), ([1300, 1, 7, 130, 129, 128, 900], (64, 1), 1),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,heads,runs", SIZES)
def test_prompts_of_every_cut(T, heads, runs, d):
    msa, g = _msa(), torch.Generator().manual_seed(sum(T))
    (Hq, Hkv), n = heads, sum(T)
    assert _runs(n, Hq, Hkv) == runs
    Q, K, V = (torch.randn((n, H, d), generator=g).to(BF16).cuda() for H in (Hq, Hkv, Hkv))
    cu = ref.offsets(T)
    O, lse, ws = msa.attn_packed(Q, K, V, cu.cuda())
    assert msa.msa_get_device_error(ws) == 0 and _has_runs(ws, runs, n, Hq, d)
    for b, (q, k, v) in enumerate(zip(Q.split(T), K.split(T), V.split(T))):
        if T[b]:
            rows = slice(int(cu[b]), int(cu[b + 1]))
            ref.assert_attention(O[rows], lse[rows], _attention(q, k, v), f"sequence {b}")


@pytest.mark.parametrize("page", [8, 64, 128])
@pytest.mark.parametrize("T,heads,runs", SIZES)
def test_chunks_of_every_cut(T, heads, runs, page):
    """Over cached prefixes of 0 to 3000 keys, in pages whose other rows are NaN."""
    msa, g = _msa(), torch.Generator().manual_seed(sum(T) + page)
    (Hq, Hkv), n, d = heads, sum(T), 128
    L = [t + (0, 1, 127, 1000, 3000, 50, 129)[b] for b, t in enumerate(T)]
    Ks, Vs, Kc, Vc, table = ref.paginate(L, page, 2, Hkv, d, BF16, g, "cuda", math.nan)
    Q = torch.randn((n, Hq, d), generator=g).to(BF16).cuda()
    cu = ref.offsets(T)
    O, lse, ws = msa.attn_paged(Q, Kc, Vc, cu.cuda(), torch.tensor(L, dtype=torch.int32).cuda(),
                                table)
    assert msa.msa_get_device_error(ws) == 0 and _has_runs(ws, runs, n, Hq, d)
    for b, q in enumerate(Q.split(T)):
        if T[b]:
            rows = slice(int(cu[b]), int(cu[b + 1]))
            ref.assert_attention(O[rows], lse[rows], _attention(q, Ks[b].cuda(), Vs[b].cuda()),
                                 f"sequence {b}")


def _assert_counts(O, lse, first, L, d, where):
    """Scores of 0 and values that are 1 in channel (j // 64) % d of key j and 0 elsewhere: O is how
    many of the keys are of a channel, over their number.  Weights and sums are exact (whole
    numbers under 2^24), the quotient rounds twice (2^-23) and O to its type; log is good to 2^-22.
    Rows are the positions first, first + 1, ... of L keys."""
    seen = torch.arange(first, L, device="cuda")[:, None] + 1
    c = torch.arange(d, device="cuda")[None]
    lap = 64 * d
    count = seen // lap * 64 + (seen % lap - 64 * c).clamp(0, 64)
    want = (count / seen.double())[:, None]
    u = ref.U[O.dtype] if O.dtype != F32 else 0.0
    off = (O.double() - want).abs() - want * (u + 2.0 ** -22)
    assert bool((off <= 0).all()), f"{where}: row and channel {torch.nonzero(off > 0)[0].tolist()}"
    x = torch.log(seen.double())
    assert bool(((lse.double() - x).abs() <= 2.0 ** -22 * (1 + x)).all()), where


def _counting(n, Hkv, d, dtype):
    V = torch.zeros((n, Hkv, d), dtype=dtype, device="cuda")
    j = torch.arange(n, device="cuda")
    V[j, :, j // 64 % d] = 1.0
    return V


COUNTED = [
    # (Hq, Hkv), d, dtype, T, L
    ((8, 2), 128, BF16, [1, 1, 20], [70001, 300, 20000]),       # many key runs
    ((64, 8), 64, BF16, [1] * 20, [16000 + 7 * i for i in range(20)]),
    ((64, 8), 128, BF16, [2500, 1, 9], [6000, 30001, 25000]),   # one run a row
    ((64, 1), 128, BF16, [1300, 1], [1300, 70000]),             # two runs, and moved sums
    ((4, 1), 64, F32, [1, 70], [9001, 5000]),
]


@pytest.mark.parametrize("heads,d,dtype,T,L", COUNTED)
def test_every_key_counts_once(heads, d, dtype, T, L):
    """Paged (pages of 16 and 64, other rows NaN) and packed with a cached prefix.  A tile or a
    half that is lost or taken twice is at least a tenth of its channel."""
    msa, g = _msa(), torch.Generator().manual_seed(len(T))
    Hq, Hkv = heads
    Q = torch.randn((sum(T), Hq, d), generator=g).to(dtype).cuda()
    cu, ck = ref.offsets(T), ref.offsets(L)
    Vs = [_counting(l, Hkv, d, dtype) for l in L]
    lens = torch.tensor(L, dtype=torch.int32, device="cuda")
    calls = [("packed", msa.attn_packed(Q, torch.zeros_like(torch.cat(Vs)), torch.cat(Vs),
                                        cu.cuda(), ck.cuda()))]
    for page in (16, 64):
        per = [-(-l // page) for l in L]
        order = torch.randperm(sum(per) + 2, generator=g).int().cuda()
        table = torch.full((len(L), max(per)), -1, dtype=torch.int32, device="cuda")
        Kc, Vc = (torch.full((sum(per) + 2, page, Hkv, d), math.nan, dtype=dtype, device="cuda")
                  for _ in range(2))
        at = 0
        for b, m in enumerate(per):
            table[b, :m] = order[at:at + m]
            rows = (order[at:at + m].long()[:, None] * page +
                    torch.arange(page, device="cuda")).flatten()[:L[b]]
            Kc.view(-1, Hkv, d)[rows], Vc.view(-1, Hkv, d)[rows] = 0.0, Vs[b]
            at += m
        calls.append((f"pages of {page}", msa.attn_paged(Q, Kc, Vc, cu.cuda(), lens, table)))
    for where, (O, lse, ws) in calls:
        assert msa.msa_get_device_error(ws) == 0
        for b in range(len(T)):
            rows = slice(int(cu[b]), int(cu[b + 1]))
            _assert_counts(O[rows], lse[rows], L[b] - T[b], L[b], d, f"{where}, sequence {b}")
