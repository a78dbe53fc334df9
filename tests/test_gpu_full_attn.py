"""Full causal attention over packed and paged keys against the 64-bit reference
(tests/serving_ref.py: the bounds are derived there), and a run of the serving operators
together."""
import math

import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _msa():
    import block_sparse_long_03_b200 as msa
    return msa


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g).to(dtype)


def _check(O, lse, Q, Ks, Vs, cu, where="", scale=0.0):
    for b, (K, V) in enumerate(zip(Ks, Vs)):
        lo, hi = int(cu[b]), int(cu[b + 1])
        ref.assert_attention(O[lo:hi], lse[lo:hi],
                             ref.attention(Q[lo:hi].cuda(), K.cuda(), V.cuda(), scale),
                             f"{where} sequence {b}")


# ---------------------------------------------------------------- packed prompts

PACKED = [
    # heads (Hq, Hkv), d, dtype, lengths
    ((4, 4), 64, BF16, [1]),
    ((8, 2), 128, BF16, [1, 2, 0, 127, 128, 129, 255, 257]),
    ((8, 1), 128, BF16, [16, 17, 32, 33, 300, 1]),
    ((7, 1), 64, BF16, [5, 36, 37, 200]),
    ((14, 2), 128, BF16, [19, 130]),
    ((32, 2), 64, BF16, [8, 9, 16, 17, 131]),
    ((64, 1), 128, BF16, [1, 2, 3, 140]),
    ((3, 1), 128, BF16, [43, 85, 86, 260]),
    ((2, 2), 128, BF16, [700, 513]),
    ((4, 1), 64, F32, [1, 33, 0, 130]),
    ((6, 2), 128, F32, [64, 5, 97]),
]


@pytest.mark.parametrize("heads,d,dtype,lens", PACKED)
def test_packed_matches_64_bits(heads, d, dtype, lens):
    msa, g = _msa(), torch.Generator().manual_seed(len(lens) + d)
    n = sum(lens)
    Q, K, V = (_randn(g, (n, H, d), dtype) for H in (heads[0], heads[1], heads[1]))
    cu = ref.offsets(lens)
    O, lse, ws = msa.attn_packed(Q.cuda(), K.cuda(), V.cuda(), cu.cuda())
    assert msa.msa_get_device_error(ws) == 0
    _check(O, lse, Q, K.split(lens), V.split(lens), cu)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_packed_slices_with_rows_outside(dtype):
    """Q, K, V as slices of one fused projection; rows before the first and behind the last
    sequence are NaN, and their outputs stay as they were."""
    msa, g = _msa(), torch.Generator().manual_seed(2)
    lens, Hq, Hkv, d, lead, tail = [70, 0, 190], 8, 2, 64, 3, 5
    n = lead + sum(lens) + tail
    fused = _randn(g, (n, Hq + 2 * Hkv, d), dtype)
    fused[:lead] = math.nan
    fused[n - tail:] = math.nan
    dev = fused.cuda()
    cu = ref.offsets(lens, lead)
    out = torch.full((n, Hq, d), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((n, Hq), 7.0, device="cuda")
    msa.attn_packed(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], cu.cuda(), out=out,
                    lse=lse)
    mine = fused[lead:n - tail]
    _check(out, lse, fused[:, :Hq], mine[:, Hq:Hq + Hkv].split(lens),
           mine[:, Hq + Hkv:].split(lens), cu)
    for x in (out, lse):
        assert bool((x[:lead] == 7).all()) and bool((x[n - tail:] == 7).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_packed_keys_of_other_lengths(dtype):
    """More keys than queries (a cached prefix), fewer (queries before the first key attend
    nothing), none at all; a caller's scale."""
    msa, g = _msa(), torch.Generator().manual_seed(4)
    T, L, Hq, Hkv, d, scale = [40, 30, 9, 1, 200], [300, 12, 0, 700, 200], 4, 2, 128, 0.03
    Q = _randn(g, (sum(T), Hq, d), dtype)
    K, V = (_randn(g, (sum(L), Hkv, d), dtype) for _ in range(2))
    cu = ref.offsets(T)
    O, lse, _ = msa.attn_packed(Q.cuda(), K.cuda(), V.cuda(), cu.cuda(), ref.offsets(L).cuda(),
                                scale=scale)
    _check(O, lse, Q, K.split(L), V.split(L), cu, scale=scale)
    assert bool((O[40:58] == 0).all()) and bool(torch.isinf(lse[40:58]).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_packed_masked_values_have_no_influence(dtype, bad):
    """NaN or infinity in the keys and values of later tokens: every earlier row has the bits it
    has without them."""
    msa, g = _msa(), torch.Generator().manual_seed(6)
    lens, Hq, Hkv, d = [200, 90], 8, 2, 128
    Q, K, V = (_randn(g, (sum(lens), H, d), dtype).cuda() for H in (Hq, Hkv, Hkv))
    cu = ref.offsets(lens).cuda()
    O, lse, _ = msa.attn_packed(Q, K, V, cu)
    for first in (150, 131, 5):
        K2, V2 = K.clone(), V.clone()
        K2[first], V2[first] = bad, bad
        V2[first + 3, :, 5] = -bad
        O2, lse2, _ = msa.attn_packed(Q, K2, V2, cu)
        same = torch.ones(sum(lens), dtype=torch.bool)
        same[first:200] = False
        assert torch.equal(O2[same], O[same]) and torch.equal(lse2[same], lse[same])
        assert not bool(torch.isfinite(O2[first]).any())


def test_packed_infinite_values_reach_the_rows_that_attend_them():
    """+inf in one channel of a value: later rows have +inf there and their other channels
    unchanged; the rows before keep their bits."""
    msa, g = _msa(), torch.Generator().manual_seed(8)
    n, Hq, Hkv, d = 300, 4, 1, 64
    Q, K, V = (_randn(g, (n, H, d), BF16).cuda() for H in (Hq, Hkv, Hkv))
    cu = ref.offsets([n]).cuda()
    O, _, _ = msa.attn_packed(Q, K, V, cu)
    V[140, 0, 9] = math.inf
    O2, _, _ = msa.attn_packed(Q, K, V, cu)
    assert bool((O2[140:, :, 9] == math.inf).all()) and torch.equal(O2[:140], O[:140])
    keep = torch.arange(d) != 9
    assert torch.equal(O2[..., keep], O[..., keep])


def test_scores_of_minus_infinity_and_huge_scores():
    """A key of -inf scores (weight 0), a row whose every score is -inf (O = 0, lse = -inf), and
    scores that grow by hundreds along the keys (the running maximum moves every tile)."""
    msa = _msa()
    n, d = 700, 64
    Q = torch.zeros((n, 1, d))
    K = torch.zeros((n, 1, d))
    Q[..., 0] = 1.0
    K[:, 0, 0] = torch.arange(n) * 8.0                 # scores j * 8 / 8 = j
    V = torch.randn((n, 1, d), generator=torch.Generator().manual_seed(1))
    Q, K, V = (x.to(BF16) for x in (Q, K, V))
    cu = ref.offsets([n]).cuda()
    O, lse, _ = msa.attn_packed(Q.cuda(), K.cuda(), V.cuda(), cu)
    _check(O, lse, Q, [K], [V], ref.offsets([n]))
    K2 = K.clone()
    K2[:5, 0, 0] = -math.inf
    O2, lse2, _ = msa.attn_packed(Q.cuda(), K2.cuda(), V.cuda(), cu)
    assert bool((O2[:5] == 0).all()) and bool((lse2[:5] == -math.inf).all())
    want = (K[5:300, 0, 0].double() / 8).logsumexp(0)             # row 299: keys 5 .. 299
    assert abs(float(lse2[299, 0]) - float(want)) <= 300 * 2.0 ** -20
    assert bool(torch.isfinite(O2[5:]).all())


# ---------------------------------------------------------------- paged

PAGED = [
    # heads, d, dtype, page, new tokens, keys
    ((32, 8), 128, BF16, 64, [1], [1]),
    ((32, 8), 128, BF16, 64, [1, 1, 1, 1], [1000, 64, 65, 4097]),
    ((64, 4), 128, BF16, 16, [1, 0, 1, 7], [129, 50, 5000, 2000]),
    ((8, 8), 64, BF16, 8, [3, 1], [700, 9]),
    ((14, 2), 64, BF16, 24, [1, 100], [333, 100]),
    ((16, 1), 128, BF16, 48, [1, 9, 17, 40], [600, 600, 17, 777]),
    ((8, 1), 128, BF16, 256, [300, 1], [300, 3000]),
    ((4, 2), 128, BF16, 128, [129, 64, 65], [900, 64, 1025]),
    ((64, 1), 64, BF16, 32, [1, 2, 5], [400, 100, 5]),
    ((4, 2), 64, F32, 5, [1, 3, 70], [33, 3, 100]),
    ((2, 1), 128, F32, 64, [1, 40], [500, 40]),
]


@pytest.mark.parametrize("heads,d,dtype,page,T,L", PAGED)
def test_paged_matches_64_bits(heads, d, dtype, page, T, L):
    """Every row of a page that holds no key is NaN."""
    msa, g = _msa(), torch.Generator().manual_seed(page + len(T))
    Ks, Vs, Kc, Vc, table = ref.paginate(L, page, 2, heads[1], d, dtype, g, "cuda", math.nan)
    Q = _randn(g, (sum(T), heads[0], d), dtype)
    cu = ref.offsets(T)
    O, lse, ws = msa.attn_paged(Q.cuda(), Kc, Vc, cu.cuda(),
                                torch.tensor(L, dtype=torch.int32).cuda(), table)
    assert msa.msa_get_device_error(ws) == 0
    _check(O, lse, Q, Ks, Vs, cu)


def test_paged_long_context():
    """Single tokens and a short chunk over 70,001 keys (split over many key runs), with 64-bit
    sums on the GPU as the reference."""
    msa, g = _msa(), torch.Generator().manual_seed(21)
    L, page, Hq, Hkv, d = [70001, 300, 20000], 64, 8, 2, 128
    T = [1, 1, 20]
    Ks, Vs, Kc, Vc, table = ref.paginate(L, page, 1, Hkv, d, BF16, g, "cuda", math.nan)
    Q = _randn(g, (sum(T), Hq, d), BF16)
    cu = ref.offsets(T)
    args = (Q.cuda(), Kc, Vc, cu.cuda(), torch.tensor(L, dtype=torch.int32).cuda(), table)
    O, lse, _ = msa.attn_paged(*args)
    _check(O, lse, Q, Ks, Vs, cu)
    again = msa.attn_paged(*args)                      # the same bits every time
    assert torch.equal(again[0], O) and torch.equal(again[1], lse)


def test_paged_cache_past_32_bit_offsets():
    """A cache of more than 2^31 values: pages at its far end."""
    msa, g = _msa(), torch.Generator().manual_seed(23)
    page, Hkv, d, Hq = 64, 8, 128, 8
    pages = (1 << 31) // (page * Hkv * d) + 8
    Kc, Vc = (torch.empty((pages, page, Hkv, d), dtype=BF16, device="cuda") for _ in range(2))
    L, ids = 150, [pages - 1, 3, pages - 4]
    K, V = (_randn(g, (L, Hkv, d), BF16) for _ in range(2))
    for i, pg in enumerate(ids):
        m = min(page, L - i * page)
        Kc[pg, :m], Vc[pg, :m] = K[i * page:i * page + m].cuda(), V[i * page:i * page + m].cuda()
        Kc[pg, m:], Vc[pg, m:] = math.nan, math.nan
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    Q = _randn(g, (2, Hq, d), BF16)
    cu = ref.offsets([2])
    O, lse, _ = msa.attn_paged(Q.cuda(), Kc, Vc, cu.cuda(), lens, table)
    _check(O, lse, Q, [K], [V], cu)
    # and a write there
    f = msa.rope_frequencies(128)
    new = _randn(g, (1, Hkv, d), BF16).cuda()
    msa.rope_append_paged(None, new, new, None, ref.offsets([1]).cuda(), lens, table, f, Kc, Vc)
    assert torch.equal(Vc[pages - 4, (L - 1) % page], new[0])
    assert torch.equal(Vc[pages - 4, (L - 2) % page], V[L - 2].cuda())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_paged_bad_sequences_are_skipped(dtype):
    """A page id past the pool, a negative one, a length above the capacity and one under the
    new tokens: O = 0, lse = -inf, MSA_ERR_BAD_PAGE_TABLE; the others as usual.  A bad id behind
    a sequence's length does not matter."""
    msa, g = _msa(), torch.Generator().manual_seed(31)
    T, L, page, Hq, Hkv, d = [1, 2, 3, 1, 20], [200, 150, 90, 70, 130], 16, 8, 2, 128
    Ks, Vs, Kc, Vc, table = ref.paginate(L, page, 2, Hkv, d, dtype, g, "cuda", math.nan)
    Q = _randn(g, (sum(T), Hq, d), dtype)
    cu = ref.offsets(T)
    bad = table.clone()
    bad[1, 3] = Kc.shape[0]
    bad[3, 0] = -1
    bad[4, -(-L[4] // page):] = 1 << 30
    lens = torch.tensor([200, 150, 2, 70, 130], dtype=torch.int32)
    O, lse, ws = msa.attn_paged(Q.cuda(), Kc, Vc, cu.cuda(), lens.cuda(), bad)
    assert msa.msa_get_device_error(ws) == 7
    for b in (1, 2, 3):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        assert bool((O[rows] == 0).all()) and bool((lse[rows] == -math.inf).all())
    for b in (0, 4):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        ref.assert_attention(O[rows], lse[rows],
                             ref.attention(Q[rows].cuda(), Ks[b].cuda(), Vs[b].cuda()), f"{b}")
    lens[:] = page * table.shape[1] + 1
    O, lse, ws = msa.attn_paged(Q.cuda(), Kc, Vc, cu.cuda(), lens.cuda(), table, workspace=ws)
    assert bool((O == 0).all()) and msa.msa_get_device_error(ws) == 7


@pytest.mark.parametrize("B,long_pages", [(31, 0), (100, 300), (300, 900), (1300, 0)])
def test_paged_bad_pages_among_many(B, long_pages):
    """Bad page ids at the first, a middle and the last page of short and long rows of batches
    of every size: those sequences give O = 0 and lse = -inf, the others as usual."""
    msa, g = _msa(), torch.Generator().manual_seed(B)
    page, Hkv, Hq, d = 8, 1, 2, 64
    max_pages = max(long_pages, 40)
    L = torch.randint(1, 40 * page + 1, (B,), generator=g)
    if long_pages:
        L[::7] = torch.randint(257 * page, long_pages * page + 1, (len(L[::7]),), generator=g)
    n_pages = -(-L // page)
    Kc, Vc = (_randn(g, (max_pages, page, Hkv, d), BF16).cuda() for _ in range(2))
    table = torch.randint(0, max_pages, (B, max_pages), generator=g, dtype=torch.int32)
    bad = torch.rand(B, generator=g) < 0.2
    for b in torch.nonzero(bad)[:, 0].tolist():
        at = (0, int(n_pages[b]) // 2, int(n_pages[b]) - 1)[b % 3]
        table[b, at] = -1 if b % 2 else max_pages
    for b in range(B):
        table[b, int(n_pages[b]):] = -(1 << 30)
    Q = _randn(g, (B, Hq, d), BF16)
    O, lse, ws = msa.attn_paged(Q.cuda(), Kc, Vc, ref.offsets([1] * B).cuda(), L.int().cuda(),
                                table.cuda())
    assert msa.msa_get_device_error(ws) == 7
    assert bool((O[bad.cuda()] == 0).all()) and bool((lse[bad.cuda()] == -math.inf).all())
    for b in torch.nonzero(~bad)[:, 0].tolist():
        rows = table[b, :int(n_pages[b])].long().cuda()
        K, V = (x[rows].reshape(-1, Hkv, d)[:int(L[b])] for x in (Kc, Vc))
        ref.assert_attention(O[b:b + 1], lse[b:b + 1],
                             ref.attention(Q[b:b + 1].cuda(), K, V), f"sequence {b}")


def test_paged_rows_outside_with_split_keys():
    """Rows before the first and behind the last sequence stay as they were where the results
    come in parts; queries as a slice of a fused projection."""
    msa, g = _msa(), torch.Generator().manual_seed(37)
    T, L, page, Hq, Hkv, d, lead, tail = [1, 0, 5], [3000, 70, 4500], 16, 8, 2, 128, 3, 4
    Ks, Vs, Kc, Vc, table = ref.paginate(L, page, 2, Hkv, d, BF16, g, "cuda", math.nan)
    n = lead + sum(T) + tail
    fused = _randn(g, (n, Hq + 4, d), BF16).cuda()
    cu = ref.offsets(T, lead)
    out = torch.full((n, Hq, d), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((n, Hq), 7.0, device="cuda")
    _, _, ws = msa.attn_paged(fused[:, :Hq], Kc, Vc, cu.cuda(),
                              torch.tensor(L, dtype=torch.int32).cuda(), table, out=out, lse=lse)
    assert msa.msa_get_device_error(ws) == 0
    _check(out, lse, fused[:, :Hq], Ks, Vs, cu)
    for x in (out, lse):
        assert bool((x[:lead] == 7).all()) and bool((x[n - tail:] == 7).all())


@pytest.mark.parametrize("cu", [[0, 5, 3, 9], [-1, 2, 3, 9], [0, 2, 3, 10]])
def test_bad_offsets_write_nothing(cu):
    msa = _msa()
    x = torch.randn((9, 2, 64), device="cuda").to(BF16)
    off = torch.tensor(cu, dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 2, 3, 9], dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(x, 7.0), torch.full((9, 2), 7.0, device="cuda")
    for cq, ck in ((off, good), (good, off)):
        ws = msa.attn_packed(x, x, x, cq, ck, out=out, lse=lse)[2]
        assert msa.msa_get_device_error(ws) == 8
        assert bool((out == 7).all()) and bool((lse == 7).all())
    msa.attn_packed(x, x, x, good, out=out, lse=lse, workspace=ws)
    assert msa.msa_get_device_error(ws) == 0 and not bool((out == 7).all())


def test_graphs_and_streams():
    """Two captured graphs with a workspace each, replayed in turn after their inputs changed,
    and a call on another stream, give the bits of plain calls."""
    msa, g = _msa(), torch.Generator().manual_seed(41)
    cases = []
    for T, L in (([1, 1, 30], [900, 2000, 500]), ([1] * 6, [3000, 5, 80, 64, 65, 1])):
        Ks, Vs, Kc, Vc, table = ref.paginate(L, 32, 1, 2, 128, BF16, g, "cuda", math.nan)
        Q = _randn(g, (sum(T), 8, 128), BF16).cuda()
        args = (Q, Kc, Vc, ref.offsets(T).cuda(), torch.tensor(L, dtype=torch.int32).cuda(), table)
        out, lse, ws = msa.attn_paged(*args)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            msa.attn_paged(*args, out=out, lse=lse, workspace=ws)
        cases.append((args, out, lse, graph, ws))      # a graph's workspace lives as long as it
    for k in range(3):
        for args, out, lse, graph, _ in cases:
            args[0].mul_(0.5)
            args[4].sub_(1).clamp_(min=31 if args[0].shape[0] == 32 else 1)
            graph.replay()
            want = msa.attn_paged(*args)
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = msa.attn_paged(*cases[0][0])
    side.synchronize()
    want = msa.attn_paged(*cases[0][0])
    assert torch.equal(got[0], want[0])


def test_paged_equals_packed():
    """The same sequences through both calls agree within twice the bound."""
    msa, g = _msa(), torch.Generator().manual_seed(51)
    T, L, Hq, Hkv, d = [60, 1, 200], [200, 333, 200], 8, 2, 128
    Ks, Vs, Kc, Vc, table = ref.paginate(L, 16, 1, Hkv, d, BF16, g, "cuda", math.nan)
    Q = _randn(g, (sum(T), Hq, d), BF16).cuda()
    cu = ref.offsets(T).cuda()
    a = msa.attn_paged(Q, Kc, Vc, cu, torch.tensor(L, dtype=torch.int32).cuda(), table)
    b = msa.attn_packed(Q, torch.cat(Ks).cuda(), torch.cat(Vs).cuda(), cu, ref.offsets(L).cuda())
    for i, (lo, hi) in enumerate(zip(cu[:-1].tolist(), cu[1:].tolist())):
        _, _, Ob, lb = ref.attention(Q[lo:hi], Ks[i].cuda(), Vs[i].cuda())
        assert bool(((a[0][lo:hi].double() - b[0][lo:hi].double()).abs() <= 2 * Ob).all())
        assert bool(((a[1][lo:hi].double() - b[1][lo:hi].double()).abs() <= 2 * lb).all())


def test_many_sequences():
    """1500 sequences of 0 to 4 tokens (more than the plan's threads), packed and paged."""
    msa, g = _msa(), torch.Generator().manual_seed(71)
    T = torch.randint(0, 5, (1500,), generator=g).tolist()
    L = [t + int(x) if t else 0 for t, x in zip(T, torch.randint(0, 40, (1500,), generator=g))]
    Hq, Hkv, d = 4, 1, 64
    Ks, Vs, Kc, Vc, table = ref.paginate(L, 8, 1, Hkv, d, BF16, g, "cuda", math.nan)
    Q = _randn(g, (sum(T), Hq, d), BF16)
    cu, ck = ref.offsets(T), ref.offsets(L)
    a = msa.attn_paged(Q.cuda(), Kc, Vc, cu.cuda(), ck.diff().to(torch.int32).cuda(), table)
    b = msa.attn_packed(Q.cuda(), torch.cat(Ks).cuda(), torch.cat(Vs).cuda(), cu.cuda(), ck.cuda())
    assert msa.msa_get_device_error(a[2]) == 0 and msa.msa_get_device_error(b[2]) == 0
    some = [i for i in range(1500) if T[i]][::37]
    for O, lse, _ in (a, b):
        for i in some:
            rows = slice(int(cu[i]), int(cu[i + 1]))
            ref.assert_attention(O[rows], lse[rows], ref.attention(Q[rows], Ks[i], Vs[i]), f"{i}")
    assert torch.equal(a[0], b[0])          # one key tile each: the same products in both


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nothing_to_do_and_no_keys(dtype):
    """No tokens: the error word is cleared.  Tokens without any key: O = 0, lse = -inf."""
    msa = _msa()
    Q = torch.randn((6, 4, 64), device="cuda").to(dtype)
    none = torch.zeros((0, 2, 64), dtype=dtype, device="cuda")
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    O, _, _ = msa.attn_packed(Q[:0], none, none, zero, workspace=ws)
    assert O.shape == (0, 4, 64) and msa.msa_get_device_error(ws) == 0
    cu = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    O, lse, ws = msa.attn_packed(Q, none, none, cu, zero)
    assert msa.msa_get_device_error(ws) == 0
    assert bool((O == 0).all()) and bool((lse == -math.inf).all())


def test_output_16_byte_aligned():
    """O 16 but not 32 bytes aligned: the same bits."""
    msa, g = _msa(), torch.Generator().manual_seed(81)
    n, H, d = 300, 2, 64
    Q, K, V = (_randn(g, (n, H, d), BF16).cuda() for _ in range(3))
    cu = ref.offsets([n]).cuda()
    want = msa.attn_packed(Q, K, V, cu)
    room = torch.zeros(n * H * d + 16, dtype=BF16, device="cuda")
    at = 8 if room.data_ptr() % 32 == 0 else 0
    out = room[at:at + n * H * d].view(n, H, d)
    assert out.data_ptr() % 32 == 16
    msa.attn_packed(Q, K, V, cu, out=out)
    assert torch.equal(out, want[0])


def test_two_calls_at_once():
    """Calls on two streams that may overlap, a workspace each, give the bits of calls alone."""
    msa, g = _msa(), torch.Generator().manual_seed(91)
    jobs = []
    for T, L in (([64] * 4, [3000, 2000, 900, 64]), ([1] * 40, [1500] * 40)):
        _, _, Kc, Vc, table = ref.paginate(L, 64, 1, 4, 128, BF16, g, "cuda", math.nan)
        Q = _randn(g, (sum(T), 16, 128), BF16).cuda()
        jobs.append((Q, Kc, Vc, ref.offsets(T).cuda(), torch.tensor(L, dtype=torch.int32).cuda(),
                     table))
    alone = [msa.attn_paged(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        got = []
        for j, st in zip(jobs, streams):
            with torch.cuda.stream(st):
                got.append(msa.attn_paged(*j))
        torch.cuda.synchronize()
        for x, y in zip(got, alone):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


# ---------------------------------------------------------------- together

def test_serving_run():
    """Two prompts prefilled in chunks and then decoded, every token's K and V entering the
    cache through rope_append_paged: each step's attn_paged against the whole sequence in 64
    bits (on the bf16 keys the cache holds, which are rope's), the whole prompts through rope
    and attn_packed give the same rows within the bounds, and msa_decode_paged reads the same
    caches (with every block kept it is full attention)."""
    msa, g = _msa(), torch.Generator().manual_seed(61)
    Hq, Hkv, d, d_idx, page, block = 8, 2, 128, 64, 32, 64
    steps = [[100, 40], [29, 0], [1, 90], [1, 1], [1, 1]]
    total = [sum(s[b] for s in steps) for b in range(2)]
    S = 192
    pages = -(-S // page)
    table = torch.randperm(2 * pages, generator=g).view(2, pages).to(torch.int32).cuda()
    Kc, Vc = (torch.full((2 * pages, page, Hkv, d), math.nan, dtype=BF16, device="cuda")
              for _ in range(2))
    Ic = torch.full((2 * pages, page, d_idx), math.nan, dtype=BF16, device="cuda")
    f = msa.rope_frequencies(d)
    raw = [[_randn(g, (n, H, d), BF16).cuda() for H in (Hq, Hkv, Hkv)] for n in total]
    idx = [_randn(g, (n, d_idx), BF16).cuda() for n in total]
    turned = []
    for b, (q, k, v) in enumerate(raw):
        pos = torch.arange(total[b], dtype=torch.int32, device="cuda")
        turned.append(msa.rope(q, k, pos, f) + (v,))
    refs = [ref.attention(*x) for x in turned]
    done = [0, 0]
    for new in steps:
        part = [slice(done[b], done[b] + new[b]) for b in range(2)]
        done = [done[b] + new[b] for b in range(2)]
        Q, K, V = (torch.cat([raw[b][i][part[b]] for b in range(2)]) for i in range(3))
        x = torch.cat([idx[b][part[b]] for b in range(2)])
        cu = ref.offsets(new).cuda()
        lens = torch.tensor(done, dtype=torch.int32, device="cuda")
        q, ws = msa.rope_append_paged(Q, K, V, x, cu, lens, table, f, Kc, Vc, Ic, Q_out=Q)
        assert msa.msa_get_device_error(ws) == 0
        O, lse, ws = msa.attn_paged(q, Kc, Vc, cu, lens, table)
        assert msa.msa_get_device_error(ws) == 0
        for b in range(2):
            rows = slice(int(cu[b]), int(cu[b + 1]))
            assert torch.equal(q[rows], turned[b][0][part[b]])
            ref.assert_attention(O[rows], lse[rows], [r[part[b]] for r in refs[b]], f"step {new}")
    # the last step again through the block-sparse call, every block kept
    Os, lses, _, ws = msa.decode_paged(_randn(g, (2, 1, Hkv, d_idx), BF16).cuda(), Ic,
                                       q.view(2, 1, Hq, d), Kc, Vc, lens, table, S=S, block=block,
                                       topk=3)
    assert msa.msa_get_device_error(ws) == 0
    for b in range(2):
        # its partial outputs are rounded to bf16 once more: one more weighted 2^-8
        r = [x[-1:] for x in refs[b]]
        ref.assert_attention(Os[b], lses[b], (r[0], r[1], 2 * r[2], r[3]), "block-sparse")
    O, lse, _ = msa.attn_packed(*(torch.cat([turned[b][i] for b in range(2)]) for i in range(3)),
                                ref.offsets(total).cuda())
    for b, O_b, l_b in zip(range(2), O.split(total), lse.split(total)):
        ref.assert_attention(O_b, l_b, refs[b], "prompts")
