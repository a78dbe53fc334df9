"""Full causal attention over key runs so long that the order and the rounding of the sums count.

A call of 2400 tokens of 64 heads over one KV head has more units than the GPU has room for, so
that no row's keys are cut into runs: every row's sums are one run (the workspace then has no
partial results).  Caches of a few pages, read again and again, stand for long contexts."""
import math

import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
T, PAGE, HEADS = 2400, 256, 64


def _msa():
    import block_sparse_long_03_b200 as msa
    return msa


def _expect(q, K, V, counts):
    """(O, lse, bound of O, of lse) in 64 bits of one token's heads q [Hq, d] over keys K, V [n, d]
    that occur counts [n] times each.

    Scores, weights and their rounding as in serving_ref.attention: A (2 e + 2^-18 + 2^-8) for the
    scores, exp and the weights' rounding to bf16 (none where all weights are powers of two), u |O|
    for O's.  Sums: at most 2^16 keys go through the tensor core's fp32 sums at once, four keys an
    addition, each cut off by less than 2^-23 of the sum: 2^14 2^-23 = 2^-9.  The row sum adds 64
    keys at a time, 2^10 of those and then runs of 2^16 keys, each rounded by 2^-24; 64 keys take
    32 + 1 additions: (2^10 + 2^6 + 33) 2^-24 < 2^-13, for the lse too."""
    d = q.shape[1]
    q, K, V, counts = q.double(), K.double(), V.double(), counts.double()
    s = q @ K.T / math.sqrt(d)
    e = float(((d + 8) * 2.0 ** -23 * (q.abs() @ K.abs().T) / math.sqrt(d)).max())
    lse = torch.logsumexp(s + counts.log(), 1)
    w = counts * torch.exp(s - lse[:, None])
    O, A = w @ V, w @ V.abs()
    r = 2.0 ** -8 if bool((s != 0).any()) else 0.0
    bound = A * (2 * e + 2.0 ** -18 + r + 2.0 ** -9 + 2.0 ** -13) + ref.U[BF16] * O.abs()
    return O, lse, bound, e + 2.0 ** -18 + 2.0 ** -13 + 2.0 ** -22 * lse.abs()


def _assert(O, lse, want, where):
    Or, lr, Ob, lb = want
    over = (O.double() - Or).abs() - Ob
    assert bool((over <= 0).all()), \
        f"{where}: O off by {float(over.max())} over the bound {float(Ob.flatten()[over.argmax()])}"
    assert bool(((lse.double() - lr).abs() <= lb).all()), where


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scores", [False, True])
def test_a_long_run_keeps_its_sum(d, scores):
    """A single token over 2^22 keys, values with a mean of 1."""
    msa, g = _msa(), torch.Generator().manual_seed(d)
    L = 1 << 22
    table = (torch.arange(L // PAGE, dtype=torch.int32) % 16).repeat(2, 1).cuda()
    K = (torch.randn((16, PAGE, 1, d), generator=g) * scores).to(BF16).cuda()
    V = (torch.rand((16, PAGE, 1, d), generator=g) + 0.5).to(BF16).cuda()
    Q = torch.randn((T + 1, HEADS, d), generator=g).to(BF16).cuda()
    lens = torch.tensor([T, L], dtype=torch.int32, device="cuda")
    O, lse, ws = msa.attn_paged(Q, K, V, ref.offsets([T, 1]).cuda(), lens, table)
    assert msa.msa_get_device_error(ws) == 0
    counts = torch.full((16 * PAGE,), L / (16 * PAGE), device="cuda")
    _assert(O[T], lse[T], _expect(Q[T], K.view(-1, d), V.view(-1, d), counts), "long run")
    counts = torch.ones(T, device="cuda")                 # the prompt's last token
    _assert(O[T - 1], lse[T - 1],
            _expect(Q[T - 1], K.view(-1, d)[:T], V.view(-1, d)[:T], counts), "prompt")


@pytest.mark.parametrize("d", [64, 128])
def test_a_chunk_whose_maximum_moves_late(d):
    """A chunk of 2400 tokens at the end of 200,001 keys whose scores rise at keys around 66,000,
    140,000 and 199,700: the running maximum moves in the first half behind a moved sum, between
    two and near the end, where only the last tokens see the keys."""
    msa, g = _msa(), torch.Generator().manual_seed(d + 1)
    L = 200001
    n = -(-L // PAGE)
    table = (torch.arange(n, dtype=torch.int32) % 16).view(1, n)
    K = torch.randn((19, PAGE, 1, d), generator=g).to(BF16)
    V = (torch.randn((19, PAGE, 1, d), generator=g) + 0.5).to(BF16)
    for i, key in enumerate((65536 + 10, 140000, 199700)):
        table[0, key // PAGE] = 16 + i
        K[16 + i] *= 4 + 4 * i
    K, V, table = K.cuda(), V.cuda(), table.cuda()
    Q = torch.randn((T, HEADS, d), generator=g).to(BF16).cuda()
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    O, lse, ws = msa.attn_paged(Q, K, V, ref.offsets([T]).cuda(), lens, table)
    assert msa.msa_get_device_error(ws) == 0
    rows = table[0].long()
    Kf, Vf = K[rows].view(-1, d)[:L], V[rows].view(-1, d)[:L]
    for t in (0, 1, 1999, 2090, 2098, 2099, 2100, 2101, 2300, T - 1):
        seen = L - T + t + 1
        _assert(O[t], lse[t], _expect(Q[t], Kf[:seen], Vf[:seen], torch.ones(seen, device="cuda")),
                f"token {t}")


def test_a_key_run_of_seconds():
    """A single token over 2^29 keys (on 16 pages, again and again) beside 2400 prompt tokens, which
    leave it one key run and one stream: 4 million tiles one after another, about 5 s, longer than the
    2 s that a wait on another role's next step may take.  The stream without keys and the check
    of the values wait for their turn meanwhile, and nothing may give up.  All scores are 0 and
    the values constant: the sums of weights are exact in fp32 (multiples of 64 up to 2^29), those of
    equal values too, so that O is the value."""
    msa, page, d, Hq = _msa(), 256, 64, 64
    L, T = 1 << 29, 2400
    table = (torch.arange(L // page, dtype=torch.int32, device="cuda") % 16).repeat(2, 1)
    value = (2.0 ** -(torch.arange(d) % 3)).to(BF16).cuda()
    Kc = torch.zeros((16, page, 1, d), dtype=BF16, device="cuda")
    Vc = value.expand(16, page, 1, d).contiguous()
    Q = torch.ones((T + 1, Hq, d), dtype=BF16, device="cuda")
    lens = torch.tensor([T, L], dtype=torch.int32, device="cuda")
    O, lse, ws = msa.attn_paged(Q, Kc, Vc, ref.offsets([T, 1]).cuda(), lens, table)
    assert ws.numel() < 11 << 20                       # no partial results (two a row: 157 MB)
    assert msa.msa_get_device_error(ws) == 0
    assert torch.equal(O, value.expand_as(O))
    want = torch.log(torch.cat([torch.arange(1, T + 1), torch.tensor([L])]).double())
    assert float((lse.cpu().double() - want[:, None]).abs().max()) <= 2.0 ** -22 * math.log(L)


@pytest.mark.parametrize("d", [64, 128])
def test_fp32_sums_of_equal_values(d):
    """fp32, one token over 2^18 keys of equal values and scores: weights of 1 and an exact row sum.
    The values of 32 keys are summed (31 roundings of at most 2^-24 of the sum), and 2^13 such sums
    are added (one each); the quotient rounds twice more."""
    msa, page, L = _msa(), 64, 1 << 18
    table = (torch.arange(L // page, dtype=torch.int32, device="cuda") % 4).view(1, -1)
    value = torch.linspace(0.55, 1.45, d, device="cuda")
    K = torch.zeros((4, page, 1, d), device="cuda")
    V = value.expand(4, page, 1, d).contiguous()
    O, lse, ws = msa.attn_paged(torch.ones((1, 2, d), device="cuda"), K, V,
                                ref.offsets([1]).cuda(), torch.tensor([L], dtype=torch.int32).cuda(),
                                table)
    assert msa.msa_get_device_error(ws) == 0
    off = (O.double() / value.double() - 1).abs()
    assert float(off.max()) <= (31 + 2 ** 13 + 2) * 2.0 ** -24, float(off.max())
    assert float((lse.double() - math.log(L)).abs().max()) <= 2.0 ** -22 * math.log(L)


@pytest.mark.parametrize("d", [64, 128])
def test_odd_values_along_a_long_run(d):
    """Infinite values and NaN, keys of -infinity and rows without weights, where a run of keys is
    taken in pieces of 65536: in the first piece, at the end of one and in the last, under tokens
    that attend them and tokens that do not."""
    msa, g = _msa(), torch.Generator().manual_seed(d + 5)
    n = 65536 + 65536 + 1000                           # keys; the last 2400 have queries
    Q = torch.randn((T, HEADS, d), generator=g).to(BF16).cuda()
    K, V = (torch.randn((n, 1, d), generator=g).to(BF16).cuda() for _ in range(2))
    Q[..., 0], K[..., 0] = 1.0, 0.0
    cq, ck = ref.offsets([T]).cuda(), ref.offsets([n]).cuda()
    first = n - T
    want, want_lse, ws = msa.attn_packed(Q, K, V, cq, ck)
    assert msa.msa_get_device_error(ws) == 0 and bool(torch.isfinite(want).all())
    at = [77, 65535, 65536, 131071, 131072, first + 1, first + 700, n - 1]
    for key in at:                                     # an infinite value, every weight positive
        V2 = V.clone()
        V2[key, 0, 3], V2[key, 0, 5] = math.inf, math.nan
        O, lse, _ = msa.attn_packed(Q, K, V2, cq, ck)
        sees = max(0, key - first)                     # the first token that attends the key
        assert torch.equal(O[:sees], want[:sees]) and torch.equal(lse, want_lse)
        assert bool((O[sees:, :, 3] == math.inf).all()) and bool(torch.isnan(O[sees:, :, 5]).all())
        keep = [c for c in range(d) if c not in (3, 5)]
        assert torch.equal(O[..., keep], want[..., keep])
    for lo, hi in ((0, 65536), (65536, 131072), (0, 131072)):   # pieces of zero weights
        K2, V2 = K.clone(), V.clone()
        K2[lo:hi, 0, 0] = -math.inf
        O1, lse1, _ = msa.attn_packed(Q, K2, V, cq, ck)
        dead = T - 1000 if hi == 131072 and lo == 0 else 0   # tokens that attend no other key
        assert bool((O1[:dead] == 0).all()) and bool((lse1[:dead] == -math.inf).all())
        assert bool(torch.isfinite(O1).all()) and bool(torch.isfinite(lse1[dead:]).all())
        V2[lo + 9, 0, 3] = math.inf
        O2, lse2, _ = msa.attn_packed(Q, K2, V2, cq, ck)
        assert torch.equal(lse2, lse1) and torch.equal(O2[:dead], O1[:dead])
        assert bool(torch.isnan(O2[dead:, :, 3]).all())
        keep = [c for c in range(d) if c != 3]
        assert torch.equal(O2[..., keep], O1[..., keep])
    K2 = K.clone()
    K2[1234] = math.nan                                # a NaN score in the first piece
    O, lse, _ = msa.attn_packed(Q, K2, V, cq, ck)
    assert bool(torch.isnan(O).all()) and bool(torch.isnan(lse).all())
