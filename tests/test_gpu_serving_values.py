"""Values and slots that must not count in the full causal attention, and infinite values that do.

The softmax is 32-bit: a key whose score is -infinity, or more than about 90 under the row's
largest, has a weight of exactly 0, and 0 times infinity is NaN, wherever the key lies.  A row
whose every score is -infinity has no weights at all: O = 0 and lse = -infinity."""
import math

import pytest
import torch

from tests import serving_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _msa():
    import block_sparse_long_03_b200 as msa
    return msa


def _prompt(dtype, n=300, Hq=4, d=64):
    """Q, K, V with Q's channel 0 at 1 and K's at 0: it sets a key's score alone."""
    g = torch.Generator().manual_seed(n)
    Q, K, V = (torch.randn((n, H, d), generator=g).to(dtype).cuda() for H in (Hq, 1, 1))
    Q[..., 0], K[..., 0] = 1.0, 0.0
    return Q, K, V, ref.offsets([n]).cuda()


@pytest.mark.parametrize("low", [-math.inf, -8.0 * 300])
def test_infinite_value_under_a_zero_weight(low):
    """Keys 5 and 140 have a weight of 0 in every row and an infinite value in one channel: NaN
    there in every row that attends them (they are in tiles that some rows attend whole and others
    in part), everything else bit for bit as with finite values."""
    msa = _msa()
    Q, K, V, cu = _prompt(BF16)
    K[5, 0, 0] = K[140, 0, 0] = low
    want, want_lse, _ = msa.attn_packed(Q, K, V, cu)
    V[5, 0, 9], V[140, 0, 33] = math.inf, -math.inf
    O, lse, _ = msa.attn_packed(Q, K, V, cu)
    assert torch.equal(lse, want_lse)
    odd = torch.zeros(O.shape, dtype=torch.bool, device="cuda")
    odd[5:, :, 9] = True
    odd[140:, :, 33] = True
    assert bool(torch.isnan(O[odd]).all()), f"{O[odd][~torch.isnan(O[odd])][:4]}"
    assert torch.equal(O[~odd], want[~odd])


def test_rows_without_weights_ignore_infinite_values():
    """The first rows' scores are all -infinity and their keys' values infinite: O = 0."""
    msa = _msa()
    Q, K, V, cu = _prompt(BF16)
    K[:5, 0, 0] = -math.inf
    V[:5, 0, 9], V[2, 0, 40] = math.inf, math.nan
    O, lse, _ = msa.attn_packed(Q, K, V, cu)
    assert bool((lse[:5] == -math.inf).all()) and bool((O[:5] == 0).all())
    assert bool(torch.isnan(O[5:, :, 9]).all()) and bool(torch.isnan(O[5:, :, 40]).all())
    keep = [c for c in range(64) if c not in (9, 40)]
    assert bool(torch.isfinite(O[..., keep]).all()) and bool(torch.isfinite(lse[5:]).all())


@pytest.mark.parametrize("d", [64, 128])
def test_fp32_rows_without_weights_ignore_infinite_values(d):
    """The same in fp32, and zero weights there."""
    msa = _msa()
    Q, K, V, cu = _prompt(F32, d=d)
    K[:5, 0, 0] = K[140, 0, 0] = -math.inf
    want, _, _ = msa.attn_packed(Q, K, V, cu)
    V[:5, 0, 9], V[140, 0, 33] = math.inf, -math.inf
    O, lse, _ = msa.attn_packed(Q, K, V, cu)
    assert bool((lse[:5] == -math.inf).all()) and bool((O[:5] == 0).all())
    odd = torch.zeros(O.shape, dtype=torch.bool, device="cuda")
    odd[5:, :, 9] = True
    odd[140:, :, 33] = True
    assert bool(torch.isnan(O[odd]).all()) and torch.equal(O[~odd], want[~odd])


def test_zero_weights_of_a_whole_key_run():
    """Single tokens over keys that are cut into runs.  A whole run (1024 keys) of scores of
    -infinity with an infinite value in it: NaN in that channel, the other channels as with finite
    values; without an infinite value nothing changes.  Every key so: O = 0."""
    msa, g = _msa(), torch.Generator().manual_seed(7)
    Hq, d, page, L = 2, 64, 64, [4096, 4096, 3000]
    _, _, Kc, Vc, table = ref.paginate(L, page, 1, 1, d, BF16, g, "cuda", math.nan)
    Q = torch.randn((3, Hq, d), generator=g).to(BF16).cuda()
    Q[..., 0] = 1.0
    run = table[0, 16:32].long()                       # keys 1024 .. 2047 of the first
    Kc[run, :, :, 0] = -math.inf
    Kc[table[2, :47].long(), :, :, 0] = -math.inf      # every key of the third
    args = (Q, Kc, Vc, ref.offsets([1, 1, 1]).cuda(), torch.tensor(L, dtype=torch.int32).cuda(),
            table)
    want, want_lse, ws = msa.attn_paged(*args)
    assert msa.msa_get_device_error(ws) == 0 and bool(torch.isfinite(want).all())
    for at in (16, 24, 31):
        Vc2 = Vc.clone()
        Vc2[table[0, at].long(), 5, 0, 9] = math.inf
        Vc2[table[2, at].long(), 5, 0, 9] = math.inf
        O, lse, _ = msa.attn_paged(Q, Kc, Vc2, *args[3:])
        assert torch.equal(lse, want_lse)
        assert bool(torch.isnan(O[0, :, 9]).all()), at
        assert bool((O[2] == 0).all()) and bool((lse[2] == -math.inf).all())
        O[0, :, 9] = want[0, :, 9]
        assert torch.equal(O, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_idle_slots_may_hold_anything(dtype):
    """Sequences without new tokens, with stale lengths and page ids, between sequences that have
    some: no error is recorded by the attention or by the cache write, and the outputs are those of
    the batch without them."""
    msa, g = _msa(), torch.Generator().manual_seed(19)
    T, L, page, Hq, Hkv, d = [2, 0, 1, 0, 0, 40, 0], [70, 50, 300, 9, 17, 64, 33], 16, 4, 2, 64
    Ks, Vs, Kc, Vc, table = ref.paginate(L, page, 1, Hkv, d, dtype, g, "cuda", math.nan)
    lens = torch.tensor(L, dtype=torch.int32)
    lens[1], lens[3], lens[4] = -7, page * table.shape[1] + 1, (1 << 31) - 1
    table[1, :], table[3, 0], table[6, 1] = -1, Kc.shape[0], 1 << 30
    Q = torch.randn((sum(T), Hq, d), generator=g).to(dtype).cuda()
    cu = ref.offsets(T)
    O, lse, ws = msa.attn_paged(Q, Kc, Vc, cu.cuda(), lens.cuda(), table)
    assert msa.msa_get_device_error(ws) == 0
    for b in (0, 2, 5):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        ref.assert_attention(O[rows], lse[rows],
                             ref.attention(Q[rows], Ks[b].cuda(), Vs[b].cuda()), f"sequence {b}")
    K, V = (torch.randn((sum(T), Hkv, d), generator=g).to(dtype).cuda() for _ in range(2))
    _, ws = msa.rope_append_paged(Q, K, V, None, cu.cuda(), lens.cuda(), table,
                                  msa.rope_frequencies(d), Kc, Vc)
    assert msa.msa_get_device_error(ws) == 0
    empty = torch.zeros_like(cu).cuda()                # a batch of idle slots alone
    O, _, ws = msa.attn_paged(Q[:0], Kc, Vc, empty, lens.cuda(), table)
    assert msa.msa_get_device_error(ws) == 0


def test_outputs_between_the_rows_of_inputs():
    """Outputs that share a buffer with inputs but no byte are not refused: in-place turns of two
    slices, turned rows between the rows of Q, and O inside the gap of a strided Q."""
    msa, g = _msa(), torch.Generator().manual_seed(23)
    n, H, d = 33, 2, 64
    f, pos = msa.rope_frequencies(d), torch.arange(n, dtype=torch.int32, device="cuda")
    room = torch.randn((2 * n, H, d), generator=g).to(BF16).cuda()
    Q, out = room[::2], room[1::2]
    want, _ = msa.rope(Q.contiguous(), None, pos, f)
    got, _ = msa.rope(Q, None, pos, f, Q_out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, want)
    room = torch.randn((n, 3 * H, d), generator=g).to(BF16).cuda()
    before = room.clone()
    msa.rope(room[:, :H], room[:, 2 * H:], pos, f, Q_out=room[:, H:2 * H], K_out=room[:, 2 * H:])
    want = msa.rope(before[:, :H].contiguous(), before[:, 2 * H:].contiguous(), pos, f)
    assert torch.equal(room[:, :H], before[:, :H])
    assert torch.equal(room[:, H:2 * H], want[0]) and torch.equal(room[:, 2 * H:], want[1])
    wide = torch.randn((2, 64 * H, d), generator=g).to(BF16).cuda()     # other strides on each side
    Q, out = wide[:, :H], wide[0, H:5 * H].view(2, 2 * H, d)[:, :H]
    want, _ = msa.rope(Q.contiguous(), None, pos[:2], f)
    msa.rope(Q, None, pos[:2], f, Q_out=out)
    assert torch.equal(out, want)
    O = wide[0, 5 * H:7 * H].view(2, H, d)
    cu = ref.offsets([2]).cuda()
    want = msa.attn_packed(Q.contiguous(), Q.contiguous(), Q.contiguous(), cu)[0]
    msa.attn_packed(Q, Q, Q, cu, out=O)
    assert torch.equal(O, want)
