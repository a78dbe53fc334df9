"""The serving operators' workloads: rotary positions, rotary positions with the write
into a paged cache, attention of new tokens over a paged cache, and attention over packed
whole prompts.

Each case names an operator and its sizes; `prepare` makes its inputs on the GPU, `run` is
one call (the library's with `own`, the formula in elementary torch operations without),
`work` the bytes and operations the call cannot do without, `exact` its value in 64 bits.

Sequence lengths are a function of the case (its "mix"), so that the work of a case does
not depend on the seed; values, page orders and positions come from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One decode step's queries and keys of 64 sequences, up to 2^20 tokens along.
        dict(name="rope_step", op="rope", n=64, Hq=32, Hkv=8, d=128, rot=128, layout="half",
             dtype="bf16", inverse=False, factor=1.0, far=1 << 20),
        # A long prompt's queries and keys; half of each head rotated, pairs side by side.
        dict(name="rope_prompt", op="rope", n=32768, Hq=64, Hkv=8, d=128, rot=64,
             layout="interleaved", dtype="bf16", inverse=False, factor=1.0, far=32768),
        # The gradient's way back, in fp32, with frequencies scaled for a longer context.
        dict(name="rope_back_f32", op="rope", n=8191, Hq=32, Hkv=8, d=64, rot=64, layout="half",
             dtype="f32", inverse=True, factor=8.0, far=131072),
        # One decode step of 64 sequences enters the cache.
        dict(name="append_step", op="append", B=64, new=1, long=2048, mix=1, Hq=32, Hkv=8,
             d=128, d_idx=64, page=64, rot=128, layout="half", dtype="bf16"),
        # Prompt chunks of a few sequences enter the cache.
        dict(name="append_chunks", op="append", B=7, new=2048, long=16384, mix=2, Hq=64, Hkv=4,
             d=128, d_idx=64, page=16, rot=64, layout="half", dtype="bf16"),
        # One token of one short conversation: what a single user waits for.
        dict(name="paged_one", op="paged", B=1, new=1, long=1000, mix=0, Hq=32, Hkv=8, d=128,
             page=64),
        # One decode step of 64 conversations of 2K to 16K tokens.
        dict(name="paged_step", op="paged", B=64, new=1, long=16384, mix=3, Hq=32, Hkv=8, d=128,
             page=64),
        # A serving step that mixes single tokens with prompt chunks of up to 512 tokens.
        dict(name="paged_mixed", op="paged", B=24, new=512, long=32768, mix=4, Hq=64, Hkv=8,
             d=128, page=16),
        # A 4096-token chunk at the end of a 128K prompt.
        dict(name="paged_chunk", op="paged", B=1, new=4096, long=131072, mix=0, Hq=32, Hkv=4,
             d=128, page=128),
        # Short prompts side by side, down to one token each.
        dict(name="prompts_short", op="prompts", B=16, total=1999, mix=5, Hq=8, Hkv=2, d=64),
        # Prompts of very different lengths in one pack.
        dict(name="prompts_packed", op="prompts", B=8, total=16384, mix=6, Hq=64, Hkv=8, d=128),
        # One 32K prompt.
        dict(name="prompt_long", op="prompts", B=1, total=32768, mix=0, Hq=32, Hkv=8, d=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "paged", "paged", "prompts", "prompts"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    R = rng.choice([1, 2, 4, 7, 8, 16])
    case = dict(op=op, Hq=Hkv * R, Hkv=Hkv, d=d)
    if op == "rope":
        case.update(n=_log_int(rng, 1, 32768), rot=rng.choice([d, d // 2, d // 4]),
                    layout=rng.choice(["half", "interleaved"]), dtype=rng.choice(["bf16", "f32"]),
                    inverse=rng.random() < 0.5, factor=rng.choice([1.0, 4.0, 32.0]),
                    far=_log_int(rng, 64, 1 << 20))
    elif op == "append":
        long = _log_int(rng, 16, 16384)
        case.update(B=_log_int(rng, 1, 64), new=_log_int(rng, 1, min(2048, long)), long=long,
                    mix=rng.randrange(1, 1 << 20), d_idx=rng.choice([0, 64, 128]),
                    page=rng.choice([16, 32, 48, 64, 128, 256]), rot=rng.choice([d, d // 2]),
                    layout=rng.choice(["half", "interleaved"]), dtype=rng.choice(["bf16", "f32"]))
    elif op == "paged":
        long = _log_int(rng, 16, 32768)
        new = 1 if rng.random() < 0.4 else _log_int(rng, 1, min(1024, long))
        most = max(1, min(64, (1 << 19) // long, (1 << 13) // new))
        case.update(B=_log_int(rng, 1, most), new=new, long=long, mix=rng.randrange(1, 1 << 20),
                    page=rng.choice([16, 32, 48, 64, 128, 256]))
    else:
        total = _log_int(rng, 16, 16384)
        case.update(B=_log_int(rng, 1, min(64, total)), total=total,
                    mix=rng.randrange(1, 1 << 20))
    return case


def _lengths(case):
    """(new tokens, keys) of each sequence."""
    rng, B = random.Random(case["mix"]), case["B"]
    if case["op"] == "prompts":
        if case["mix"] == 0:
            return [case["total"]], [case["total"]]
        w = [math.exp(rng.uniform(0.0, 3.5)) for _ in range(B)]
        T = [max(1, int(case["total"] * x / sum(w))) for x in w]
        T[T.index(max(T))] += case["total"] - sum(T)
        return T, T
    if case["mix"] == 0:
        return [case["new"]] * B, [case["long"]] * B
    lo = max(1, case["long"] // 8)
    L = [rng.randint(lo, case["long"]) for _ in range(B)]
    # two thirds of a mixed batch decode one token, the others bring a chunk
    T = [1 if case["new"] == 1 or rng.random() < 0.67 else min(l, _log_int(rng, 1, case["new"]))
         for l in L]
    if case["new"] > 1:
        T[0] = min(L[0], case["new"])
    return T, L


# ---------------------------------------------------------------- inputs

def _frequencies(rot, factor):
    """theta_i = 10000^(-2i/rot) radians a token; for a context `factor` times longer the slow
    ones (under one turn in 4096 tokens) are divided by factor, the fast ones (over 32 turns)
    kept, and those between blended linearly in their number of turns."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    turns = 4096.0 * f / (2.0 * math.pi)
    keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * keep + (f / factor) * (1.0 - keep)


def _offsets(lengths):
    off = [0]
    for x in lengths:
        off.append(off[-1] + x)
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    dt = DTYPES[case.get("dtype", "bf16")]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    s = dict(case)
    if case["op"] == "rope":
        n = case["n"]
        s.update(Q=normal(n, Hq, d), K=normal(n, Hkv, d), inv_freq=_frequencies(case["rot"],
                                                                                  case["factor"]),
                 positions=torch.randint(0, case["far"], (n,), generator=g, device="cuda",
                                         dtype=torch.int32),
                 mscale=1.0 + 0.1 * math.log(case["factor"]))
        return s
    T, L = _lengths(case)
    s.update(T=T, L=L, cu_seqlens=_offsets(T), Q=normal(sum(T), Hq, d))
    if case["op"] == "prompts":
        s.update(K=normal(sum(T), Hkv, d), V=normal(sum(T), Hkv, d))
        return s
    page = case["page"]
    per = [-(-x // page) for x in L]
    num_pages = sum(per) + 3
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(L), max(per)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    s.update(block_table=table, seq_lens=torch.tensor(L, dtype=torch.int32, device="cuda"),
             K_cache=normal(num_pages, page, Hkv, d), V_cache=normal(num_pages, page, Hkv, d))
    if case["op"] == "append":
        s.update(K=normal(sum(T), Hkv, d), V=normal(sum(T), Hkv, d),
                 inv_freq=_frequencies(case["rot"], 1.0), k_idx=None, k_idx_cache=None)
        if case["d_idx"]:
            s.update(k_idx=normal(sum(T), case["d_idx"]),
                     k_idx_cache=normal(num_pages, page, case["d_idx"]))
    return s


# ---------------------------------------------------------------- the plain forms

def _rotate(x, positions, inv_freq, layout, mscale=1.0, inverse=False):
    rot = 2 * inv_freq.numel()
    angle = positions.double()[:, None, None] * inv_freq        # far positions: 64-bit angles
    c = (angle.cos() * mscale).float()
    s = (angle.sin() * (-mscale if inverse else mscale)).float()
    x = x.float()
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _new_positions(s):
    """(sequence, position) of every new token, and the cache row that position has."""
    cu, n = s["cu_seqlens"].long(), s["Q"].shape[0]
    token = torch.arange(n, device="cuda")
    b = torch.searchsorted(cu, token, right=True) - 1
    p = s["seq_lens"].long()[b] - cu[b + 1] + token
    page = s["page"]
    return b, p, s["block_table"].long()[b, p // page] * page + p % page


def _attend(q, k, v, hidden=None):
    """softmax(q k^T / sqrt(d)) v in 32 bits over the last two axes; hidden: True where a key is
    not attended.  (o, lse)"""
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(q.shape[-1]))
    if hidden is not None:
        x.masked_fill_(hidden, -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    return torch.matmul(x, v) / total, (top + total.log()).squeeze(-1)


def _one_sequence(Q, K, V):
    """Causal attention of the last T of L positions: Q [T, Hq, d], K, V [L, Hkv, d]; scores are
    kept to 2^31 values at a time."""
    (T, Hq, d), (L, Hkv, _) = Q.shape, K.shape
    R = Hq // Hkv
    q = Q.float().view(T, Hkv, R, d).permute(1, 2, 0, 3)
    k, v = (x.float().permute(1, 0, 2)[:, None] for x in (K, V))
    key = torch.arange(L, device="cuda")
    step = max(1, (1 << 31) // (L * Hq))
    parts = []
    for t in range(0, T, step):
        row = torch.arange(t, min(T, t + step), device="cuda")
        parts.append(_attend(q[:, :, t:t + step], k, v, key > (row + L - T)[:, None]))
    o = torch.cat([x for x, _ in parts], 2).permute(2, 0, 1, 3).reshape(T, Hq, d)
    lse = torch.cat([x for _, x in parts], 2).permute(2, 0, 1).reshape(T, Hq)
    return o.to(Q.dtype), lse


def _plain_prompts(s):
    got = [_one_sequence(*x) for x in zip(*(s[n].split(s["T"]) for n in ("Q", "K", "V")))]
    return {"O": torch.cat([o for o, _ in got]), "lse": torch.cat([x for _, x in got])}


def _plain_paged(s):
    Q, Kc, Vc, T, L = s["Q"], s["K_cache"], s["V_cache"], s["T"], s["L"]
    Hq, Hkv, d = Q.shape[1], Kc.shape[2], Q.shape[2]
    if max(T) == 1:                                   # a decode step: one padded batch
        B = len(T)
        k, v = (x[s["block_table"].long()].view(B, -1, Hkv, d).permute(0, 2, 1, 3).float()
                for x in (Kc, Vc))
        hidden = torch.arange(k.shape[2], device="cuda") >= s["seq_lens"][:, None]
        o, lse = _attend(Q.float().view(B, Hkv, Hq // Hkv, d), k, v, hidden[:, None, None])
        return {"O": o.reshape(B, Hq, d).to(Q.dtype), "lse": lse.reshape(B, Hq)}
    got = [_one_sequence(q, Kc[t.long()].view(-1, Hkv, d)[:n], Vc[t.long()].view(-1, Hkv, d)[:n])
           for q, t, n in zip(Q.split(T), s["block_table"], L)]
    return {"O": torch.cat([o for o, _ in got]), "lse": torch.cat([x for _, x in got])}


def _plain_append(s):
    _, p, row = _new_positions(s)
    turn = (p, s["inv_freq"], s["layout"])
    s["K_cache"].view(-1, *s["K"].shape[1:])[row] = _rotate(s["K"], *turn).to(s["K"].dtype)
    s["V_cache"].view(-1, *s["V"].shape[1:])[row] = s["V"]
    if s["k_idx"] is not None:
        s["k_idx_cache"].view(-1, s["d_idx"])[row] = s["k_idx"]
    return {"Q": _rotate(s["Q"], *turn).to(s["Q"].dtype), "K_cache": s["K_cache"],
            "V_cache": s["V_cache"], "k_idx_cache": s["k_idx_cache"]}


def _plain_rope(s):
    turn = (s["positions"], s["inv_freq"], s["layout"], s["mscale"], s["inverse"])
    return {"Q": _rotate(s["Q"], *turn).to(s["Q"].dtype),
            "K": _rotate(s["K"], *turn).to(s["K"].dtype)}


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        import block_sparse_long_03_b200 as msa
        if s["op"] == "rope":
            q, k = msa.rope(s["Q"], s["K"], s["positions"], s["inv_freq"], layout=s["layout"],
                            mscale=s["mscale"], inverse=s["inverse"])
            return {"Q": q, "K": k}
        if s["op"] == "append":
            q, _ = msa.rope_append_paged(s["Q"], s["K"], s["V"], s["k_idx"], s["cu_seqlens"],
                                         s["seq_lens"], s["block_table"], s["inv_freq"],
                                         s["K_cache"], s["V_cache"], s["k_idx_cache"],
                                         layout=s["layout"])
            return {"Q": q, "K_cache": s["K_cache"], "V_cache": s["V_cache"],
                    "k_idx_cache": s["k_idx_cache"]}
        if s["op"] == "paged":
            o, lse, _ = msa.attn_paged(s["Q"], s["K_cache"], s["V_cache"], s["cu_seqlens"],
                                       s["seq_lens"], s["block_table"])
        else:
            o, lse, _ = msa.attn_packed(s["Q"], s["K"], s["V"], s["cu_seqlens"])
        return {"O": o, "lse": lse}
    return {"rope": _plain_rope, "append": _plain_append, "paged": _plain_paged,
            "prompts": _plain_prompts}[s["op"]](s)


# ---------------------------------------------------------------- what a pass needs

def work(case):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    size = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "rope":
        n, rot = case["n"], case["rot"]
        values = n * (Hq + Hkv)
        return {"bytes": 2 * values * d * size + 4 * n + 4 * rot, "flops": 3 * values * rot}
    T, L = _lengths(case)
    n = sum(T)
    if case["op"] == "append":
        row = 2 * (Hq + 2 * Hkv) * d * size + 2 * case["d_idx"] * size
        return {"bytes": n * (row + 4), "flops": 3 * n * (Hq + Hkv) * case["rot"]}
    pairs = sum(t * (l - t) + t * (t + 1) // 2 for t, l in zip(T, L))
    return {"bytes": 2 * n * Hq * d * 2 + 4 * n * Hq + 2 * sum(L) * Hkv * d * 2,
            "flops": 4 * d * Hq * pairs}


# ---------------------------------------------------------------- in 64 bits

def _exact_turn(x, positions, inv_freq, layout, mscale=1.0, inverse=False):
    """Each pair as a complex number times mscale e^(+-i angle)."""
    n, rot = inv_freq.numel(), 2 * inv_freq.numel()
    angle = positions.double().view(-1, 1, 1) * inv_freq.view(1, 1, -1)
    unit = torch.polar(torch.full_like(angle, mscale), -angle if inverse else angle)
    y = x.double().clone()
    re, im = ((slice(0, n), slice(n, rot)) if layout == "half"
              else (slice(0, rot, 2), slice(1, rot, 2)))
    z = torch.complex(y[..., re], y[..., im]) * unit
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_rows(Q, K, V):
    T, L, R, d = Q.shape[0], K.shape[0], Q.shape[1] // K.shape[1], Q.shape[2]
    o = torch.empty(Q.shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(Q.shape[:2], dtype=torch.float64, device="cuda")
    step = max(1, (1 << 28) // L)
    for h in range(Q.shape[1]):
        k, v = K[:, h // R].double(), V[:, h // R].double()
        for t in range(0, T, step):
            e = min(T, t + step)
            seen = L - T + e                              # no row of this piece sees more keys
            x = Q[t:e, h].double() @ k[:seen].T / math.sqrt(d)
            late = torch.arange(seen, device="cuda")[None] - torch.arange(t, e, device="cuda")[:, None]
            x[late > L - T] = -math.inf
            lse[t:e, h] = torch.logsumexp(x, 1)
            o[t:e, h] = torch.exp(x - lse[t:e, h, None]) @ v[:seen]
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "rope":
        turn = (s["positions"], s["inv_freq"], s["layout"], s["mscale"], s["inverse"])
        return {"Q": _exact_turn(s["Q"], *turn), "K": _exact_turn(s["K"], *turn)}
    first, rows, page = 0, [], s.get("page")
    O, lse = [], []
    for b, (t, l) in enumerate(zip(s["T"], s["L"])):
        q = s["Q"][first:first + t]
        if s["op"] == "prompts":
            k, v = s["K"][first:first + t], s["V"][first:first + t]
        else:
            j = torch.arange(l, device="cuda")
            where = s["block_table"][b].long()[j.div(page, rounding_mode="floor")] * page + j % page
            rows.append((where[l - t:], j[l - t:]))
            k, v = (s[n].flatten(0, 1)[where] for n in ("K_cache", "V_cache"))
        first += t
        if s["op"] != "append":
            o, x = _exact_rows(q, k, v)
            O.append(o)
            lse.append(x)
    if s["op"] != "append":
        return {"O": torch.cat(O), "lse": torch.cat(lse)}
    where, p = (torch.cat(x) for x in zip(*rows))
    got = {"Q": _exact_turn(s["Q"], p, s["inv_freq"], s["layout"])}
    for name, new in (("K", _exact_turn(s["K"], p, s["inv_freq"], s["layout"])), ("V", s["V"]),
                      ("k_idx", s["k_idx"])):
        cache = s[name + "_cache"]
        if cache is not None:
            cache = cache.double()
            cache.flatten(0, 1)[where] = new.double()
        got[name + "_cache"] = cache
    return got
