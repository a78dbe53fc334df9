"""64-bit references of the serving operators (rotary positions, the paged cache write, full
causal attention) in plain torch, and error bounds worked out from the operators' roundings.

Rounding to a type is off by at most u = finfo(type).eps / 2 of the value."""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def rope(x, positions, inv_freq, layout, mscale=1.0, inverse=False):
    """(y, bound) in fp64.  fp32 arithmetic: the angle's remainder is rounded to 2^-25 turns
    (1.9e-7 rad), sincospif is good to 2 ulp (2.4e-7 for values up to 1), and the factor mscale,
    the two products and the sum round four times (4 u): at most 6.7e-7 (|a| + |b|) mscale;
    7e-7 is taken.  Then one rounding to the type."""
    rot = 2 * inv_freq.numel()
    ang = positions.double()[:, None, None] * inv_freq.double()
    c, s = ang.cos() * mscale, ang.sin() * (-mscale if inverse else mscale)
    y = x.double().clone()
    bound = torch.zeros_like(y)
    ia = torch.arange(rot // 2) if layout == "half" else torch.arange(0, rot, 2)
    ib = ia + (rot // 2 if layout == "half" else 1)
    a, b = x.double()[..., ia], x.double()[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    err = 7e-7 * (a.abs() + b.abs()) * abs(mscale)
    u = U[x.dtype]
    bound[..., ia] = err + u * (y[..., ia].abs() + err)
    bound[..., ib] = err + u * (y[..., ib].abs() + err)
    return y, bound


def attention(Q, K, V, scale=0.0):
    """One sequence: Q [T, Hq, d] at the last T of K's L positions.  (O, lse, O_bound, lse_bound)
    in fp64.

    A score is a d-term fp32 sum, off by at most e = scale (d + 8) 2^-23 sum |q k| (each of the
    additions may truncate, and the scaling rounds); with the running maximum m it enters
    exp(s - m) where the factor scale log2(e) is rounded too: (s - m) 2^-23 more.  exp itself is
    good to 2^-21.  The sums over L keys add at most L 2^-23 relative.  So with
    A = sum w |v|:  |dO| <= A (2 e + 2 L 2^-23 + 2^-18 + r) + u |O| , r = 2^-8 for bf16 (the
    weights' rounding for the product with V), 0 for fp32, where 2^-18 covers 2^-23 times
    scores up to 2 * 12 and the 2^-21 terms."""
    T, Hq, d = Q.shape
    L, Hkv = K.shape[0], K.shape[1]
    scale = scale if scale > 0 else 1.0 / math.sqrt(d)
    dev = Q.device
    O = torch.zeros((T, Hq, d), dtype=torch.float64, device=dev)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=dev)
    Ob, lb = torch.zeros_like(O), torch.zeros_like(lse)
    if T == 0 or L == 0:
        return O, lse, Ob, lb
    r, u = (2.0 ** -8 if Q.dtype == torch.bfloat16 else 0.0), U[Q.dtype]
    late = torch.arange(L, device=dev)[None] > torch.arange(L - T, L, device=dev)[:, None]
    some = ~late.all(1)
    for h in range(Hq):
        g = h // (Hq // Hkv)
        q, k, v = Q[:, h].double(), K[:, g].double(), V[:, g].double()
        s = (q @ k.T) * scale
        e = scale * (d + 8) * 2.0 ** -23 * (q.abs() @ k.abs().T)
        s = s.masked_fill(late, -math.inf)
        x = torch.logsumexp(s, 1)
        w = torch.exp(s - torch.where(some, x, 0.0)[:, None])
        for t in range(T):                       # values a row does not attend take no part
            n = L - T + t + 1
            if n <= 0:
                continue
            O[t, h] = w[t, :n] @ v[:n]
            A = w[t, :n] @ v[:n].abs()
            em = float(e[t, :n].max())
            Ob[t, h] = A * (2 * em + 2 * L * 2.0 ** -23 + 2.0 ** -18 + r) + u * O[t, h].abs()
            lse[t, h] = x[t]
            lb[t, h] = em + L * 2.0 ** -23 + 2.0 ** -18 + 2.0 ** -22 * float(x[t].abs())
    return O, lse, Ob, lb


def assert_attention(O, lse, ref, where=""):
    """Kernel outputs of one sequence against `attention`'s."""
    Or, lr, Ob, lb = (x.cpu() for x in ref)
    O, lse = O.double().cpu(), lse.double().cpu()
    empty = torch.isinf(lr) & (lr < 0)
    assert torch.equal(lse[empty], lr[empty]), f"{where}: lse of empty rows"
    assert bool((O[empty] == 0).all()), f"{where}: O of empty rows"
    dl, dO = (lse - lr).abs()[~empty], (O - Or).abs()
    assert bool(torch.isfinite(O).all()), f"{where}: O not finite"
    assert bool((dl <= lb[~empty]).all()), f"{where}: lse off by {float((dl - lb[~empty]).max())}"
    over = dO - Ob
    assert bool((over <= 1e-30).all()), \
        f"{where}: O off by {float(dO.flatten()[over.argmax()])}, " \
        f"bound {float(Ob.flatten()[over.argmax()])}, at {over.argmax().item()}"


def paginate(lens, page, num_extra, heads, d, dtype, g, device="cpu", fill=None):
    """Caches with the sequences' keys on shuffled pages: (K [per sequence], V, K_cache,
    V_cache, block_table).  `fill`: the value of every row that holds no key."""
    per = [-(-n // page) for n in lens]
    total = sum(per) + num_extra
    order = torch.randperm(total, generator=g)
    table = torch.full((len(lens), max(max(per), 1)), -1, dtype=torch.int32)
    shape = (total, page, heads, d)
    Kc, Vc = (torch.full(shape, fill if fill is not None else 0.0, dtype=dtype) for _ in range(2))
    Ks, Vs, at = [], [], 0
    for b, n in enumerate(lens):
        K, V = (torch.randn((n, heads, d), generator=g).to(dtype) for _ in range(2))
        Ks.append(K)
        Vs.append(V)
        for i in range(per[b]):
            pg = int(order[at])
            at += 1
            table[b, i] = pg
            part = slice(i * page, min(n, (i + 1) * page))
            Kc[pg, :part.stop - part.start] = K[part]
            Vc[pg, :part.stop - part.start] = V[part]
    return Ks, Vs, Kc.to(device), Vc.to(device), table.to(device)


def offsets(lens, start=0, device="cpu"):
    out = [start]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=device)
