"""Helpers shared by the tests of the KV serving operators: caches filled through the
binding, and attention in 64 bits over what hq_kv_read reconstructs."""
from __future__ import annotations

import math

import torch

import synth

# scaled-coordinate rms of about 2 bits per scalar at k = 0 on N(0, 1) rows
ALPHA = {"E8": 0.17 * 8, "D4": 0.8, "A2": 0.6, "Z": 0.8}


def pair(heads, appends, lat, k=0, dither=1, dk=0, alpha=None, seed=3, rotation=None, alphas=None, vk=None, spare=64):
    """(K cache, V cache) after appends of the given sizes; alphas: one per append (V's are 1.3 times K's)."""
    import lattice_entropy_coded_b200 as hq
    total = sum(appends)
    K, V = synth.kv(heads, max(total, 1), seed=seed)
    # outlier channels of x50 would leave one token with all the weight
    K = torch.where(K.float().abs() > 5, K.float() / 12, K.float()).to(torch.bfloat16)
    base = (ALPHA[lat] if alpha is None else alpha) * 2.0 ** k
    out = []
    for i, x in enumerate((K, V)):
        kk = k if i == 0 or vk is None else vk
        c = hq.KVCache(heads, total + spare, hq.make_params(lat, 1.0, kk, seed * 2 + i, dither, dk_last=dk),
                       bits_per_scalar=32.0, max_appends=len(appends) + 8, max_append_tokens=max(list(appends) + [spare]),
                       rotation=None if rotation is None else rotation[i])
        t = 0
        for j, n in enumerate(appends):
            a = base if alphas is None else alphas[j]
            c.append(x[:, t:t + n].contiguous().cuda(), a * (1.3 if i else 1.0))
            t += n
        assert hq.read_stats(c.stats)["status"] == 0
        out.append(c)
    torch.cuda.synchronize()
    return out


def vectors(cache, length=None, fill=0.0):
    """What the cache holds, fp64 [heads, length, 128] (positions it does not hold: `fill`)."""
    n = cache.tokens if length is None else length
    out = torch.full((cache.heads, max(n, 1), 128), fill, dtype=torch.float32, device="cuda")
    if n:
        cache.read(out[:, :n], n)
    return out[:, :n].double()


def seen(n_q, length, window, sinks, mask=None, held=None):
    """bool [n_q, length (+ n_q drafts)] from the definition, one entry at a time."""
    depth = [0] * n_q if mask is None else [bin(int(m) & ((1 << n_q) - 1)).count("1") for m in mask]
    rows = []
    for i in range(n_q):
        p = length - n_q + i if mask is None else length - 1 + depth[i]
        at = [(t, held is None or held(t)) for t in range(length)]
        if mask is not None:
            at += [(length - 1 + depth[j], bool((int(mask[i]) >> j) & 1)) for j in range(n_q)]
        rows.append([ok and t <= p and (window == 0 or t > p - window or t < sinks) for t, ok in at])
    return torch.tensor(rows, dtype=torch.bool, device="cuda").reshape(n_q, -1)


def attend(q, k, v, keep, group, scale):
    """fp64: (out [n_q, heads * group, 128], lse, sum of p |v|, scale |q| max |k|), for q [n_q, heads * group, 128]."""
    heads = k.shape[0]
    qd = q.double().unflatten(1, (heads, group))
    s = torch.einsum("nhgd,htd->nhgt", qd, k) * scale
    s = s.masked_fill(~keep[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True) if s.shape[-1] else torch.full((*s.shape[:-1], 1), -math.inf, device=s.device).double()
    p = torch.exp(s - top.clamp(min=-1e300))
    total = p.sum(-1, keepdim=True)
    w = p / torch.where(total > 0, total, 1.0)
    vis = keep.any(0)
    vv = torch.where(vis[None, :, None], v, 0.0)        # what nothing sees does not matter
    kk = torch.where(vis[None, :, None], k, 0.0)
    out = torch.einsum("nhgt,htd->nhgd", w, vv).flatten(1, 2)
    lse = (top.clamp(min=-1e300) + torch.log(total)).squeeze(-1)
    lse = torch.where(total.squeeze(-1) > 0, lse, -math.inf).flatten(1, 2)
    pv = torch.einsum("nhgt,ht->nhg", w, vv.norm(dim=-1)).flatten(1, 2)
    kn = kk.norm(dim=-1).amax(-1) if kk.shape[1] else torch.zeros(heads, device=q.device).double()
    qk = (qd.norm(dim=-1) * kn[:, None] * abs(scale)).flatten(1, 2)
    return out, lse, pv, qk


def tolerance(pv, qk, dither, tokens):
    """Bound of a row's L2 error and of its lse's, from the roundings alone (the rotation keeps L2 norms):
      scores    codes in fp16 (2^-11 of each: exact without dither for the codes here), the query as two fp16
                (2^-21 with the sum of both parts), fp32 sums of 128 products and of the rotations' stages
                (2^-24 each, 300 of them): |error| <= B = qk (2^-11 dither + 2^-21 + 300 2^-24);
      softmax   weights off by exp(2 B) - 1, and by the exponential's own 2^-22 and the weight's rounding to
                fp16, 2^-11 (2^-25 of the row's largest below 2^-14: tokens 2^-25 in all);
      values    codes in fp16 2^-11 (dither), sums in fp32 over the tokens, 2^-24 a product."""
    b = qk * (2.0 ** -11 * dither + 2.0 ** -21 + 300 * 2.0 ** -24)
    soft = torch.expm1(2 * b) + 2.0 ** -20
    rel = soft + 2.0 ** -11 + 2.0 ** -11 * dither + (tokens + 300) * 2.0 ** -24
    return rel * pv, b + 2.0 ** -18


def check(out, lse, q, k, v, keep, group, scale, dither):
    ref, rl, pv, qk = attend(q, k, v, keep, group, scale)
    tol, tl = tolerance(pv, qk, dither, keep.shape[1])
    # weights below 2^-14 of the largest round by up to 2^-25 of it
    tol = tol + keep.shape[1] * 2.0 ** -25 * torch.where(pv > 0, v.abs().nan_to_num().norm(dim=-1).amax() if v.numel() else 0.0, 0.0)
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    err = (out.double() - ref).norm(dim=-1)
    lim = tol + half * ref.norm(dim=-1) + 1e-30
    assert torch.isfinite(out).all()
    assert bool((err <= lim).all()), f"worst error / bound {float((err / lim).max()):.3f}"
    empty = ~torch.isfinite(rl)
    assert bool((out[empty] == 0).all())
    if lse is not None:
        assert torch.equal(torch.isinf(lse), empty) and bool((lse[empty] < 0).all())
        d = (lse.double() - rl)[~empty].abs()
        assert bool((d <= (tl + 2.0 ** -22 * rl.abs())[~empty]).all()), f"lse off by {float(d.max())}"
    return float((err / lim).max()) if err.numel() else 0.0
