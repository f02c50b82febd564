"""Operators of a decode step over compressed KV caches: what they are measured on.

A serving step of a model whose K and V live in HyperQuant caches (heads of 128, as
everywhere in this package) needs, next to the append, the read and the scores:

  norm_rope  per-head RMS norm of the new queries and keys and their position rotation;
  attention  attention of one or a few query tokens over the compressed K and V, with a
             sliding window and first tokens that stay visible (sinks);
  tree       the same for a tree of drafted tokens, whose own K and V are not cached yet;
  repack     a copy of ranges of a cache's tokens into another cache, re-cut into full
             chunks: fork, roll back, evict, merge one-token appends.

Cases are dicts; `prepare` makes the inputs on the GPU from the seed, the compressed caches
included (encoded here, in torch, by the format's definition), `run` makes one pass: in
elementary torch operations, or, where `own` is true, through the package's entry points.
"""
import math

import torch

own = False

D = 128                                  # head dimension = tile
N = {"Z": 1, "A2": 2, "D4": 4, "E8": 8}   # coordinates of a lattice block
# operating points of a cache: (lattice, Rice k, reduction of k for a block's last symbol)
# -> rms of the scaled coordinates and the bits per scalar that it gives (with dither)
POINTS = {
    ("E8", 0, 0): (1.53, 2.00), ("E8", 0, 1): (1.00, 1.70), ("E8", 1, 0): (3.30, 3.00), ("E8", 2, 1): (6.75, 3.97),
    ("D4", 1, 0): (1.90, 2.95), ("A2", 1, 1): (1.30, 2.76), ("Z", 1, 0): (1.60, 2.90), ("E8", 3, 0): (13.8, 5.00),
}
SCALE = 1.0 / math.sqrt(D)
OUTLIERS, OUTLIER_SCALE = 4, 8.0         # K channels of each head with larger entries


def listed():
    return [
        # one new token of a model with 32 query and 8 KV heads, far into a long text
        rope_case("norm_rope, one token", 1, 32, 8, 100003),
        # the drafted tokens of one speculative step
        rope_case("norm_rope, 61 tokens", 61, 32, 8, 4099),
        # the chunk of a long prompt; interleaved pairs, a part of each head rotated
        rope_case("norm_rope, 8191 tokens", 8191, 32, 8, 0, rot=64, interleaved=1),
        # a chat turn: a short prompt and the tokens generated since, appended one by one
        attn_case("attention, 1 of 300", "E8", 0, 0, 1, 8, 4, 300, ones=44),
        # one token over the 8 x 32768-token cache at 2 bits
        attn_case("attention, 1 of 32768", "E8", 0, 0, 1, 8, 4, 32768),
        # a window of 4096 tokens and 4 sinks over a longer cache without dither, at 4 bits
        attn_case("attention, window of 65536", "E8", 2, 1, 0, 8, 4, 65536, window=4096, sinks=4),
        # a small tree of drafts over a mid-sized cache
        attn_case("tree, 15 of 4099", "E8", 0, 0, 1, 8, 4, 4099, n_q=15, tree=1),
        # the largest tree, at the full cache
        attn_case("tree, 64 of 32768", "E8", 0, 0, 1, 8, 4, 32768, n_q=64, tree=1),
        # a chain of drafts over a Z cache of a model with one query head per KV head
        attn_case("tree, 5 of 1023", "Z", 1, 0, 0, 16, 1, 1023, n_q=5, tree=1, window=512, sinks=3),
        # a text generated token by token, merged into full chunks
        pack_case("repack, merge 1000", "E8", 0, 0, 8, 1000, 0, 0, 1000, ones=1000),
        # eviction: 4 sinks and the last 8191 tokens stay
        pack_case("repack, evict 32768", "E8", 0, 0, 8, 32768, 4, 24577, 32768),
        # a fork of a whole long cache at 4 bits
        pack_case("repack, fork 65535", "E8", 2, 1, 8, 65535, 0, 0, 65535),
    ]


def rope_case(name, tokens, heads_q, heads_k, pos0, rot=128, interleaved=0, norm=1):
    return dict(name=name, op="norm_rope", tokens=tokens, heads_q=heads_q, heads_k=heads_k, pos0=pos0, rot=rot,
                interleaved=interleaved, norm=norm)


def attn_case(name, lat, k, dk, dither, heads, group, length, n_q=1, tree=0, window=0, sinks=0, ones=0):
    """ones: the last of the tokens that were appended one by one (the others: 256 at a time)."""
    return dict(name=name, op="attention", lattice=lat, k=k, dk=dk, dither=dither, heads=heads, group=group,
                length=length, n_q=n_q, tree=tree, window=window, sinks=sinks, ones=ones)


def pack_case(name, lat, k, dk, heads, length, first, lo, hi, ones=0):
    """Kept: tokens [0, first) and [lo, hi)."""
    return dict(name=name, op="repack", lattice=lat, k=k, dk=dk, dither=1, heads=heads, length=length, first=first,
                lo=lo, hi=hi, ones=ones)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm_rope", "attention", "attention", "tree", "tree", "repack"))
    lat, k, dk = rng.choice(list(POINTS))
    heads = rng.choice((1, 2, 4, 8, 8))
    if op == "norm_rope":
        c = rope_case(None, _log(rng, 1, 8191), rng.choice((1, 7, 8, 24, 32)), rng.choice((1, 2, 5, 8)),
                      rng.randrange(200000), rng.choice((128, 128, 64, 96, 2)), rng.randrange(2),
                      rng.choice((1, 1, 0)))
    elif op == "repack":
        length = _log(rng, 1, 65535)
        lo = rng.randrange(length)
        hi = rng.randint(lo + 1, length)
        ones = rng.choice((0, 0, min(length, _log(rng, 1, 700))))
        c = pack_case(None, lat, k, dk, heads, length, rng.choice((0, min(lo, 4), min(lo, 33))), lo, hi, ones)
    else:
        length = _log(rng, 1, 32768)
        window, sinks = rng.choice(((0, 0), (0, 0), (_log(rng, 1, 8192), rng.choice((0, 1, 4, 40)))))
        n_q = _log(rng, 1, 64) if op == "tree" else min(length, rng.choice((1, 1, 1, 2, 5)))
        c = attn_case(None, lat, k, dk, rng.choice((1, 1, 0)), heads, rng.choice((1, 2, 4, 4, 7, 8)), length, n_q,
                      int(op == "tree"), window, sinks, rng.choice((0, 0, min(length, _log(rng, 1, 300)))))
    del c["name"]
    return c


def work(case):
    """Bytes and operations no implementation can do without: each visible compressed token read once, queries
    and outputs once; two products of 128 per query and visible token."""
    c = case
    if c["op"] == "norm_rope":
        elems = c["tokens"] * (c["heads_q"] + c["heads_k"]) * D
        return {"bytes": 4 * elems + 256 + 4 * c["rot"], "flops": elems * (3 * c["norm"] + 3)}
    bits = POINTS[c["lattice"], c["k"], c["dk"]][1]
    if c["op"] == "repack":
        return {"bytes": 2 * (c["first"] + c["hi"] - c["lo"]) * c["heads"] * D * bits / 8, "flops": 0}
    rows = c["n_q"] * c["heads"] * c["group"]
    n = c["length"]
    if c["window"]:
        n = min(n, c["sinks"] + c["window"] + (0 if c["tree"] else c["n_q"] - 1))
    drafts = c["n_q"] if c["tree"] else 0
    return {"bytes": 2 * n * c["heads"] * D * bits / 8 + 4 * rows * D + 4 * drafts * c["heads"] * D,
            "flops": 4 * rows * (n + drafts / 2) * D}


# ---------------------------------------------------------------------- the format, in elementary operations
def _i64(v):
    return v - (1 << 64) if v >= 1 << 63 else v


def _shr(z, n):
    """Logical shift right of int64 words."""
    return (z >> n) & ((1 << (64 - n)) - 1)


def _splitmix(s, i):
    z = (i + 1) * _i64(0x9E3779B97F4A7C15) + _i64(s)
    z = (z ^ _shr(z, 30)) * _i64(0xBF58476D1CE4E5B9)
    z = (z ^ _shr(z, 27)) * _i64(0x94D049BB133111EB)
    return z ^ _shr(z, 31)


def _signs(seed, device):
    """The sign diagonal D as +-1 (fp32 [128])."""
    h = _splitmix(seed ^ 0x5349474E, torch.arange(D, device=device))
    return torch.where(h < 0, -1.0, 1.0).float()


def _fwht(x):
    """Unnormalised Walsh-Hadamard transform of the last dimension, radix-2 stages 1, 2, ..., 64."""
    shape = x.shape
    h = 1
    while h < D:
        y = x.reshape(-1, D // (2 * h), 2, h)
        x = torch.stack((y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]), 2)
        h *= 2
    return x.reshape(shape)


def _first_max(x):
    """One-hot of the first largest entry of the last dimension."""
    i = torch.arange(x.shape[-1], device=x.device)
    hit = x == x.max(-1, keepdim=True).values
    first = torch.where(hit, i, x.shape[-1]).min(-1, keepdim=True).values
    return i == first


def _dn(y):
    """Nearest point of D_n: rounded coordinates; on an odd sum the farthest one goes to its other neighbour."""
    f = torch.round(y)
    r = y - f
    odd = f.sum(-1, keepdim=True).remainder(2) != 0
    step = torch.where(r >= 0, 1.0, -1.0).to(y.dtype)
    return f + torch.where(odd & _first_max(r.abs()), step, 0.0)


def _nearest(lat, v):
    """Codes (as floats) of the nearest lattice points of v [..., 128]."""
    n = N[lat]
    if n == 1:
        return torch.round(v)
    v = v.unflatten(-1, (-1, n))
    if lat == "D4":
        q = _dn(v)
    elif lat == "E8":
        a, b = 2 * _dn(v * 0.5), 2 * _dn((v - 1) * 0.5) + 1
        da, db = (v - a).double().square().sum(-1, keepdim=True), (v - b).double().square().sum(-1, keepdim=True)
        q = torch.where(db < da, b, a)
    else:
        t = torch.stack((v[..., 0], v[..., 1] * torch.tensor(1 / math.sqrt(3), dtype=v.dtype)), -1)
        a, b = 2 * torch.round(t), 2 * torch.round(t - 0.5) + 1
        da, db = ((v - _point(lat, c)).double().square().sum(-1, keepdim=True) for c in (a, b))
        q = torch.where(db < da, b, a)
    return q.flatten(-2)


def _point(lat, q):
    """The points that codes stand for; q [..., 128] or [..., 2]."""
    if lat != "A2":
        return q
    w = torch.tensor([0.5, math.sqrt(3) / 2], dtype=q.dtype, device=q.device)
    return (q.unflatten(-1, (-1, 2)) * w).flatten(-2)


def _uniform(lat, seed, tokens, heads):
    """The dither's uniforms on the lattice's box, fp32 [heads, tokens, 128]; tokens: their positions."""
    dev = tokens.device
    pair = (tokens[None, :, None] * heads + torch.arange(heads, device=dev)[:, None, None]) * (D // 2)
    h = _splitmix(seed ^ 0x44495448, pair + torch.arange(D // 2, device=dev))
    r = torch.stack((_shr(h, 40), _shr(h, 8) & 0xFFFFFF), -1).flatten(-2).float() * 2.0 ** -24
    box = torch.tensor({"Z": [1.0], "A2": [1.0, math.sqrt(3)], "D4": [2.0], "E8": [4.0]}[lat], device=dev)
    return r * box.repeat(D // box.numel())


def _dither(lat, seed, tokens, heads):
    w = _uniform(lat, seed, tokens, heads)
    return w - _point(lat, _nearest(lat, w))


def _symbols(lat, q):
    """Codes (int64 [..., 128]) -> (zigzag symbols, coset bits [..., 16] or None)."""
    n = N[lat]
    if n == 1:
        m, coset = q, None
    else:
        b = q.unflatten(-1, (-1, n))
        coset = None
        if lat == "E8":
            coset = b[..., 0] & 1
            b = (b - coset[..., None]) >> 1
        p = b[..., :-1].sum(-1) & 1
        m = torch.cat((b[..., :-1], ((b[..., -1] - p) >> 1)[..., None]), -1).flatten(-2)
    return (m << 1) ^ (m >> 63), coset


def _codes(lat, z, coset):
    """The inverse of _symbols."""
    m = (z >> 1) ^ -(z & 1)
    n = N[lat]
    if n == 1:
        return m
    b = m.unflatten(-1, (-1, n))
    p = b[..., :-1].sum(-1) & 1
    q = torch.cat((b[..., :-1], (2 * b[..., -1] + p)[..., None]), -1)
    if lat == "E8":
        q = 2 * q + coset[..., None]
    return q.flatten(-2)


def _rice(lat, k, dk, device):
    """Rice parameter of each of a tile's 128 symbols, and where its remainder bits start."""
    kk = torch.full((D,), k, dtype=torch.int64, device=device)
    if N[lat] > 1:
        kk[N[lat] - 1 :: N[lat]] = max(k - dk, 0)
    return kk, torch.cumsum(kk, 0) - kk


def _chunks(starts, counts, heads, device):
    """Where tokens go for appends of counts[a] tokens from position starts[a] on: per (head, cached token) the chunk
    and the tile in it; tiles per chunk; the tokens' positions; the first chunk of each append."""
    starts, counts = (torch.tensor(v, dtype=torch.int64, device=device) for v in (starts, counts))
    per = (counts + 31) // 32
    first = torch.cumsum(per * heads, 0) - per * heads
    a = torch.repeat_interleave(torch.arange(len(counts), device=device), counts)
    i = torch.arange(len(a), device=device) - (torch.cumsum(counts, 0) - counts)[a]
    chunk = first[a] + torch.arange(heads, device=device)[:, None] * per[a] + i // 32
    tiles = torch.zeros(int((per * heads).sum()), dtype=torch.int64, device=device)
    tiles.index_add_(0, chunk.flatten(), torch.ones_like(chunk).flatten())
    return chunk, (i % 32).expand_as(chunk), tiles, starts[a] + i, first


def _planes(lat, tiles, rem_bits):
    """Words of each chunk's coset and remainder planes."""
    return ((16 * tiles + 31) // 32 if lat == "E8" else 0 * tiles), (tiles * rem_bits + 31) // 32


def _encode(lat, k, dk, z, coset, where):
    """Symbols [heads, tokens, 128] -> stream words (int32) and chunk offsets."""
    chunk, ti, tiles, _, _ = where
    dev = z.device
    kk, kpos = _rice(lat, k, dk, dev)
    rem = int(kk.sum())
    run = torch.cumsum((z >> kk) + 1, -1)                      # a codeword's end within its tile's unary bits
    order = torch.cumsum(tiles, 0) - tiles
    tile = (order[chunk] + ti)                                 # index among all tiles, in stream order
    length = torch.zeros(tile.numel(), dtype=torch.int64, device=dev)
    length[tile.flatten()] = run[..., -1].flatten()
    end = torch.cumsum(length, 0)
    ustart = (end - length) - (end - length)[order].repeat_interleave(tiles)
    ubits = torch.zeros_like(tiles).index_add_(0, torch.repeat_interleave(torch.arange(len(tiles), device=dev), tiles),
                                               length)
    nc, nr = _planes(lat, tiles, rem)
    off = torch.zeros(len(tiles) + 1, dtype=torch.int64, device=dev)
    off[1:] = torch.cumsum(nc + nr + (ubits + 31) // 32, 0)
    bits = torch.zeros(int(off[-1]) * 32, dtype=torch.uint8, device=dev)
    if lat == "E8":
        pos = (32 * off[:-1][chunk] + 16 * ti)[..., None] + torch.arange(16, device=dev)
        bits[pos.flatten()] = coset.flatten().to(torch.uint8)
    base = 32 * (off[:-1] + nc)[chunk] + rem * ti
    for j in range(k):
        on = kk > j
        bits[(base[..., None] + (kpos + j)[on]).flatten()] = ((z[..., on] >> j) & 1).flatten().to(torch.uint8)
    base = 32 * (off[:-1] + nc + nr)[chunk] + ustart[tile]
    bits[(base[..., None] + run - 1).flatten()] = 1
    by = torch.arange(32, device=dev)
    words = torch.cat([(b.view(-1, 32).long() << by).sum(-1) for b in bits.split(1 << 26)])
    return torch.where(words >= 1 << 31, words - (1 << 32), words).int(), off


def _decode(lat, k, dk, words, off, where):
    """The inverse of _encode: -> (symbols, coset bits)."""
    chunk, ti, tiles, _, _ = where
    dev = words.device
    kk, kpos = _rice(lat, k, dk, dev)
    rem = int(kk.sum())
    nc, nr = _planes(lat, tiles, rem)
    words = words[: int(off[-1])]
    bits = ((words[:, None] >> torch.arange(32, device=dev)) & 1).to(torch.uint8).flatten()
    size = off[1:] - off[:-1]
    into = torch.arange(len(words), device=dev) - off[:-1].repeat_interleave(size)
    unary = bits.view(-1, 32) * (into >= (nc + nr).repeat_interleave(size))[:, None].to(torch.uint8)
    ends = unary.flatten().nonzero().flatten()                  # 128 per tile, in stream order
    first = 128 * (torch.cumsum(tiles, 0) - tiles)
    before = torch.cat((ends.new_zeros(1), ends[:-1] + 1))
    before[first] = 32 * (off[:-1] + nc + nr)
    quot = (ends - before).view(-1, D)[(first // D)[chunk] + ti]
    z = quot << kk
    base = 32 * (off[:-1] + nc)[chunk] + rem * ti
    for j in range(k):
        on = kk > j
        z[..., on] += bits[base[..., None] + (kpos + j)[on]].long() << j
    coset = None
    if lat == "E8":
        pos = (32 * off[:-1][chunk] + 16 * ti)[..., None] + torch.arange(16, device=dev)
        coset = bits[pos].long()
    return z, coset


def _appends(case):
    """Token positions at which the cache's appends start, and their sizes."""
    bulk = case["length"] - case["ones"]
    counts = [min(256, bulk - t) for t in range(0, bulk, 256)] + [1] * case["ones"]
    starts, t = [], 0
    for n in counts:
        starts.append(t)
        t += n
    return starts, counts


def _codes_of(case, g, seed, outliers):
    """What a cache holds: codes [heads, tokens, 128] of random vectors, and alpha."""
    lat, heads, n = case["lattice"], case["heads"], case["length"]
    dev = g.device
    x = torch.randn(heads, n, D, generator=g, device=dev)
    if outliers:
        ch = torch.rand(heads, D, generator=g, device=dev).argsort(-1)[:, :OUTLIERS]
        x *= torch.ones(heads, D, device=dev).scatter_(1, ch, OUTLIER_SCALE)[:, None]
    x = x.to(torch.bfloat16).float()
    alpha = POINTS[lat, case["k"], case["dk"]][0]
    if outliers:
        alpha /= math.sqrt((D - OUTLIERS + OUTLIERS * OUTLIER_SCALE ** 2) / D)
    alpha = float(torch.tensor(alpha, dtype=torch.float32))
    v = _fwht(x * _signs(seed, dev)) * (alpha / math.sqrt(D))
    if case["dither"]:
        v += _dither(lat, seed, torch.arange(n, device=dev), heads)
    return _nearest(lat, v).long(), alpha


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(starts, counts, first, alpha):
    """The append table's rows: 32 bytes each."""
    fwd, inv = alpha / math.sqrt(D), 1.0 / (alpha * math.sqrt(D))
    n = len(starts)
    dev = first.device
    ints = torch.stack((first, torch.tensor(starts, device=dev)), 1).view(torch.uint8).view(n, 16)
    count = torch.tensor(counts, dtype=torch.int32, device=dev)[:, None].view(torch.uint8)
    f = torch.tensor([[alpha, fwd, inv]], dtype=torch.float32, device=dev).expand(n, 3).contiguous().view(torch.uint8)
    return torch.cat((ints, count, f), 1).flatten()


def _cache(case, q, alpha, seed):
    """A compressed cache as a program holds it: buffers on the device, counters on the host."""
    starts, counts = _appends(case)
    dev = q.device
    where = _chunks(starts, counts, case["heads"], dev)
    z, coset = _symbols(case["lattice"], q)
    words, off = _encode(case["lattice"], case["k"], case["dk"], z, coset, where)
    return {"words": words, "offsets": off, "table": _rows(starts, counts, where[4], alpha),
            "tail": off[-1].expand(2).contiguous(), "stats": torch.zeros(40, dtype=torch.uint8, device=dev),
            "alpha": alpha, "seed": seed, "starts": starts, "counts": counts}


def _seeds(seed):
    return (seed * 2 + 1) & 0xFFFFFFFF, (seed * 2 + 2) & 0xFFFFFFFF


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "norm_rope":
        return _prepare_rope(case, g)
    if case["op"] == "repack":
        q, alpha = _codes_of(case, g, _seeds(seed)[0], True)
        src = _cache(case, q, alpha, _seeds(seed)[0])
        kept = [(0, case["first"])] * (case["first"] > 0) + [(case["lo"], case["hi"])]
        chunks = case["heads"] * sum((b - a + 31) // 32 for a, b in kept)
        dev = q.device
        # room for the kept tokens at their rate and a margin, as a program sizes a cache before it knows its stream
        room = 1.15 * work(case)["bytes"] / 2 / 4 + 40 * chunks
        dst = {"words": torch.zeros(int(room), dtype=torch.int32, device=dev),
               "offsets": torch.zeros(chunks + 1, dtype=torch.int64, device=dev),
               "table": torch.zeros(32 * len(kept), dtype=torch.uint8, device=dev),
               "tail": torch.zeros(2, dtype=torch.int64, device=dev),
               "stats": torch.zeros(40, dtype=torch.uint8, device=dev), "seed": src["seed"]}
        return {"case": case, "src": src, "dst": dst, "kept": kept}
    state = {"case": case}
    for name, s in zip("kv", _seeds(seed)):
        q, alpha = _codes_of(case, g, s, name == "k")
        state[name] = _cache(case, q, alpha, s)
        del q
    state.update(_queries(case, g))
    return state


def _queries(case, g):
    n, heads = case["n_q"], case["heads"]
    dev = g.device
    s = {"q": torch.randn(n, heads * case["group"], D, generator=g, device=dev).to(torch.bfloat16)}
    if case["tree"]:
        s["kd"], s["vd"] = (torch.randn(heads, n, D, generator=g, device=dev).to(torch.bfloat16) for _ in "kv")
        # each draft's parent is an earlier one, or the last cached token
        parent = (torch.rand(n, generator=g, device=dev) * torch.arange(n, device=dev)).long() - 1
        parent = torch.where(torch.rand(n, generator=g, device=dev) < 0.5, torch.arange(n, device=dev) - 1, parent)
        mask, up = [], parent.tolist()
        for i in range(n):
            mask.append((mask[up[i]] if up[i] >= 0 else 0) | (1 << i))
        s["mask"] = torch.tensor([_i64(m) for m in mask], device=dev)
    return s


def _prepare_rope(case, g):
    n, hq, hk = case["tokens"], case["heads_q"], case["heads_k"]
    dev = g.device
    half = case["rot"] // 2
    return {"case": case,
            # the projection's output: queries, keys and values of each token in one row
            "qkv": torch.randn(n, (hq + 2 * hk), D, generator=g, device=dev).to(torch.bfloat16),
            "wq": (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16),
            "wk": (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16),
            "freq": 500000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half),
            "pos": case["pos0"] + torch.arange(n, device=dev),
            "q": torch.empty(n, hq, D, dtype=torch.bfloat16, device=dev),
            "k": torch.empty(hk, n, D, dtype=torch.bfloat16, device=dev)}


# ---------------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    return {"norm_rope": _plain_rope, "attention": _plain_attention, "repack": _plain_repack}[state["case"]["op"]](state)


def _plain_rope(s):
    c = s["case"]
    half = c["rot"] // 2
    angle = s["pos"].double()[:, None] * s["freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def one(x, w):
        x = x.float()
        if c["norm"]:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        r = x[..., : c["rot"]]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :half], r[..., half:])
        u, v = a * cos - b * sin, b * cos + a * sin
        r = torch.stack((u, v), -1).flatten(-2) if c["interleaved"] else torch.cat((u, v), -1)
        return torch.cat((r, x[..., c["rot"] :]), -1)

    hq, hk = c["heads_q"], c["heads_k"]
    return {"q": one(s["qkv"][:, :hq], s["wq"]).to(torch.bfloat16),
            "k": one(s["qkv"][:, hq : hq + hk], s["wk"]).transpose(0, 1).contiguous().to(torch.bfloat16)}


def _plain_read(case, cache):
    """Every cached vector, fp32 [heads, tokens, 128]."""
    lat = case["lattice"]
    dev = cache["words"].device
    where = _chunks(cache["starts"], cache["counts"], case["heads"], dev)
    z, coset = _decode(lat, case["k"], case["dk"], cache["words"], cache["offsets"], where)
    x = _point(lat, _codes(lat, z, coset).float())
    if case["dither"]:
        x = x - _dither(lat, cache["seed"], where[3], case["heads"])
    x = _fwht(x * (1.0 / (cache["alpha"] * math.sqrt(D))))
    return x * _signs(cache["seed"], dev)


def _seen(c, mask, device):
    """Which cached tokens (and drafts) each query sees: bool [n_q, length (+ n_q)]."""
    t = torch.arange(c["length"], device=device)
    if c["tree"]:
        drafts = (mask[:, None] >> torch.arange(c["n_q"], device=device)) & 1
        pos = c["length"] - 1 + drafts.sum(-1)
    else:
        pos = c["length"] - c["n_q"] + torch.arange(c["n_q"], device=device)
    t, keep = t[None], t[None] <= pos[:, None]
    if c["tree"]:
        t, keep = torch.cat((t, pos[None]), 1), torch.cat((keep, drafts > 0), 1)
    if c["window"]:
        keep = keep & ((t > pos[:, None] - c["window"]) | (t < c["sinks"]))
    return keep


def _attend(c, q, k, v, keep):
    """q [n_q, heads * group, 128]; k, v [heads, tokens, 128]; keep [n_q, tokens]."""
    q = q.unflatten(1, (c["heads"], c["group"])).permute(1, 2, 0, 3)
    s = (q.flatten(1, 2) @ k.transpose(1, 2)).unflatten(1, (c["group"], c["n_q"])) * SCALE
    s = s.masked_fill(~keep, -math.inf)
    top = s.max(-1, keepdim=True).values.clamp(min=-3e38)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(1, 2) @ v).unflatten(1, (c["group"], c["n_q"])) / torch.where(total > 0, total, 1.0)
    return o.permute(2, 0, 1, 3).flatten(1, 2)


def _plain_attention(s):
    c = s["case"]
    k, v = _plain_read(c, s["k"]), _plain_read(c, s["v"])
    if c["tree"]:
        k, v = torch.cat((k, s["kd"].float()), 1), torch.cat((v, s["vd"].float()), 1)
    return _attend(c, s["q"].float(), k, v, _seen(c, s.get("mask"), k.device)).to(torch.bfloat16)


def _plain_repack(s):
    c, src, dst = s["case"], s["src"], s["dst"]
    dev = src["words"].device
    where = _chunks(src["starts"], src["counts"], c["heads"], dev)
    z, coset = _decode(c["lattice"], c["k"], c["dk"], src["words"], src["offsets"], where)
    starts, counts = [a for a, _ in s["kept"]], [b - a for a, b in s["kept"]]
    to = _chunks(starts, counts, c["heads"], dev)
    z, coset = z[:, to[3]], None if coset is None else coset[:, to[3]]
    words, off = _encode(c["lattice"], c["k"], c["dk"], z, coset, to)
    out = torch.zeros_like(dst["words"])
    out[: len(words)] = words
    return {"words": out, "offsets": off, "table": _rows(starts, counts, to[4], src["alpha"])}


# ---------------------------------------------------------------------- through the package
def _handle(hq, case, cache, tokens, chunks, appends):
    p = hq.make_params(case["lattice"], 1.0, case["k"], cache["seed"], case["dither"], dk_last=case["dk"])
    return hq.hq_kv_cache(cache["words"].data_ptr(), cache["words"].numel(), cache["offsets"].data_ptr(),
                          cache["offsets"].numel(), cache["table"].data_ptr(), cache["table"].numel() // 32,
                          cache["tail"].data_ptr(), cache["stats"].data_ptr(), case["heads"], D, p, tokens, chunks,
                          appends)


def _own_cache(hq, case, cache):
    return _handle(hq, case, cache, case["length"], cache["offsets"].numel() - 1, len(cache["counts"]))


def _run_own(s):
    import lattice_entropy_coded_b200 as hq
    c = s["case"]
    if c["op"] == "norm_rope":
        if "spec" not in s:
            s["spec"] = hq.rope_spec(rot_dim=c["rot"], interleaved=c["interleaved"], norm=c["norm"], eps=1e-6)
        n, m = c["heads_q"], c["heads_k"]
        hq.hq_qk_norm_rope(s["qkv"][:, :n], s["qkv"][:, n : n + m].transpose(0, 1), s["spec"], s["freq"], s["q"], s["k"],
                           s["wq"], s["wk"], positions=s["pos"])
        return {"q": s["q"], "k": s["k"]}
    if c["op"] == "repack":
        if "from" not in s:
            s["from"], s["to"] = _own_cache(hq, c, s["src"]), _handle(hq, c, s["dst"], 0, 0, 0)
            s["ws"] = torch.empty(hq.hq_kv_repack_workspace_bytes(c["heads"], s["kept"]), dtype=torch.uint8,
                                  device=s["dst"]["words"].device)
        hq.hq_kv_repack(s["from"], s["to"], s["kept"], s["ws"])
        return {n: s["dst"][n] for n in ("words", "offsets", "table")}
    if "ck" not in s:
        s["ck"], s["cv"] = _own_cache(hq, c, s["k"]), _own_cache(hq, c, s["v"])
        s["spec"] = hq.attn_spec(c["length"], SCALE, c["n_q"], c["group"], window=c["window"], sinks=c["sinks"])
        s["ws"] = torch.empty(hq.hq_kv_attention_workspace_bytes(c["heads"], s["spec"]), dtype=torch.uint8,
                              device=s["q"].device)
        s["out"] = torch.empty_like(s["q"])
    if c["tree"]:
        hq.hq_kv_tree_attention(s["ck"], s["cv"], s["spec"], s["q"], s["kd"], s["vd"], s["mask"], s["out"], s["ws"])
    else:
        hq.hq_kv_attention(s["ck"], s["cv"], s["spec"], s["q"], s["out"], s["ws"])
    return s["out"]


# ---------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    """What the operators are defined to give, in 64 bits: the cached vectors come from the codes that were
    encoded, through the dense Hadamard matrix; a repacked stream is whole numbers only."""
    g = _generator(seed)
    if case["op"] == "repack":
        return None
    if case["op"] == "norm_rope":
        return _exact_rope(case, _prepare_rope(case, g))
    kv = [_exact_vectors(case, *_codes_of(case, g, s, i == 0), s) for i, s in enumerate(_seeds(seed))]
    s = _queries(case, g)
    if case["tree"]:
        kv = [torch.cat((x, s[n].double()), 1) for x, n in zip(kv, ("kd", "vd"))]
    return _exact_softmax(case, s["q"].double(), kv[0], kv[1], s.get("mask"))


def _exact_vectors(case, q, alpha, seed):
    lat, dev = case["lattice"], q.device
    n = N[lat]
    z = q.double()
    if case["dither"]:
        w = _uniform(lat, seed, torch.arange(q.shape[1], device=dev), case["heads"]).double().view(-1, n)
        z = z - (w - _exact_closest(lat, w)).view(z.shape) if lat != "A2" else z
    if lat == "A2":
        step = torch.tensor([0.5, math.sqrt(0.75)], dtype=torch.float64, device=dev)
        z = (z.view(-1, 2) * step)
        z = (z - (w - _exact_closest(lat, w)) if case["dither"] else z).view(q.shape)
    i = torch.arange(D, device=dev)
    ones = sum(((i[:, None] & i) >> b) & 1 for b in range(7))
    h = (1.0 - 2.0 * (ones & 1)).double()
    d = 1.0 - 2.0 * (_splitmix(seed ^ 0x5349474E, i) < 0).double()
    return (z @ h) * d / (alpha * math.sqrt(D))


def _exact_closest(lat, w):
    """The closest lattice point of each row: the lattice as a union of scaled integer lattices with even sums."""
    def even(y):
        f = (y + 0.5).floor()
        f = torch.where((y + 0.5 == f) & (f.remainder(2) == 1), f - 1, f)   # halves to the even side
        gap = y - f
        far = gap.abs().argmax(-1, keepdim=True)
        move = torch.where(gap.gather(-1, far) >= 0, 1.0, -1.0).double() * f.sum(-1, keepdim=True).remainder(2)
        return f.scatter_add(-1, far, move)

    if lat == "Z":
        return torch.round(w)
    if lat == "D4":
        return even(w)
    if lat == "E8":
        cands = [2 * even(w / 2), 2 * even((w - 1) / 2) + 1]
    else:
        unit = torch.tensor([1.0, math.sqrt(3.0)], dtype=torch.float64, device=w.device)
        cands = [torch.round(w / unit) * unit, (torch.round(w / unit - 0.5) + 0.5) * unit]
    dist = [(w - c).square().sum(-1, keepdim=True) for c in cands]
    return torch.where(dist[1] < dist[0], cands[1], cands[0])


def _exact_softmax(c, q, k, v, mask):
    """Query by query: the visible tokens' softmax, and its average of their values."""
    out = torch.zeros_like(q)
    for i in range(c["n_q"]):
        at = list(range(c["length"]))
        pos = c["length"] - c["n_q"] + i
        if c["tree"]:
            depth = lambda j: bin(int(mask[j]) & 0xFFFFFFFFFFFFFFFF).count("1")  # noqa: E731
            pos = c["length"] - 1 + depth(i)
            at += [c["length"] - 1 + depth(j) if (int(mask[i]) >> j) & 1 else pos + 1 for j in range(c["n_q"])]
        at = torch.tensor(at, device=q.device)
        see = at <= pos
        if c["window"]:
            see &= (at > pos - c["window"]) | (at < c["sinks"])
        if bool(see.any()):
            qi = q[i].view(c["heads"], c["group"], D)
            s = torch.einsum("hgd,htd->hgt", qi, k[:, see]) / math.sqrt(D)
            out[i] = torch.einsum("hgt,htd->hgd", torch.softmax(s, -1), v[:, see]).reshape(-1, D)
    return out


def _exact_rope(c, s):
    """Pairs as complex numbers, turned by their angle."""
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=s["freq"].device), s["pos"].double()[:, None] * s["freq"])
    half = c["rot"] // 2
    hq, hk = c["heads_q"], c["heads_k"]
    got = []
    for x, w in ((s["qkv"][:, :hq], s["wq"]), (s["qkv"][:, hq : hq + hk], s["wk"])):
        x = x.double()
        if c["norm"]:
            x = x / (x.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
        i = torch.arange(half, device=x.device)
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        y = torch.complex(x[..., a], x[..., b]) * turn[:, None]
        x = x.clone()
        x[..., a], x[..., b] = y.real, y.imag
        got.append(x)
    return {"q": got[0], "k": got[1].transpose(0, 1)}
