"""Attention over V whose appends have scales far apart, and beside tokens that take nearly all the weight: what a row
sees keeps its bits, whatever else lies in the cache.  Errors are bounded by the visible tokens alone."""
import math

import pytest
import torch

import kvtest as T

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def _hq():
    import lattice_entropy_coded_b200 as hq
    return hq


def _cache(heads, parts, lat, seed, dither, k=0):
    """A cache of appends (x [heads, n, 128], alpha); with each token's scale, fp64 [tokens]."""
    hq = _hq()
    total = sum(x.shape[1] for x, _ in parts)
    c = hq.KVCache(heads, total + 64, hq.make_params(lat, 1.0, k, seed, dither), bits_per_scalar=40.0,
                   max_appends=len(parts) + 8, max_append_tokens=max(x.shape[1] for x, _ in parts))
    e = []
    for x, alpha in parts:
        c.append(x.to(torch.bfloat16).contiguous(), alpha)
        e += [1.0 / (alpha * math.sqrt(128))] * x.shape[1]
    assert hq.read_stats(c.stats)["status"] == 0
    return c, torch.tensor(e, dtype=torch.float64, device="cuda")


def _check(out, lse, q, ck, cv, e, keep, group):
    """kvtest.tolerance (roundings relative to each visible token's share), and what fp16 adds at its lower end:
    weights times scales below 2^-25 of the row's largest are off by up to 2^-36 of it (they stand at 2^11 of that or
    more, and fp16's last place is 2^-24), codes by up to 2^-17 a coordinate (half of z / 256's steps of 2^-24)."""
    k, v = T.vectors(ck), T.vectors(cv)
    heads = k.shape[0]
    vis = keep.any(0)
    ref, rl, pv, qk = T.attend(q, k, v, keep, group, SCALE)
    tol, tl = T.tolerance(pv, qk, 1, int(vis.sum()))
    s = torch.einsum("nhgd,htd->nhgt", q.double().unflatten(1, (heads, group)), k) * SCALE
    w = torch.softmax(s.masked_fill(~keep[:, None, None], -math.inf), -1)
    z = torch.where(keep[:, None], v.norm(dim=-1) / e, 0.0)             # [n_q, heads, tokens]: codes a row sees
    low = 2.0 ** -36 * (w * e).amax(-1) * z.sum(-1)[..., None] + 2.0 ** -17 * math.sqrt(128) * (w * e).sum(-1)
    lim = tol + low.flatten(1, 2) + 2.0 ** -24 * ref.norm(dim=-1)
    err = (out.double() - ref).norm(dim=-1)
    assert torch.isfinite(out).all()
    assert bool((err <= lim).all()), f"worst error / bound {float((err / lim).max()):.3g}"
    assert bool(((lse.double() - rl).abs() <= tl + 2.0 ** -22 * rl.abs()).all())


def _run(ck, cv, e, q, group, window=0, sinks=0):
    hq = _hq()
    n_q, n = q.shape[0], ck.tokens
    out, lse = torch.full(q.shape, float("nan"), device="cuda"), torch.full(q.shape[:2], float("nan"), device="cuda")
    hq.KVAttention(ck, cv, group, SCALE, window, sinks)(q, out, lse=lse)
    _check(out, lse, q, ck, cv, e, T.seen(n_q, n, window, sinks), group)
    for c in (ck, cv):
        assert hq.read_stats(c.stats)["status"] == 0


def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


# few heads: steps of one chunk; many: a warp to a chunk; above 16 rows (4 queries times the group) the other kernel
LAYOUTS = [(2, 1), (2, 4), (2, 8), (2, 40), (300, 1), (300, 4), (150, 8)]
RATIOS = [2.0 ** 4 * 1.1, 2.0 ** 10 * 1.3, 2.0 ** 14 * 1.7, 2.0 ** 18 * 0.9, 2.0 ** 24 * 1.1, 2.0 ** 60 * 1.3]


@pytest.mark.parametrize("lat,dither", [("E8", 1), ("E8", 0), ("Z", 1), ("D4", 0)])
@pytest.mark.parametrize("heads,group", LAYOUTS)
@pytest.mark.parametrize("ratio", RATIOS)
def test_large_values_hidden_by_position(lat, dither, heads, group, ratio):
    """The last tokens' values are `ratio` times the others'; the first queries come before them."""
    g = torch.Generator(device="cuda").manual_seed(1)
    n_q, a = 4, T.ALPHA[lat] * 1.07
    sizes, sizes_v = [64, 40, 1, 30, 3], [1.0, 1.0, 0.7, 1.0, ratio]
    kp = [(_rand(g, heads, n, 128), a) for n in sizes]
    vp = [(_rand(g, heads, n, 128) * m, a / m) for n, m in zip(sizes, sizes_v)]
    ck, _ = _cache(heads, kp, lat, 3, dither)
    cv, e = _cache(heads, vp, lat, 4, dither)
    q = _rand(g, n_q, heads * group, 128).to(torch.bfloat16)
    _run(ck, cv, e, q, group)


@pytest.mark.parametrize("heads,group", LAYOUTS)
@pytest.mark.parametrize("ratio", RATIOS)
def test_large_values_hidden_by_the_window(heads, group, ratio):
    """Large values at the far end of the window: the first queries see them, the last does not; between the sinks
    and the window lie larger ones still, which none sees."""
    g = torch.Generator(device="cuda").manual_seed(2)
    a = T.ALPHA["E8"]
    sizes, mags = [4, 200, 2, 50], [1.0, ratio * 3, ratio, 1.0]
    kp = [(_rand(g, heads, n, 128), a) for n in sizes]
    vp = [(_rand(g, heads, n, 128) * m, a / m) for n, m in zip(sizes, mags)]
    ck, _ = _cache(heads, kp, "E8", 5, 1)
    cv, e = _cache(heads, vp, "E8", 6, 1)
    q = _rand(g, 3, heads * group, 128).to(torch.bfloat16)
    _run(ck, cv, e, q, group, window=50, sinks=4)


@pytest.mark.parametrize("heads,group", [(1, 1), (150, 1), (1, 24), (150, 24)])
@pytest.mark.parametrize("ratio", RATIOS)
def test_large_values_without_weight_and_small_ones_with_it(heads, group, ratio):
    """Keys against the query under the large values: their product with the weight is small, or not, either way."""
    g = torch.Generator(device="cuda").manual_seed(3)
    a = T.ALPHA["E8"]
    one = _rand(g, 1, 1, 128)
    q = (one + 0.05 * _rand(g, 1, heads * group, 128)).to(torch.bfloat16)
    away = -30.0 * one / one.norm()
    kp = [(_rand(g, heads, 96, 128) * 0.3, a), (away + 0.1 * _rand(g, heads, 8, 128), a), (_rand(g, heads, 40, 128) * 0.3, a)]
    for mags in ((1.0, ratio, 1.0), (1.0, 1.0, ratio), (ratio, 1.0, ratio)):
        vp = [(_rand(g, heads, x.shape[1], 128) * m, a / m) for (x, _), m in zip(kp, mags)]
        ck, _ = _cache(heads, kp, "E8", 7, 1)
        cv, e = _cache(heads, vp, "E8", 8, 1)
        _run(ck, cv, e, q, group)


@pytest.mark.parametrize("heads,group", [(1, 1), (100, 1), (1, 24), (100, 24)])
@pytest.mark.parametrize("bits", [10, 16, 24, 26, 30])
def test_a_sink_that_takes_the_weight(heads, group, bits):
    """The first token has 2^bits times the weight of each other and a value near zero: the others' sum is the output."""
    g = torch.Generator(device="cuda").manual_seed(4)
    n, a = 700, T.ALPHA["E8"]
    one = _rand(g, 1, 1, 128)
    q = (one + 0.01 * _rand(g, 1, heads * group, 128)).to(torch.bfloat16)
    k = 0.02 * _rand(g, heads, n, 128)
    k[:, 0] = one[0, 0] / one.norm() * (bits * math.log(2) / (SCALE * float(one.norm())))
    v = 1.0 + 0.1 * _rand(g, heads, n, 128)
    v[:, 0] = 0
    # (codes without dither: the sink's value is zero)
    ck, _ = _cache(heads, [(k, 8 * a)], "E8", 9, 0, 3)
    cv, e = _cache(heads, [(v, 4 * a)], "E8", 10, 0, 3)
    _run(ck, cv, e, q, group)
