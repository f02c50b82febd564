"""hq_kv_attention and hq_kv_tree_attention against attention in 64 bits over what hq_kv_read
reconstructs; the tolerances are derived in kvtest.tolerance."""
import pytest
import torch

import kvtest as T

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def _hq():
    import lattice_entropy_coded_b200 as hq
    return hq


def _queries(n_q, heads, seed=1, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n_q, heads, 128, generator=g, device="cuda") * std).to(torch.bfloat16)


def _run(k, v, group, n_q=1, window=0, sinks=0, length=None, dtype=torch.float32, q=None, scale=SCALE, dither=1, held=None):
    hq = _hq()
    n = k.tokens if length is None else length
    q = _queries(n_q, k.heads * group) if q is None else q
    out = torch.full((n_q, k.heads * group, 128), float("nan"), dtype=dtype, device="cuda")
    lse = torch.full((n_q, k.heads * group), float("nan"), device="cuda")
    hq.KVAttention(k, v, group, scale, window, sinks)(q, out, length=n, lse=lse)
    keep = T.seen(n_q, n, window, sinks, held=held)
    T.check(out, lse, q, T.vectors(k, n), T.vectors(v, n), keep, group, scale, dither)
    for c in (k, v):
        assert hq.read_stats(c.stats)["status"] == 0
    return out, lse


def _tree(k, v, group, parents, window=0, sinks=0, length=None, dtype=torch.float32, dither=1, bad_hidden=True):
    """parents[i]: an earlier draft, or -1 (the last cached token)."""
    hq = _hq()
    n_q, n = len(parents), k.tokens if length is None else length
    mask = []
    for i, p in enumerate(parents):
        mask.append((mask[p] if p >= 0 else 0) | 1 << i)
    return _masked(k, v, group, mask, n_q, n, window, sinks, dtype, dither)


def _masked(k, v, group, mask, n_q, n, window=0, sinks=0, dtype=torch.float32, dither=1):
    hq = _hq()
    q = _queries(n_q, k.heads * group, 5)
    kd, vd = _queries(k.heads, n_q, 6), _queries(k.heads, n_q, 7)
    m = torch.tensor([x - (1 << 64) if x >> 63 else x for x in mask], device="cuda")
    out = torch.full((n_q, k.heads * group, 128), float("nan"), dtype=dtype, device="cuda")
    lse = torch.full((n_q, k.heads * group), float("nan"), device="cuda")
    hq.KVAttention(k, v, group, SCALE, window, sinks).tree(q, kd, vd, m, out, length=n, lse=lse)
    keep = T.seen(n_q, n, window, sinks, mask)
    kk, vv = (torch.cat((T.vectors(c, n), d.double()), 1) for c, d in ((k, kd), (v, vd)))
    T.check(out, lse, q, kk, vv, keep, group, SCALE, dither)
    return out, lse


@pytest.mark.parametrize("lat", ["E8", "D4", "A2", "Z"])
@pytest.mark.parametrize("dither", [0, 1])
@pytest.mark.parametrize("k,dk", [(0, 0), (1, 0), (2, 1), (6, 0), (9, 3)])
def test_every_stream_form(lat, dither, k, dk):
    """Remainders in windows, one by one and with a second parameter; chunks in the stage and in place (k = 9)."""
    a, b = T.pair(2, [33, 64, 1, 1, 40], lat, k, dither, dk)
    _run(a, b, 4, n_q=3, dither=dither)


def test_k_and_v_of_different_parameters_and_scales():
    a, b = T.pair(2, [64, 1, 31, 32], "E8", 0, 1, alphas=[1.0, 7.0, 0.2, 1.4], vk=3)
    _run(a, b, 2, n_q=2)


@pytest.mark.parametrize("length", [1, 2, 8, 9, 16, 17, 31, 32, 33, 127, 128, 129, 300])
def test_lengths(length):
    a, b = T.pair(1, [length], "E8")
    _run(a, b, 3)
    if length > 1:
        _run(a, b, 1, n_q=2)


@pytest.mark.parametrize("heads,group,n_q", [(1, 1, 1), (1, 16, 1), (1, 17, 1), (3, 7, 5), (8, 4, 8), (2, 64, 1), (1, 64, 64),
                                             (5, 1, 33), (16, 2, 1), (300, 1, 1)])
def test_head_layouts(heads, group, n_q):
    a, b = T.pair(heads, [70], "E8" if heads < 100 else "Z")
    _run(a, b, group, n_q=n_q, length=69)


@pytest.mark.parametrize("appends", [[256] * 16 + [3], [1] * 77, [40, 1, 1, 1, 500, 1, 7]])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (33, 4), (100, 40), (64, 1000000), (5000, 3)])
def test_windows_and_sinks(appends, window, sinks):
    a, b = T.pair(2, appends, "E8")
    _run(a, b, 2, n_q=min(3, a.tokens), window=window, sinks=sinks)


def test_long_cache():
    """Many splits: 20000 tokens, far scores among them."""
    a, b = T.pair(2, [4096] * 4 + [3616], "E8", 0)
    _run(a, b, 4)
    _run(a, b, 4, n_q=16)
    _run(a, b, 4, n_q=2, window=6000, sinks=5)


def test_part_of_a_cache():
    a, b = T.pair(2, [64, 64], "D4")
    for n in (1, 63, 64, 65, 100):
        _run(a, b, 2, length=n)


@pytest.mark.parametrize("std", [1e-20, 0.01, 30.0])
def test_query_sizes(std):
    a, b = T.pair(1, [200], "E8")
    _run(a, b, 4, q=_queries(1, 4, std=std))


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-6, 1.0])
def test_scales(scale):
    a, b = T.pair(1, [200], "E8", dither=0)
    _run(a, b, 4, scale=scale, dither=0)


def test_dense_rotation():
    hq = _hq()
    rot = [hq.hq_haar_rotation(5), hq.hq_haar_rotation(6)]
    torch.cuda.synchronize()
    a, b = T.pair(2, [100, 1, 30], "E8", 1, alpha=0.7, rotation=rot)
    _run(a, b, 4, n_q=3)
    a, b = T.pair(2, [100, 1, 30], "E8", 1, alpha=0.7, rotation=[None, rot[1]])
    _run(a, b, 4, n_q=3, window=50, sinks=2)
    _tree(a, b, 2, [-1, 0, 0, 2])


def test_bf16_output_and_strides():
    """A query and an output inside wider rows, head-major; what lies between them stays."""
    hq = _hq()
    a, b = T.pair(3, [90], "E8")
    n_q, group, heads = 4, 2, 6
    wide = _queries(heads, n_q * 3, 9).reshape(heads, n_q, 3 * 128)
    q = wide[:, :, 128:256].transpose(0, 1)
    for dtype in (torch.bfloat16, torch.float32):
        buf = torch.full((heads, n_q, 160), 7.0, dtype=dtype, device="cuda")
        out = buf[:, :, 16:144].transpose(0, 1)
        hq.KVAttention(a, b, group)(q, out)
        T.check(out, None, q, T.vectors(a), T.vectors(b), T.seen(n_q, 90, 0, 0), group, SCALE, 1)
        assert bool((buf[:, :, :16] == 7).all()) and bool((buf[:, :, 144:] == 7).all())


def test_one_query_broadcast_over_heads():
    """A head stride of zero: every head reads one query."""
    hq = _hq()
    a, b = T.pair(2, [50], "E8")
    q = _queries(1, 1).expand(1, 4, 128)
    out = torch.empty(1, 4, 128, device="cuda")
    hq.KVAttention(a, b, 2)(q, out)
    T.check(out, None, q, T.vectors(a), T.vectors(b), T.seen(1, 50, 0, 0), 2, SCALE, 1)


def test_rows_that_see_nothing():
    """Positions dropped by a repack: queries whose window covers only those give zeros, lse -infinity."""
    hq = _hq()
    a, b = T.pair(2, [256, 44], "E8")
    caches = []
    for c in (a, b):
        d = hq.KVCache(2, 400, c.cache.params, bits_per_scalar=16.0, max_appends=8, max_append_tokens=64)
        caches.append(c.repack(d, [(0, 4), (200, 300)]))
    held = lambda t: t < 4 or t >= 200  # noqa: E731
    ka, kb = caches
    assert torch.equal(T.vectors(ka)[:, 200:], T.vectors(a)[:, 200:])
    _run(ka, kb, 2, n_q=3, held=held)
    _run(ka, kb, 2, n_q=3, window=10, length=150, held=held)                # nothing at all
    out, lse = _run(ka, kb, 2, n_q=8, window=3, length=205, held=held)       # some rows empty, some not
    assert bool(torch.isinf(lse).any()) and not bool(torch.isinf(lse).all())
    _run(ka, kb, 2, n_q=3, window=10, sinks=2, length=150, held=held)


@pytest.mark.parametrize("parents", [[-1], [-1, 0], [-1, 0, 0, 1, 1, 2, -1, 6], list(range(-1, 63)), [-1] * 64,
                                     [-1] + [i // 2 for i in range(30)]])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2, 0), (20, 3)])
def test_trees(parents, window, sinks):
    a, b = T.pair(2, [64, 33], "E8")
    _tree(a, b, 3, parents, window, sinks)


def test_trees_at_other_lengths():
    a, b = T.pair(1, [300, 1, 1], "Z", 1, 0)
    for n in (0, 1, 33, 302):
        _tree(a, b, 1, [-1, 0, 1, 1, 3], length=n, dither=0)
    _tree(a, b, 1, [-1, 0, 1, 1, 3], window=3, sinks=2, dtype=torch.bfloat16, dither=0)


def test_tree_masks_as_given():
    """Masks that are no tree: rows without themselves, later drafts, bits past n_q; none of them breaks the rule."""
    a, b = T.pair(2, [40], "E8")
    for n in (0, 40):
        _masked(a, b, 2, [0, 0b1, (1 << 64) - 1, 0b0100], 4, n)
    _masked(a, b, 2, [0b11, 0b111, 0b110, 0b1000], 4, 40, window=2, sinks=1)


def test_invisible_drafts_may_hold_anything():
    hq = _hq()
    a, b = T.pair(2, [40], "E8")
    q, kd, vd = _queries(3, 4), _queries(2, 3, 2), _queries(2, 3, 3)
    m = torch.tensor([0b001, 0b011, 0b001], device="cuda")      # no row sees draft 2
    at = hq.KVAttention(a, b, 2)
    want = at.tree(q, kd, vd, m, torch.empty(3, 4, 128, device="cuda")).clone()
    kd[:, 2], vd[:, 2] = float("nan"), float("inf")
    assert torch.equal(at.tree(q, kd, vd, m, torch.empty(3, 4, 128, device="cuda")), want)


def test_a_query_of_nan_or_infinity_stays_in_its_row():
    hq = _hq()
    a, b = T.pair(2, [140], "E8")
    q = _queries(2, 4)
    at = hq.KVAttention(a, b, 2)
    want = at(q, torch.empty(2, 4, 128, device="cuda")).clone()
    q[0, 1, 5], q[1, 3, 0] = float("nan"), float("inf")
    got = at(q, torch.empty(2, 4, 128, device="cuda"))
    rows = torch.ones(2, 4, dtype=torch.bool, device="cuda")
    rows[0, 1] = rows[1, 3] = False
    assert torch.equal(got[rows], want[rows]) and not torch.isfinite(got[~rows]).any()


def test_corrupt_chunk_counts_as_zero_vectors():
    hq = _hq()
    a, b = T.pair(2, [128], "E8")
    for c, other in ((a, b), (b, a)):
        keep_off = c.offsets.clone()
        c.offsets[2], c.offsets[3] = keep_off[3], keep_off[2]
        q = _queries(1, 4)
        out = torch.empty(1, 4, 128, device="cuda")
        hq.KVAttention(a, b, 2)(q, out)
        assert hq.read_stats(c.stats)["status"] == hq.HQ_ST_CORRUPT
        assert hq.read_stats(other.stats)["status"] == 0
        T.check(out, None, q, T.vectors(a), T.vectors(b), T.seen(1, 128, 0, 0), 2, SCALE, 1)
        c.offsets.copy_(keep_off)
        c.stats.zero_()


def test_a_bit_flipped_in_the_unary_plane():
    hq = _hq()
    a, b = T.pair(1, [64], "E8")
    end = int(b.offsets[1])
    b.words[end - 2] ^= 1 << 7
    q = _queries(1, 2)
    out = torch.empty(1, 2, 128, device="cuda")
    hq.KVAttention(a, b, 2)(q, out)
    assert hq.read_stats(b.stats)["status"] == hq.HQ_ST_CORRUPT
    T.check(out, None, q, T.vectors(a), T.vectors(b), T.seen(1, 64, 0, 0), 2, SCALE, 1)


def test_v_appended_otherwise_than_k_is_reported():
    """Equal counters, other ranges: V's tokens count as zeros and V is marked."""
    hq = _hq()
    a, _ = T.pair(1, [33, 64], "E8")
    _, b = T.pair(1, [64, 33], "E8")
    assert (a.cache.chunks, a.cache.appends) == (b.cache.chunks, b.cache.appends)
    out = torch.empty(1, 2, 128, device="cuda")
    hq.KVAttention(a, b, 2)(_queries(1, 2), out)
    assert hq.read_stats(b.stats)["status"] == hq.HQ_ST_CORRUPT and bool(torch.isfinite(out).all())


def test_same_bits_every_time_and_across_splits_of_the_batch():
    hq = _hq()
    a, b = T.pair(4, [2048, 77], "E8")
    q = _queries(2, 16)
    at = hq.KVAttention(a, b, 4)
    first = at(q, torch.empty(2, 16, 128, device="cuda")).clone()
    for _ in range(3):
        assert torch.equal(at(q, torch.empty(2, 16, 128, device="cuda")), first)


def test_captured_replayed_and_on_another_stream():
    """Two graphs that share one workspace, replayed one after the other, on a stream of their own."""
    hq = _hq()
    a, b = T.pair(2, [256, 9], "E8")
    at = hq.KVAttention(a, b, 2)
    q1, q2 = _queries(1, 4, 1), _queries(3, 4, 2)
    o1, o2 = torch.empty(1, 4, 128, device="cuda"), torch.empty(3, 4, 128, device="cuda")
    want1, want2 = at(q1, torch.empty_like(o1)).clone(), at(q2, torch.empty_like(o2)).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for q, o in ((q1, o1), (q2, o2)):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                at(q, o)
            graphs.append(g)
        for _ in range(2):
            o1.fill_(float("nan")), o2.fill_(float("nan"))
            for g in graphs:
                g.replay()
    side.synchronize()
    assert torch.equal(o1, want1) and torch.equal(o2, want2)
    o1.fill_(float("nan"))
    torch.cuda.synchronize()
    at(q1, o1, cuda_stream=side)
    side.synchronize()
    assert torch.equal(o1, want1)


def test_two_calls_at_once_with_a_workspace_each():
    hq = _hq()
    a, b = T.pair(2, [256], "E8")
    q = [_queries(2, 4, i) for i in range(2)]
    want = [hq.KVAttention(a, b, 2)(x, torch.empty(2, 4, 128, device="cuda")).clone() for x in q]
    ats = [hq.KVAttention(a, b, 2) for _ in q]
    outs = [torch.empty(2, 4, 128, device="cuda") for _ in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(5):
        for at, x, o, s in zip(ats, q, outs, streams):
            at(x, o, cuda_stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_lse_merges_two_halves():
    """Two disjoint windows of one cache joined by their lse are the whole."""
    hq = _hq()
    a, b = T.pair(1, [64, 64], "E8", dither=0)
    q = _queries(1, 2)
    at = hq.KVAttention(a, b, 2)
    o, l = torch.empty(1, 2, 128, device="cuda"), torch.empty(1, 2, device="cuda")
    at(q, o, lse=l)
    lo, ll = torch.empty_like(o), torch.empty_like(l)
    at(q, lo, length=64, lse=ll)
    late = hq.KVAttention(a, b, 2, window=64)
    ho, hl = torch.empty_like(o), torch.empty_like(l)
    late(q, ho, lse=hl)
    m = torch.logaddexp(ll, hl)
    got = lo * torch.exp(ll - m)[..., None] + ho * torch.exp(hl - m)[..., None]
    # each of the three is within 2^-11 and a little of its own sum of p |v|
    assert float((got - o).norm()) <= 3 * (2.0 ** -11 + 2.0 ** -15) * float(T.attend(
        q, T.vectors(a), T.vectors(b), T.seen(1, 128, 0, 0), 2, SCALE)[2].norm())
    assert float((m - l).abs().max()) < 1e-4


@pytest.mark.parametrize("k", [0, 1])
def test_dither_of_many_blocks(k):
    """A window of one token returns that token's value: half a million E8 blocks, of which some hundred lie so near
    a border that the fast dither leaves them to the exact one.  A wrong lattice point would move a vector by an
    eighth of its length and more; fp16 codes by 2^-11."""
    hq = _hq()
    heads, n = 4096, 8
    a, b = T.pair(heads, [n], "E8", k, spare=0)
    at = hq.KVAttention(a, b, 1, window=1)
    v = T.vectors(b)
    q = _queries(1, heads)
    for t in range(n):
        out = at(q, torch.empty(1, heads, 128, device="cuda"), length=t + 1)
        err = (out[0].double() - v[:, t]).norm(dim=-1)
        assert bool((err <= 2.0 ** -10 * v[:, t].norm(dim=-1)).all())


@pytest.mark.parametrize("ones", [127, 128, 129, 300])
def test_more_appends_than_the_table_sample(ones):
    """The append table is searched through a sample of 128 appends; a token an append, and longer ones between."""
    a, b = T.pair(2, [40] + [1] * ones + [33, 1, 70], "E8")
    _run(a, b, 2, n_q=2)
    _run(a, b, 16, n_q=2)                                   # many rows
    _run(a, b, 2, n_q=3, window=90, sinks=41)
    _run(a, b, 2, length=40 + ones // 2, window=20, sinks=3)


def test_scales_far_apart_among_many_rows():
    """Appends whose alphas differ by 2^12: the rarest scale must not swamp the others."""
    a, b = T.pair(1, [32, 32, 40, 1, 1], "E8", 0, 0, alphas=[1.0, 1.0, 4.0, 0.5, 2.0])
    _run(a, b, 3, dither=0)
    _run(a, b, 32, n_q=2, dither=0)


def test_dense_rotation_of_many_rows():
    hq = _hq()
    rot = [hq.hq_haar_rotation(5), hq.hq_haar_rotation(6)]
    torch.cuda.synchronize()
    a, b = T.pair(2, [100, 1, 30], "E8", 1, alpha=0.7, rotation=rot)
    _run(a, b, 12, n_q=12)
    _tree(a, b, 8, [-1, 0, 0, 2, 3, 3, 3])


def test_many_rows_bf16_strides_and_bad_rows():
    """attention of 130 rows a head (two blocks, the second of two rows): NaN and infinity stay in their rows, a
    corrupt chunk counts as zeros, what lies between the output's rows stays."""
    hq = _hq()
    a, b = T.pair(2, [256, 20], "D4")
    q = _queries(26, 10)
    buf = torch.full((26, 10, 136), 7.0, device="cuda")
    out = buf[:, :, :128]
    at = hq.KVAttention(a, b, 5)
    at(q, out)
    T.check(out, None, q, T.vectors(a), T.vectors(b), T.seen(26, 276, 0, 0), 5, SCALE, 1)
    assert bool((buf[:, :, 128:] == 7).all())
    want = out.clone()
    q[3, 1, 5], q[25, 9, 0] = float("nan"), float("inf")
    at(q, out)
    rows = torch.ones(26, 10, dtype=torch.bool, device="cuda")
    rows[3, 1] = rows[25, 9] = False
    assert torch.equal(out[rows], want[rows]) and not torch.isfinite(out[~rows]).any()
    q[3, 1, 5], q[25, 9, 0] = 0, 0
    keep = b.offsets.clone()
    b.offsets[2], b.offsets[3] = keep[3], keep[2]
    at(q, out)
    assert hq.read_stats(b.stats)["status"] == hq.HQ_ST_CORRUPT and hq.read_stats(a.stats)["status"] == 0
    T.check(out, None, q, T.vectors(a), T.vectors(b), T.seen(26, 276, 0, 0), 5, SCALE, 1)


def test_rows_of_many_heads_and_blocks():
    """More rows than a CTA takes (64 queries x 9 heads a KV head: three blocks of rows)."""
    a, b = T.pair(2, [300], "Z", 1)
    _run(a, b, 9, n_q=64)
    _run(a, b, 9, n_q=64, window=40, sinks=2, length=290)


@pytest.mark.parametrize("lat", ["E8", "D4", "A2", "Z"])
@pytest.mark.parametrize("dither", [0, 1])
@pytest.mark.parametrize("k,dk", [(0, 0), (1, 0), (2, 1), (9, 3)])
def test_every_stream_form_of_many_rows(lat, dither, k, dk):
    a, b = T.pair(2, [33, 64, 1, 1, 40], lat, k, dither, dk)
    _run(a, b, 6, n_q=5, dither=dither)


def test_first_positions_dropped():
    """A cache that starts at position 37: sinks and windows that reach before it see nothing there."""
    hq = _hq()
    a, b = T.pair(2, [256, 44], "E8")
    pair = []
    for c in (a, b):
        d = hq.KVCache(2, 400, c.cache.params, bits_per_scalar=32.0, max_appends=8, max_append_tokens=64)
        pair.append(c.repack(d, [(37, 120), (125, 300)], cuda_stream=torch.cuda.current_stream()))
    held = lambda t: 37 <= t < 120 or t >= 125  # noqa: E731
    for group, n_q in ((2, 3), (10, 3)):
        for window, sinks, length in ((0, 0, 300), (50, 40, 300), (50, 4, 140), (20, 10, 37), (20, 10, 30), (400, 4, 300)):
            _run(*pair, group, n_q=n_q, window=window, sinks=sinks, length=length, held=held)


def test_repack_on_a_stream_given_by_its_handle():
    hq = _hq()
    a, b = T.pair(1, [64], "E8")
    side = torch.cuda.Stream()
    d = hq.KVCache(1, 100, a.cache.params, bits_per_scalar=32.0, max_appends=8, max_append_tokens=64)
    torch.cuda.synchronize()
    a.repack(d, cuda_stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(T.vectors(d), T.vectors(a))
