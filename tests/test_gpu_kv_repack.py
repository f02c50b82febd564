"""hq_kv_repack against the oracle: a repacked range is bit for bit the stream that one append of those
tokens at their positions writes, and what it leaves out is left out."""
import numpy as np
import pytest
import torch

import kvtest as T
import oracle as O
import synth
from hqtest import assert_same_words

pytestmark = pytest.mark.gpu
A = {"E8": 1.4, "D4": 0.9, "A2": 0.6, "Z": 0.8}


def _hq():
    import lattice_entropy_coded_b200 as hq
    return hq


def _source(heads, appends, lat, k=0, dither=1, dk=0, alpha=None, seed=4, bits=32.0, rotation=None):
    hq = _hq()
    total = sum(appends)
    x, _ = synth.kv(heads, total, seed=seed)
    alpha = A[lat] * 2.0 ** k if alpha is None else alpha
    alphas = alpha if isinstance(alpha, list) else [alpha] * len(appends)
    c = hq.KVCache(heads, total, hq.make_params(lat, 1.0, k, seed, dither, dk_last=dk), bits_per_scalar=bits,
                   max_appends=len(appends) + 1, max_append_tokens=max(appends), rotation=rotation)
    t = 0
    for n, a in zip(appends, alphas):
        c.append(x[:, t:t + n].contiguous().cuda(), a)
        t += n
    assert hq.read_stats(c.stats)["status"] == 0
    return c, x, alphas


def _dest(src, ranges, bits=32.0, appends=8):
    hq = _hq()
    n = sum(b - a for a, b in ranges)
    d = hq.KVCache(src.heads, n + 64, src.cache.params, bits_per_scalar=bits, max_appends=len(ranges) + appends,
                   max_append_tokens=64)
    d.rotation = src.rotation
    d.words.fill_(-7)
    d.offsets.fill_(-1)
    d.stats.fill_(255)
    return d


def _oracle(x, ranges, lat, alpha, k, seed, dither, dk=0, rot=None):
    words, offs, base, bits = [], [], 0, 0
    for (a, b), al in zip(ranges, alpha):
        s, off, pb = O.kv_append(x[:, a:b].contiguous(), a, O.LATTICES[lat], al, k, seed, dither, base_word=base,
                                 dk_last=dk, rot=rot)
        words.append(s)
        offs.append(off[:-1])
        base = int(off[-1])
        bits += pb
    return np.concatenate(words), np.concatenate(offs + [np.array([base], np.uint64)]), bits


def _check(src, dst, x, ranges, lat, alphas, k=0, dither=1, dk=0, seed=4, rot=None):
    hq = _hq()
    torch.cuda.synchronize()
    w, off, bits = _oracle(x, ranges, lat, alphas, k, seed, dither, dk, rot)
    end, n = int(off[-1]), len(off) - 1
    assert_same_words(dst.words[:end].cpu().numpy().view(np.uint32), dst.offsets[:n + 1].cpu().numpy().view(np.uint64),
                      w, off)
    assert bool((dst.words[end:] == -7).all()) and bool((dst.offsets[n + 1:] == -1).all())
    st, ss = hq.read_stats(dst.stats), hq.read_stats(src.stats)
    assert st == dict(status=0, payload_bits=bits, stream_words=end, max_symbol=ss["max_symbol"],
                      max_abs_code=ss["max_abs_code"], int8_overflow_count=0)
    assert dst.tokens == ranges[-1][1] and dst.cache.chunks == n and dst.cache.appends == len(ranges)
    # the values that were there, and nothing where nothing is
    got = T.vectors(dst, fill=5.0)
    want = torch.full_like(got, 5.0)
    full = T.vectors(src)
    for a, b in ranges:
        want[:, a:b] = full[:, a:b]
    assert torch.equal(got, want)


@pytest.mark.parametrize("lat", ["E8", "D4", "A2", "Z"])
@pytest.mark.parametrize("k,dk", [(0, 0), (1, 0), (1, 1), (2, 1), (5, 0), (11, 0)])
@pytest.mark.parametrize("dither", [0, 1])
def test_every_stream_form(lat, k, dk, dither):
    src, x, al = _source(2, [40, 1, 1, 64, 3, 30], lat, k, dither, dk)
    ranges = [(0, 5), (7, 104), (110, 139)]
    dst = src.repack(_dest(src, ranges), ranges)
    _check(src, dst, x, ranges, lat, al, k, dither, dk)


@pytest.mark.parametrize("appends,ranges", [
    ([1], [(0, 1)]),
    ([1] * 100, [(0, 100)]),
    ([1] * 100, [(3, 4), (4, 5), (99, 100)]),
    ([100], [(0, 100)]),
    ([100], [(31, 33), (33, 64), (65, 96)]),
    ([4, 3, 2, 1, 5] * 7, [(0, 105)]),
    ([256, 256, 17], [(0, 4), (300, 529)]),
    ([700], [(i * 21, i * 21 + 20) for i in range(32)]),
    ([1] * 300 + [64], [(0, 1), (7, 331), (340, 364)]),
    ([17] * 20, [(0, 340)]),
    ([96, 31, 64], [(0, 96), (96, 191)]),
])
@pytest.mark.parametrize("heads", [1, 3])
def test_cuts(appends, ranges, heads):
    src, x, al = _source(heads, appends, "E8")
    dst = src.repack(_dest(src, ranges), ranges)
    _check(src, dst, x, ranges, "E8", al * len(ranges))


def test_many_chunks():
    """More chunks than the second launch has warps: each CTA walks several."""
    src, x, al = _source(8, [4096] * 10 + [1] * 3, "E8")
    ranges = [(1, 40963)]
    dst = src.repack(_dest(src, ranges), ranges)
    _check(src, dst, x, ranges, "E8", al)


def test_large_symbols():
    """Unary runs of many words to a tile, in chunks of one token and of many."""
    src, x, al = _source(2, [1, 1, 40, 1], "E8", alpha=60.0, bits=900.0)
    ranges = [(0, 43)]
    dst = src.repack(_dest(src, ranges, bits=900.0), ranges)
    _check(src, dst, x, ranges, "E8", al)


def test_scales_by_range():
    """One alpha to a range; a range over two is marked, and what lies under the second reads as zero symbols."""
    hq = _hq()
    src, x, _ = _source(1, [32, 32, 32], "E8", alpha=[1.0, 1.0, 2.0])
    ranges = [(0, 64), (64, 96)]
    dst = src.repack(_dest(src, ranges), ranges)
    _check(src, dst, x, ranges, "E8", [1.0, 2.0])
    bad = src.repack(_dest(src, [(0, 96)]), [(0, 96)])
    assert hq.read_stats(bad.stats)["status"] == hq.HQ_ST_CORRUPT
    assert torch.equal(T.vectors(bad)[:, :64], T.vectors(src)[:, :64])


def test_dense_rotation():
    hq = _hq()
    Q = hq.hq_haar_rotation(9)
    torch.cuda.synchronize()
    src, x, al = _source(2, [50, 1], "E8", 1, alpha=0.7, rotation=Q)
    dst = src.repack(_dest(src, [(2, 51)]), [(2, 51)])
    _check(src, dst, x, [(2, 51)], "E8", al, 1, rot=Q.cpu().numpy())


def test_appends_go_on_after_a_repack_and_a_second_repack():
    """Fork, append to both, merge again: the streams are the oracle's throughout."""
    hq = _hq()
    src, x, al = _source(2, [33] + [1] * 9, "E8")
    more, _ = synth.kv(2, 20, seed=77)
    dst = src.repack(_dest(src, [(0, 42)], appends=32))
    for t in range(20):
        dst.append(more[:, t:t + 1].contiguous().cuda(), al[0])
    both = torch.cat((x, more), 1)
    again = dst.repack(_dest(dst, [(0, 62)]), [(0, 4), (30, 62)])
    _check(dst, again, both, [(0, 4), (30, 62)], "E8", al)
    # dropped positions cannot come back
    bad = again.repack(_dest(again, [(0, 62)]), [(0, 62)])
    assert hq.read_stats(bad.stats)["status"] == hq.HQ_ST_CORRUPT


def test_empty():
    hq = _hq()
    src, _, _ = _source(2, [10], "E8")
    dst = src.repack(_dest(src, [(0, 10)]), [(0, 10)])
    hq.hq_kv_repack(src.cache, dst.cache, [], None)
    torch.cuda.synchronize()
    assert (dst.tokens, dst.cache.chunks, dst.cache.appends) == (0, 0, 0)
    assert hq.read_stats(dst.stats)["stream_words"] == 0 and dst.tail.tolist() == [0, 0] and int(dst.offsets[0]) == 0
    x, _ = synth.kv(2, 7, seed=1)
    dst.append(x.cuda(), 1.0)
    w, off, _ = _oracle(x, [(0, 7)], "E8", [1.0], 0, 4, 1)
    assert_same_words(dst.words[:int(off[-1])].cpu().numpy().view(np.uint32),
                      dst.offsets[:len(off)].cpu().numpy().view(np.uint64), w, off)


def test_capacity_is_reported_and_nothing_is_written_past_it():
    hq = _hq()
    src, x, al = _source(2, [64], "E8")
    dst = _dest(src, [(0, 64)])
    need = src.repack(_dest(src, [(0, 64)]))
    words = hq.read_stats(need.stats)["stream_words"]
    dst.cache.cap_words = words - 5
    src.repack(dst)
    st = hq.read_stats(dst.stats)
    assert st["status"] == hq.HQ_ST_CAPACITY and st["stream_words"] == words
    assert torch.equal(dst.words[:words - 5], need.words[:words - 5]) and bool((dst.words[words - 5:] == -7).all())


def test_corrupt_source_chunk():
    """Its tiles become zero symbols; the others are as they were."""
    hq = _hq()
    src, x, al = _source(1, [64, 1, 1], "E8")
    good = T.vectors(src)
    src.offsets[1] = src.offsets[2] + 5
    dst = src.repack(_dest(src, [(0, 66)]))
    assert hq.read_stats(dst.stats)["status"] == hq.HQ_ST_CORRUPT
    assert torch.equal(T.vectors(dst)[:, 64 + 1:], good[:, 65:])


def test_captured_and_replayed():
    hq = _hq()
    src, x, al = _source(2, [64, 1], "E8")
    dst = _dest(src, [(0, 65)])
    ws = torch.empty(hq.hq_kv_repack_workspace_bytes(2, [(0, 65)]), dtype=torch.uint8, device="cuda")
    src.repack(_dest(src, [(0, 65)]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hq.hq_kv_repack(src.cache, dst.cache, [(0, 65)], ws)
    for _ in range(2):
        dst.words.fill_(-7)
        g.replay()
        _check(src, dst, x, [(0, 65)], "E8", al)


def test_on_another_stream():
    src, x, al = _source(2, [300], "E8")
    dst = _dest(src, [(0, 300)])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    src.repack(dst, cuda_stream=side)
    side.synchronize()
    _check(src, dst, x, [(0, 300)], "E8", al)
