"""What hq_kv_repack writes for tokens that it cannot copy: zero symbols, bit for bit, beside sound tokens in the same new
chunk.  The expected stream is put together here, tile by tile, from the source's bits."""
import numpy as np
import pytest
import torch

import synth
from hqtest import assert_same_words

pytestmark = pytest.mark.gpu
N = {"Z": 1, "A2": 2, "D4": 4, "E8": 8}
ALPHA = {"E8": 1.4, "D4": 0.9, "A2": 0.6, "Z": 0.8}
HEADS = 2


def _hq():
    import lattice_entropy_coded_b200 as hq
    return hq


def _bits(words):
    return np.unpackbits(words.view(np.uint8), bitorder="little")


def _words(bits):
    return np.packbits(np.concatenate((bits, np.zeros(-len(bits) % 32, np.uint8))), bitorder="little").view(np.uint32)


def _tiles(words, n, coset, rem):
    """(coset bits, remainder bits, unary bits) of each tile of a chunk."""
    b = _bits(words)
    nc, nr = (coset * n + 31) // 32 * 32, (rem * n + 31) // 32 * 32
    ends = np.flatnonzero(b[nc + nr:])[127::128] + 1
    assert len(ends) == n
    starts = np.concatenate(([0], ends[:-1]))
    return [(b[coset * i:coset * (i + 1)], b[nc + rem * i:nc + rem * (i + 1)], b[nc + nr + s:nc + nr + e])
            for i, (s, e) in enumerate(zip(starts, ends))]


def _run(lat, k, dk, appends, ranges, bad_chunks=(), alphas=None):
    """bad_chunks: (append, head, chunk of it); a terminator of each is cleared."""
    hq = _hq()
    total, base = sum(appends), ALPHA[lat] * 2.0 ** k
    params = hq.make_params(lat, 1.0, k, 4, 1, dk_last=dk)
    src = hq.KVCache(HEADS, total, params, bits_per_scalar=32.0, max_appends=len(appends) + 1, max_append_tokens=max(appends))
    x, t = synth.kv(HEADS, total, seed=6)[0], 0
    alphas = alphas or [1.0] * len(appends)
    for n, a in zip(appends, alphas):
        src.append(x[:, t:t + n].contiguous().cuda(), base * a)
        t += n
    torch.cuda.synchronize()
    words, off = src.words.cpu().numpy().view(np.uint32), src.offsets.cpu().numpy()
    coset, n = 16 if lat == "E8" else 0, N[lat]
    rem = 128 // n * ((n - 1) * k + max(k - dk, 0)) if n > 1 else 128 * k
    tile_of, chunk, pos = {}, 0, 0
    for a, (count, alpha) in enumerate(zip(appends, alphas)):
        for h in range(HEADS):
            for j in range((count + 31) // 32):
                m = min(32, count - 32 * j)
                bad = (a, h, j) in bad_chunks
                for i, tile in enumerate(_tiles(words[off[chunk]:off[chunk + 1]], m, coset, rem)):
                    tile_of[h, pos + 32 * j + i] = (None if bad else tile, alpha)
                if bad:
                    w = int(off[chunk + 1]) - 1
                    last = int(words[w])
                    src.words[w] = int(np.uint32(last & (last - 1)).view(np.int32))
                chunk += 1
        pos += count
    zero = (np.zeros(coset, np.uint8), np.zeros(rem, np.uint8), np.ones(128, np.uint8))
    out, offs, bits, lost = [], [0], 0, 0
    for lo, hi in ranges:
        for h in range(HEADS):
            for t0 in range(lo, hi, 32):
                tiles = []
                for t in range(t0, min(t0 + 32, hi)):
                    tile, alpha = tile_of.get((h, t), (None, None))
                    ok = tile is not None and alpha == tile_of[h, lo][1]
                    lost += not ok
                    tiles.append(tile if ok else zero)
                planes = [np.concatenate([x[p] for x in tiles]) for p in range(3)]
                bits += sum(map(len, planes))
                out += [_words(p) for p in planes]
                offs.append(offs[-1] + sum(len(w) for w in out[-3:]))
    dst = hq.KVCache(HEADS, sum(b - a for a, b in ranges) + 64, params, bits_per_scalar=32.0, max_appends=len(ranges) + 1,
                     max_append_tokens=64)
    dst.words.fill_(-7)
    src.repack(dst, ranges)
    st = hq.read_stats(dst.stats)
    assert lost and st["status"] == hq.HQ_ST_CORRUPT and st["payload_bits"] == bits and st["stream_words"] == offs[-1]
    assert_same_words(dst.words[:offs[-1]].cpu().numpy().view(np.uint32), dst.offsets[:len(offs)].cpu().numpy().view(np.uint64),
                      np.concatenate(out), np.array(offs, np.uint64))
    assert bool((dst.words[offs[-1]:] == -7).all())


FORMS = [("E8", 0, 0), ("E8", 1, 1), ("E8", 2, 0), ("D4", 1, 0), ("A2", 1, 1), ("Z", 0, 0), ("Z", 3, 0), ("D4", 5, 2)]


@pytest.mark.parametrize("lat,k,dk", FORMS)
@pytest.mark.parametrize("every", [2, 3, 5, 16])
def test_bad_one_token_chunks_among_good_ones(lat, k, dk, every):
    """Runs of one tile and of several, more and fewer than a plane copies run by run; the heads differ."""
    bad = [(a, h, 0) for a in range(70) for h in range(HEADS) if a % every == h]
    _run(lat, k, dk, [1] * 70, [(0, 70)], bad)


@pytest.mark.parametrize("lat,k,dk", FORMS)
@pytest.mark.parametrize("bad", [[(1, 0, 0)], [(1, 0, 0), (1, 1, 2)], [(0, 0, 0), (2, 1, 0)], [(1, 0, 0), (1, 0, 1), (1, 0, 2)]])
@pytest.mark.parametrize("ranges", [[(0, 110)], [(3, 40), (41, 109)], [(5, 37), (37, 101)]])
def test_bad_chunks_across_the_new_ones(lat, k, dk, bad, ranges):
    """Chunks of 32 tokens that fall into two new ones each, or make one whole."""
    if any(a in (0, 2) for a, _, _ in bad) and ranges[0][0] == 5:
        ranges = [(0, 5), (5, 110)]
    _run(lat, k, dk, [5, 96, 9], ranges, bad)


@pytest.mark.parametrize("lat,k,dk", FORMS)
def test_tokens_of_another_scale(lat, k, dk):
    _run(lat, k, dk, [20, 1, 1, 30], [(0, 52)], alphas=[1.0, 2.0, 1.0, 1.0])
    _run(lat, k, dk, [1, 1, 1, 64], [(0, 67)], alphas=[1.0, 0.5, 1.0, 1.0], bad_chunks=[(3, 1, 1)])
