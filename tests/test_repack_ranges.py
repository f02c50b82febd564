"""The ranges of a repack as a program may give them: any iterable of pairs, and nothing else."""
import pytest
import torch

PAIRS = [(0, 4), (10, 50)]
FORMS = [lambda: iter(PAIRS), lambda: (p for p in PAIRS), lambda: zip((0, 10), (4, 50)), lambda: tuple(PAIRS),
         lambda: [list(p) for p in PAIRS], lambda: torch.tensor(PAIRS), lambda: map(tuple, PAIRS)]


@pytest.mark.parametrize("bad", [[(0, 4, 10)], [(0,)], [(0, 4), (10, 50, 60, 70)], [()]])
def test_anything_but_pairs_is_an_error(bad):
    import lattice_entropy_coded_b200 as hq
    with pytest.raises(ValueError):
        hq.hq_kv_repack_workspace_bytes(2, bad)


class _Cache:
    """KVCache.repack over a binding that records its calls (no GPU)."""

    def __init__(self, hq):
        self.heads, self.tokens, self.rotation, self.cache = 2, 60, None, None
        self.words = torch.empty(1)
        self.repack = hq.KVCache.repack.__get__(self)


@pytest.mark.parametrize("form", FORMS)
def test_every_iterable_reaches_the_library_whole(form, monkeypatch):
    import contextlib
    import lattice_entropy_coded_b200 as hq
    got = []
    monkeypatch.setattr(hq, "hq_kv_repack", lambda s, d, r, ws, st=None: got.append((list(hq._ranges(r)[0]), ws.numel())))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    src = _Cache(hq)
    src.repack(_Cache(hq), form())
    assert got == [([0, 4, 10, 50], hq.hq_kv_repack_workspace_bytes(2, PAIRS))]


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
def test_every_iterable_copies_the_same(form):
    import lattice_entropy_coded_b200 as hq
    import synth
    src = hq.KVCache(2, 60, hq.make_params("E8", 1.0, 0, 3, 1), bits_per_scalar=16.0, max_appends=4, max_append_tokens=64)
    src.append(synth.kv(2, 60, seed=2)[0].cuda(), 1.4)
    a, b = (hq.KVCache(2, 100, src.cache.params, bits_per_scalar=16.0, max_appends=4, max_append_tokens=64) for _ in "ab")
    src.repack(a, PAIRS)
    src.repack(b, form())
    end = hq.read_stats(a.stats)["stream_words"]
    assert hq.read_stats(b.stats)["stream_words"] == end and b.tokens == a.tokens == 50
    assert torch.equal(a.words[:end], b.words[:end])
