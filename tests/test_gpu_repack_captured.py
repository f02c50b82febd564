"""KVCache.repack inside a captured graph, its workspace the graph's own: replayed between other work, on its stream and
with the stream given."""
import pytest
import torch

import kvtest as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [None, "stream", "handle"])
def test_captured_with_other_allocations_and_replayed(given):
    import lattice_entropy_coded_b200 as hq
    a, _ = T.pair(2, [100, 1, 1, 200], "E8")
    ranges = [(0, 4), (90, 302)]
    dst = [hq.KVCache(2, 400, a.cache.params, bits_per_scalar=32.0, max_appends=8, max_append_tokens=64) for _ in range(3)]
    a.repack(dst[0], ranges)
    end = hq.read_stats(dst[0].stats)["stream_words"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            how = {None: None, "stream": side, "handle": side.cuda_stream}[given]
            a.repack(dst[1], ranges, cuda_stream=how)
            over = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")    # where the workspace may have been
            a.repack(dst[2], ranges, cuda_stream=how)
            over += 1
        for _ in range(3):
            for d in dst[1:]:
                d.words.fill_(-7), d.offsets.fill_(-1), d.stats.fill_(255)
            g.replay()
    side.synchronize()
    for d in dst[1:]:
        assert hq.read_stats(d.stats) == hq.read_stats(dst[0].stats) and d.tokens == 302
        assert torch.equal(d.words[:end], dst[0].words[:end]) and bool((d.words[end:] == -7).all())
        assert torch.equal(T.vectors(d), T.vectors(dst[0]))
    assert bool((over == 0).all())
