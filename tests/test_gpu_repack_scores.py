"""hq_kv_scores and hq_kv_read over a repacked cache: the tokens it holds as before, dropped positions untouched."""
import pytest
import torch

import kvtest as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("ranges", [[(0, 4), (200, 300)], [(37, 90), (91, 92), (250, 300)], [(299, 300)], [(10, 20)]])
def test_scores_of_what_is_held(ranges, rotated):
    import lattice_entropy_coded_b200 as hq
    rot = [hq.hq_haar_rotation(5), None] if rotated else None
    torch.cuda.synchronize()
    a, _ = T.pair(2, [256, 44], "E8", rotation=rot)
    d = hq.KVCache(2, 400, a.cache.params, bits_per_scalar=32.0, max_appends=8, max_append_tokens=64)
    a.repack(d, ranges)
    n = ranges[-1][1]
    q = torch.randn(8, 128, device="cuda").to(torch.bfloat16)
    whole = a.scores(q, 4, torch.empty(8, 300, device="cuda"))
    for length in (n, n - 1, (ranges[0][0] + ranges[0][1]) // 2):
        got = d.scores(q, 4, torch.full((8, 300), 9.0, device="cuda")[:, :max(length, 1)], length)
        vec = d.read(torch.full((2, max(length, 1), 128), 9.0, device="cuda"), length)
        full = a.read(torch.empty(2, 300, 128, device="cuda"))
        held = torch.zeros(300, dtype=torch.bool, device="cuda")
        for lo, hi in ranges:
            held[lo:hi] = True
        held = held[:max(length, 1)] & (torch.arange(max(length, 1), device="cuda") < length)
        assert torch.equal(got[:, held], whole[:, :held.numel()][:, held]) and bool((got[:, ~held] == 9).all())
        assert torch.equal(vec[:, held], full[:, :held.numel()][:, held]) and bool((vec[:, ~held] == 9).all())
    assert hq.read_stats(d.stats)["status"] == 0
