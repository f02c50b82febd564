"""Codes over the codec's whole range, the largest that no status flags among them: attention keeps them finite, and a row
that does not see their tokens does not know of them."""
import pytest
import torch

import kvtest as T

pytestmark = pytest.mark.gpu
ALPHA = 8192.0
# the largest coordinate, in codes: symbols stay below 2^22 (E8's last of a block: 4 m + 2 p + c, the others 2 m + c)
LARGEST = {("E8", 7): 8.2e6, ("E8", 5): 4.1e6, ("D4", 3): 4.1e6, ("D4", 0): 2.0e6, ("Z", 5): 2.0e6, ("A2", 1): 2.0e6}


def _hq():
    import lattice_entropy_coded_b200 as hq
    return hq


def _cache(x, lat, dither, seed):
    """Under the rotation of 1: codes are alpha x."""
    hq = _hq()
    c = hq.KVCache(x.shape[0], x.shape[1], hq.make_params(lat, 1.0, 13, seed, dither), bits_per_scalar=120.0, max_appends=2,
                   max_append_tokens=256, rotation=torch.eye(128, device="cuda"))
    c.append(x.to(torch.bfloat16), ALPHA)
    assert hq.read_stats(c.stats)["status"] == 0
    return c


@pytest.mark.parametrize("heads,group", [(1, 1), (2, 8), (300, 1)])     # steps of one chunk, many rows, a warp to a chunk
@pytest.mark.parametrize("lat,at", list(LARGEST))
@pytest.mark.parametrize("dither", [0, 1])
@pytest.mark.parametrize("where", ["k", "v", "kv"])
def test_the_largest_codes(heads, group, lat, at, dither, where):
    hq = _hq()
    g = torch.Generator(device="cuda").manual_seed(3)
    n, n_q = 150, 4
    big, clean = [], []
    for i, name in enumerate("kv"):
        x = torch.randn(heads, n, 128, generator=g, device="cuda")
        y = x.clone()
        if name in where:
            y[:, 100, 96 + at], y[:, 149, 32 + at] = LARGEST[lat, at] / ALPHA, -LARGEST[lat, at] / ALPHA
        clean.append(_cache(x, lat, dither, 3 + i))
        big.append(_cache(y, lat, dither, 3 + i))
    q = torch.randn(n_q, heads * group, 128, generator=g, device="cuda").to(torch.bfloat16)
    for window in (0, 40):
        out, want = (torch.empty(q.shape, device="cuda") for _ in "ab")
        hq.KVAttention(*big, group, window=window)(q, out)
        T.check(out, None, q, T.vectors(big[0]), T.vectors(big[1]), T.seen(n_q, n, window, 0), group, 128 ** -0.5, 1)
        if window:      # token 100 is outside every window, 149 later than all queries but the last
            hq.KVAttention(*clean, group, window=window)(q, want)
            assert torch.equal(out[:3], want[:3])
    for c in big:
        assert hq.read_stats(c.stats)["status"] == 0
