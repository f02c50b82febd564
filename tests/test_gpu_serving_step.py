"""The KV operators as a decode loop uses them: norm and rotation, append, attention, a tree of drafts whose
accepted tokens are appended, eviction and merge, all through one pair of caches."""
import pytest
import torch

import kvtest as T

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
HEADS, GROUP = 2, 3


def _hq():
    import lattice_entropy_coded_b200 as hq
    return hq


def _project(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, HEADS * GROUP + 2 * HEADS, 128, generator=g, device="cuda").to(torch.bfloat16)


def test_decode_with_drafts_eviction_and_merge():
    hq = _hq()
    params = [hq.make_params("E8", 1.0, 1, 5 + i, 1) for i in range(2)]
    make = lambda: [hq.KVCache(HEADS, 400, p, bits_per_scalar=8.0, max_appends=128, max_append_tokens=128)  # noqa: E731
                    for p in params]
    caches, alpha, window, sinks = make(), (3.3, 3.3), 100, 4
    freq = 10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
    spec = hq.rope_spec()
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    gone = set()

    def layer(x, pos0, positions=None):
        n, hq_ = x.shape[0], HEADS * GROUP
        q = torch.empty(n, hq_, 128, dtype=torch.bfloat16, device="cuda")
        k = torch.empty(HEADS, n, 128, dtype=torch.bfloat16, device="cuda")
        hq.hq_qk_norm_rope(x[:, :hq_], x[:, hq_:hq_ + HEADS].transpose(0, 1), spec, freq, q, k, w, w, positions, pos0)
        return q, k, x[:, hq_ + HEADS:].transpose(0, 1)

    def append(k, v):
        for c, x, a in zip(caches, (k, v), alpha):
            c.append(x.contiguous(), a)

    def check(q, out, mask=None, kd=None, vd=None):
        n = caches[0].tokens
        keep = T.seen(q.shape[0], n, window, sinks, mask, lambda t: t not in gone)
        kk, vv = (T.vectors(c) for c in caches)
        if kd is not None:
            kk, vv = torch.cat((kk, kd.double()), 1), torch.cat((vv, vd.double()), 1)
        T.check(out, None, q, kk, vv, keep, GROUP, SCALE, 1)

    # the prompt, then tokens one by one
    q, k, v = layer(_project(77, 1), 0)
    append(k, v)
    at = hq.KVAttention(*caches, GROUP, window=window, sinks=sinks)
    out = torch.empty(64, HEADS * GROUP, 128, dtype=torch.bfloat16, device="cuda")
    check(q[-64:], at(q[-64:], out))
    for step in range(40):
        q, k, v = layer(_project(1, 10 + step), caches[0].tokens)
        append(k, v)
        o = at(q, out[:1])
    check(q, o)
    # drafts: a small tree, of which one path is accepted
    parents = [-1, 0, 0, 2]
    mask = []
    for i, p in enumerate(parents):
        mask.append((mask[p] if p >= 0 else 0) | 1 << i)
    depth = torch.tensor([bin(m).count("1") for m in mask], device="cuda")
    q, k, v = layer(_project(4, 99), 0, caches[0].tokens - 1 + depth)
    v = v.contiguous()
    o = at.tree(q, k, v, torch.tensor(mask, device="cuda"), out[:4])
    check(q, o, mask, k, v)
    path = [0, 2, 3]
    was = caches[0].tokens
    append(k[:, path], v[:, path])
    assert caches[0].tokens == was + 3
    # evict what no later query sees, merge the one-token appends, and go on
    total = caches[0].tokens
    kept = [(0, sinks), (total - window, total)]
    fresh = make()
    for c, d in zip(caches, fresh):
        c.repack(d, kept)
    before = [c.cache.chunks for c in caches]
    caches[:] = fresh
    gone.update(range(sinks, total - window))
    assert caches[0].cache.chunks < before[0]
    at = hq.KVAttention(*caches, GROUP, window=window, sinks=sinks)
    for step in range(3):
        q, k, v = layer(_project(1, 200 + step), caches[0].tokens)
        append(k, v)
        check(q, at(q, out[:1]))
    for c in caches:
        assert hq.read_stats(c.stats)["status"] == 0
